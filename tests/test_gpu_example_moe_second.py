"""The example's layer has first derivatives only: a second one is an error, not
a result that lacks terms."""
import pytest

from test_gpu_example_moe import ex  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_second_derivative_is_refused(ex):  # noqa: F811
    import torch
    layer, g = ex.make(4, 128, 96)
    x, ids, weights = ex.route(g, 10, 128, 4, 2)
    x.requires_grad_()
    weights.requires_grad_()
    y = layer.train(x, ids, weights)
    # (terms beside the layer's, so that a missing second derivative is not an error by itself)
    loss = (y * y).sum() + (x ** 3).sum() + (weights ** 3).sum()
    dx, dw = torch.autograd.grad(loss, (x, weights), create_graph=True)
    for first, to in ((dx, x), (dw, weights)):
        with pytest.raises(RuntimeError, match="differentiate twice"):
            torch.autograd.grad(first.sum(), to, retain_graph=True)
