"""The example's expert layer, served and trained, against the formulas in 64
bits on the same 4-bit weights.  Its bf16 steps round about six times between
x and a gradient (rows, gate, up, their product, z, y; back the same), each by
at most 2^-8 of a value and by 2^-8/sqrt(3) in the mean square of uniform
errors: 8 * 2^-8 bounds the norms with room for the cancellation between
terms; f32 sums of up to 1408 terms stay below 1408 * 2^-24 * 8."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    spec = importlib.util.spec_from_file_location(
        "moe_w4_layer", os.path.join(ROOT, "examples", "moe_w4_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("dtype,bound", [("bfloat16", 8 * 2.0 ** -8),
                                         ("float32", 8 * 1408 * 2.0 ** -24)])
@pytest.mark.parametrize("T,experts,H,F,k", [(1, 4, 128, 96, 1), (9, 8, 256, 352, 2),
                                             (200, 3, 130, 201, 3), (64, 8, 512, 1408, 2)])
def test_layer(ex, dtype, bound, T, experts, H, F, k):
    import torch
    print("expert layer", dtype, T, experts, H, F, k, flush=True)
    if T == 1:   # its only token would be the padding one: two tokens
        T = 2
    errors = ex.compare(T, experts, H, F, k, getattr(torch, dtype))
    for name, err in errors.items():
        assert err <= bound, (name, err)


def test_serving_in_a_graph(ex):
    """The serving path captured once and replayed on new tokens."""
    import torch
    layer, g = ex.make(8, 256, 352)
    x, ids, weights = ex.route(g, 12, 256, 8, 2)
    x = x.bfloat16()
    layer.serve(x, ids, weights)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.serve(x, ids, weights)
    for _ in range(3):
        x2, ids2, w2 = ex.route(g, 12, 256, 8, 2)
        x.copy_(x2.bfloat16())
        ids.copy_(ids2)
        weights.copy_(w2)
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer.serve(x, ids, weights))
