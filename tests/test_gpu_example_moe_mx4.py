"""The expert layer of the example with MXFP4 weights: served and trained on float
rows against the formulas in 64 bits on the same weights, and served on MXFP4 rows
step by step.

Norms of the float rows' errors: about six roundings to the type between x and a
gradient, each at most 2^-8 (bf16) of a value: 8 * 2^-8 holds with room for the
cancellation between terms; f32 sums of up to 1408 terms stay below 8 * 1408 * 2^-24.
A router weight's gradient is the single number <dy, z>, which may cancel to any
extent: |<dy, z'> - <dy, z>| <= |dy| |z' - z| <= bound |dy| |z| (Cauchy-Schwarz), so
its error is counted against |dy| |z| and not against the gradient itself.

With 4-bit rows one rounding of h may move a code of the next product by a step, so
each step is compared with the definition on the rows it got: sums of exact products
within (3 n / 32 + 64) 2^-23 of the sum of magnitudes and one rounding, the combined
rows within one rounding of each weight's product, of the k sums and of the output."""
import numpy as np
import pytest

from oracle import mx4_f64 as mx
from test_gpu_example_moe import ex  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,bound", [("bfloat16", 8 * 2.0 ** -8),
                                         ("float32", 8 * 1408 * 2.0 ** -24)])
@pytest.mark.parametrize("T,experts,H,F,k", [(2, 4, 128, 96, 1), (9, 8, 256, 352, 2),
                                             (200, 3, 130, 201, 3), (64, 8, 512, 1408, 2)])
def test_layer(ex, dtype, bound, T, experts, H, F, k):  # noqa: F811
    import torch
    print("MXFP4 expert layer", dtype, T, experts, H, F, k, flush=True)
    layer, g = ex.make(experts, H, F, mx=True)
    x, ids, weights = ex.route(g, T, H, experts, k)
    ids[0] = -1                                         # a padding token
    x = x.to(getattr(torch, dtype))
    dy = torch.randn(T, H, generator=g, device="cuda").to(x.dtype)
    x64, w64 = x.double().requires_grad_(), weights.double().requires_grad_()
    y64 = layer.dense(x64, ids, w64)
    y64.backward(dy.double())
    xt, wt = x.clone().requires_grad_(), weights.clone().requires_grad_()
    yt = layer.train(xt, ids, wt)
    yt.backward(dy)
    with torch.no_grad():
        one = torch.ones(T, 1, dtype=torch.float64, device="cuda")
        z = torch.stack([layer.dense(x64, ids[:, j:j + 1], one) for j in range(k)], dim=1)
        scale = dy.double().norm(dim=1)[:, None] * z.norm(dim=2)
        for name, got, want, size in (
                ("served", layer.serve(x, ids, weights), y64, y64.norm()),
                ("trained", yt, y64, y64.norm()), ("dx", xt.grad, x64.grad, x64.grad.norm()),
                ("dweights", wt.grad, w64.grad, scale.norm())):
            err = float((got.double() - want).norm() / size)
            print("%s %.3g" % (name, err))
            assert err <= bound, (name, err)


def _values(m):
    return mx.values(m.codes.cpu().numpy(), m.scales.cpu().numpy(), m.K)


def _product(got, rows, w, counts, eps):
    """got [M, N] against rows (f64) of sorted experts times w (f64 [E, N, K])."""
    tol = (3 * rows.shape[1] / 32 + 64) * 2.0 ** -23
    at = 0
    for e, n in enumerate(counts):
        want = rows[at:at + n] @ w[e].T
        size = np.abs(rows[at:at + n]) @ np.abs(w[e]).T
        off = np.abs(got[at:at + n].double().cpu().numpy() - want)
        assert (off <= tol * size + 1.01 * eps * np.abs(want)).all(), (e, off.max())
        at += n


@pytest.mark.parametrize("dtype,eps", [("bfloat16", 2.0 ** -8), ("float32", 2.0 ** -24)])
@pytest.mark.parametrize("T,experts,H,F,k", [(1, 4, 128, 96, 2), (9, 8, 256, 352, 2),
                                             (200, 3, 130, 201, 3), (300, 4, 512, 704, 2)])
def test_four_bit_rows_step_by_step(ex, dtype, eps, T, experts, H, F, k):  # noqa: F811
    import torch
    qp = ex.qp
    print("MXFP4 rows and weights", dtype, T, experts, H, F, k, flush=True)
    layer, g = ex.make(experts, H, F, mx=True, rows4=True)
    x, ids, weights = ex.route(g, T, H, experts, k)
    if T > 1:
        ids[0] = -1                                     # a padding token
    x = x.to(getattr(torch, dtype))
    offsets, row_of_slot, slot_of_row = qp.qmoe_sort(ids, experts)
    counts = np.diff(offsets.cpu().numpy())
    assert counts.sum() == int((ids >= 0).sum())

    a = qp.qquantize_rows_mx4(x, "ceil")
    codes, scales = mx.quantize(x.double().cpu().numpy(), ceil=True)
    assert np.array_equal(a.codes.cpu().numpy(), codes)
    assert np.array_equal(a.scales.cpu().numpy(), scales)
    M = int(counts.sum())
    token = slot_of_row.cpu().numpy()[:M] // k
    h = qp.qgemm_a4w4_mx_experts(a, layer.up, offsets, rows=slot_of_row, row_div=k,
                                 out_dtype=x.dtype)
    _product(h, _values(a)[token], _values(layer.up), counts, eps)

    act = layer._gate(h)
    b = qp.qquantize_rows_mx4(act, "ceil")
    codes, scales = mx.quantize(act[:M].double().cpu().numpy(), ceil=True)
    assert np.array_equal(b.codes[:M].cpu().numpy(), codes)
    assert np.array_equal(b.scales[:M].cpu().numpy(), scales)
    z = qp.qgemm_a4w4_mx_experts(b, layer.down, offsets, out_dtype=x.dtype)
    _product(z, _values(b)[:M], _values(layer.down), counts, eps)

    y = layer.serve(x, ids, weights)
    z64 = z.double().cpu().numpy()
    row = row_of_slot.cpu().numpy().reshape(T, k)
    w64 = weights.double().cpu().numpy()
    want = np.zeros((T, H))
    size = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            if row[t, j] >= 0:
                want[t] += w64[t, j] * z64[row[t, j]]
                size[t] += np.abs(w64[t, j] * z64[row[t, j]])
    off = np.abs(y.double().cpu().numpy() - want)
    assert (off <= (2 * k) * 2.0 ** -24 * size * 1.01 + 1.01 * eps * np.abs(want)
            + eps * 2 * k * 2.0 ** -24 * size).all(), off.max()
    if T > 1:
        assert not y[0].any()


@pytest.mark.parametrize("rows4", [False, True])
def test_serving_in_a_graph(ex, rows4):  # noqa: F811
    """Captured once, replayed on new tokens with eager calls between."""
    import torch
    layer, g = ex.make(8, 256, 352, mx=True, rows4=rows4)
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


def test_a_second_derivative_is_refused(ex):  # noqa: F811
    import torch
    layer, g = ex.make(4, 128, 96, mx=True)
    x, ids, weights = ex.route(g, 10, 128, 4, 2)
    x.requires_grad_()
    weights.requires_grad_()
    y = layer.train(x, ids, weights)
    loss = (y * y).sum() + (x ** 3).sum() + (weights ** 3).sum()
    dx, dw = torch.autograd.grad(loss, (x, weights), create_graph=True)
    for first, to in ((dx, x), (dw, weights)):
        with pytest.raises(RuntimeError, match="differentiate twice"):
            torch.autograd.grad(first.sum(), to, retain_graph=True)


def test_matrices_of_a_checkpoint(ex):  # noqa: F811
    """A layer made from codes and scales is the one that quantized them itself."""
    import torch
    first, g = ex.make(4, 128, 96, mx=True)
    again = ex.MxExpertLayer(*(ex.qp.mx4_tensor(m.codes.clone(), m.scales.contiguous(), m.K)
                               for m in (first.up, first.down)))
    x, ids, weights = ex.route(g, 10, 128, 4, 2)
    assert torch.equal(first.serve(x, ids, weights), again.serve(x, ids, weights))
