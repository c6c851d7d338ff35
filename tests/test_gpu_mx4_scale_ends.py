"""MXFP4 weights whose scales are the smallest and the largest there are, in every kernel
of the products and the gradient and with every row type: the smallest make weights that
are subnormal bf16 values, 2^-128 and up, the largest of these tests weights just below
the f32 range; they are as exact as others.  Above it (a scale of 253 or 254 and a large
code) a weight counts as infinite.  Tolerances as in test_gpu_mx4.py: rows are scaled so
that no term and no sum leaves the normal f32 range."""
import pytest

import mx4_card as card

pytestmark = pytest.mark.gpu

LOW, HIGH = (0, 3), (236, 253)


@pytest.fixture(scope="module")
def qp():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import conv_qpack_weights_amd as qp
    return qp


def _rows(g, M, K, dtype, exponent, odd):
    """Rows of about 2^exponent, none of their values below a 64th of it."""
    import torch
    x = torch.randn(M, K + 3, generator=g)
    return card.rows(torch.copysign(x.abs().clamp_min(2.0 ** -6), x) * 2.0 ** exponent, dtype, odd)


KERNELS = [("rows16x16", 5, 300), ("rows16x32", 30, 4010), ("rows16x48", 13, 9000),
           ("rows16x64", 61, 4030), ("tile32x64", 146, 4900), ("tile32x128", 500, 4010),
           ("tile128x128", 1100, 4010), ("tile128x128", 1000, 4010), ("tile256x256", 4090, 4090)]


@pytest.mark.parametrize("end", ["low", "high"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kernel,M,N", KERNELS)
def test_products(qp, kernel, M, N, dtype, end):
    import torch
    g = torch.Generator().manual_seed(M)
    K = 330
    W, w = card.matrix(qp, g, N, K, scales=LOW if end == "low" else HIGH)
    name = qp.qgemm_mx_kernel_name("w4", M, W, card.DTYPE[dtype])
    assert name == kernel or (dtype == "f32" and kernel.startswith("tile"))
    print("mx4 ends", name, M, N, dtype, end, flush=True)
    # (f16 rows at the low end: terms from 2^-128 2^3 on, sums of about 2^-114, whose
    # tolerance is far above f32's steps of 2^-149)
    exponent = {"f32": 60, "bf16": 60, "f16": 15 - 6}[dtype] if end == "low" else \
        {"f32": -60, "bf16": -60, "f16": -8}[dtype]
    for odd in (False, True):
        X, x = _rows(g, M, K, dtype, exponent, odd)
        want, size = x @ card.t(w), x.abs() @ card.t(w).abs()
        card.close(qp.qgemm_w4_mx(X, W, out_dtype=torch.float32), want, size, K, "f32", "odd=%s" % odd)


@pytest.mark.parametrize("end", ["low", "high"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kernel,M,K", [("rows16x128", 5, 300), ("rows16x128", 140, 1500),
                                        ("tile128x128", 2100, 4010), ("tile256x256", 4090, 4090)])
def test_gradient(qp, kernel, M, K, dtype, end):
    import torch
    g = torch.Generator().manual_seed(K)
    N = 330
    W, w = card.matrix(qp, g, N, K, scales=LOW if end == "low" else HIGH)
    name = qp.qgemm_mx_kernel_name("w4_dx", M, W, card.DTYPE[dtype]).split("/")[0]
    assert name == kernel or dtype == "f32"
    print("mx4 gradient ends", name, M, K, dtype, end, flush=True)
    for odd in (False, True):
        dY, dy = _rows(g, M, N, dtype, 60 if end == "low" else -60, odd)
        card.close(qp.qgemm_w4_mx_dx(dY, W), dy @ w, dy.abs() @ w.abs(), N, dtype, "odd=%s" % odd)


@pytest.mark.parametrize("a_scales,w_scales", [((0, 3), (252, 255)), ((252, 255), (0, 3)),
                                               ((236, 255), (1, 20))])
@pytest.mark.parametrize("kernel,M,N", [("rows16x16", 5, 300), ("rows16x32", 45, 4010),
                                        ("tile64x64", 250, 4010), ("tile128x128", 1100, 4010),
                                        ("tile256x256", 4090, 4090)])
def test_both_operands_at_their_ends(qp, kernel, M, N, a_scales, w_scales):
    """MXFP4 rows: the scales meet in the products, no value is formed alone."""
    import torch
    g = torch.Generator().manual_seed(N)
    K = 330
    W, w = card.matrix(qp, g, N, K, scales=w_scales)
    A, a = card.matrix(qp, g, M, K, scales=a_scales)
    assert qp.qgemm_mx_kernel_name("a4w4", M, W) == kernel
    print("mx4 both ends", kernel, M, N, a_scales, w_scales, flush=True)
    card.close(qp.qgemm_a4w4_mx(A, W), a @ card.t(w), a.abs() @ card.t(w).abs(), K,
           "f32", "a4w4")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kernel,M,N", KERNELS)
def test_weights_above_the_range(qp, kernel, M, N, dtype):
    """Their outputs are infinities or NaN -- with bf16 rows, a single one against no zero,
    the infinity of its sign -- and no others are touched."""
    import torch
    g = torch.Generator().manual_seed(M)
    K = 330
    W, w = card.matrix(qp, g, N, K)
    out = torch.tensor([1, N // 2, N - 1], device="cuda")
    W.scales[out, 3] = torch.tensor([253, 254, 254], dtype=torch.uint8, device="cuda")
    W.codes[out, 48:64] = 0
    # 6, -2 and 6 times their scales, alone in their blocks
    W.codes[out, 50] = torch.tensor([0x07, 0x0c, 0x07], dtype=torch.uint8, device="cuda")
    print("mx4 above the range", kernel, M, N, dtype, flush=True)
    X, x = _rows(g, M, K, dtype, -8, False)
    y = qp.qgemm_w4_mx(X, W, out_dtype=torch.float32)
    assert not torch.isfinite(y[:, out]).any()
    if dtype == "bf16":
        sign = torch.sign(x[:, 100, None]) * torch.tensor([1.0, -1.0, 1.0], device="cuda")
        assert torch.equal(y[:, out], (sign * float("inf")).float())
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[out] = False
    card.close(y[:, rest], x @ card.t(w[rest]), x.abs() @ card.t(w[rest]).abs(), K,
           "f32", "others")
    dY, dy = _rows(g, 20, N, dtype, -8, False)
    d = qp.qgemm_w4_mx_dx(dY, W)
    assert not torch.isfinite(d[:, 100]).any()
    cols = torch.ones(K, dtype=torch.bool, device="cuda")
    cols[96:128] = False
    v = w[:, cols]
    card.close(d[:, cols], dy @ v, dy.abs() @ v.abs(), N, dtype, "other columns")
