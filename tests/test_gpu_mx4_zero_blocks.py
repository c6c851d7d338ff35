"""Weights with blocks of zeros (padded channels, pruned weights; the quantizer gives
them the smallest scale): the scale of a zero block, NaN's aside, has no part in the
results -- in the tiles not even in how their sums are formed: f16 rows do not begin
again with more pieces.  The kernels of few rows (rows at odd addresses take them in
place of the tiles of 32 rows) choose the pieces of f16 rows step by step: two sums of the same exact terms, each off by at most (3 K / 32 + 64) 2^-23 of the
terms' magnitudes."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qp():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import conv_qpack_weights_amd as qp
    return qp


CASES = [("w4", "rows16x16", 5, 300), ("w4", "rows16x32", 30, 4010), ("w4", "rows16x48", 13, 9000),
         ("w4", "rows16x64", 61, 4030), ("w4", "tile32x64", 146, 4900),
         ("w4", "tile32x128", 500, 4010), ("w4", "tile128x128", 1100, 4010),
         ("w4", "tile128x128", 1000, 4010), ("w4", "tile256x256", 4090, 4090),
         ("w4_dx", "rows16x128", 5, 300), ("w4_dx", "tile128x128", 2100, 4010),
         ("w4_dx", "tile256x256", 4090, 4090)]


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("product,kernel,M,N", CASES)
def test_a_zero_blocks_scale_has_no_part(qp, product, kernel, M, N, dtype, odd):
    import torch
    K = 330
    g = torch.Generator().manual_seed(M + N)
    rows, cols = (K, N) if product == "w4_dx" else (N, K)     # (the gradient: N columns)
    w = torch.randn(rows, cols, generator=g).cuda()
    G = -(-cols // 32)
    # a block in a channel, a channel, the last block of all, and signed zeros
    none = torch.zeros(rows, G, dtype=torch.bool)
    none[torch.arange(rows), torch.randint(0, G, (rows,), generator=g)] = True
    none[rows // 2] = True
    none[:, G - 1] = True
    none = none.cuda()
    w[none.repeat_interleave(32, 1)[:, :cols]] *= 0.0
    W = qp.qquantize_rows_mx4(w, "ceil")
    assert (W.scales[none] == 0).all() and (W.codes.view(rows, G, 16)[none] != 0).any()
    assert qp.qgemm_mx_kernel_name(product, M, W, {"f16": torch.float16, "bf16": torch.bfloat16}[
        dtype]).split("/")[0] == kernel
    print("mx4 zero blocks", product, kernel, M, N, dtype, odd, flush=True)
    X = torch.randn(M, K + 3, generator=g).to(torch.float16 if dtype == "f16" else torch.bfloat16).cuda()
    X = X[:, 1:1 + K] if odd else X[:, :K].contiguous()
    if product == "w4_dx":
        run = lambda: qp.qgemm_w4_mx_dx(X, W)
    else:
        run = lambda: qp.qgemm_w4_mx(X, W, out_dtype=torch.float32)
    given = run()                                             # (scales as the quantizer gives them)
    W.scales[none] = 127
    plain = run()
    assert torch.isfinite(plain).all()
    steps = kernel.startswith("rows") or (odd and kernel.startswith("tile32"))
    if product == "w4" and steps and dtype == "f16":
        v = qp.qdequantize_rows_mx4(W).double()
        bound = 2 * (3 * K / 32 + 64) * 2.0 ** -23 * (X.double().abs() @ v.abs().t().contiguous())
        same = lambda a, b: bool(((a.double() - b.double()).abs() <= bound).all())
    else:
        same = torch.equal
    assert same(given, plain)
    choose = torch.randint(0, 5, (rows, G), generator=g).cuda()
    any_scale = torch.tensor([0, 1, 80, 200, 254], dtype=torch.uint8, device="cuda")[choose]
    W.scales.copy_(torch.where(none, any_scale, W.scales))
    assert same(run(), plain)


def test_a_zero_block_of_nan_scale_is_nan(qp):
    import torch
    g = torch.Generator().manual_seed(1)
    for M in (5, 300):
        W = qp.qquantize_rows_mx4(torch.randn(70, 96, generator=g).cuda())
        W.codes[3, :16] = 0
        W.scales[3, 0] = 255
        X = torch.randn(M, 96, generator=g).half().cuda()
        y = qp.qgemm_w4_mx(X, W)
        assert torch.isnan(y[:, 3]).all() and torch.isfinite(y[:, :3]).all()
        d = qp.qgemm_w4_mx_dx(torch.randn(M, 70, generator=g).half().cuda(), W)
        assert torch.isnan(d[:, :32]).all() and torch.isfinite(d[:, 32:]).all()
