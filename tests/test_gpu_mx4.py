"""MXFP4 rows (qquantize_rows_mx4, qdequantize_rows_mx4) and the products with
MXFP4 weights (qgemm_a4w4_mx*, qgemm_w4_mx*, their gradients) against the
definitions in 64 bits.

Quantization is exact: codes and scales are compared bit by bit.  Tolerances of
the products, per output: every product of two values is exact, the sums are f32.
With A the sum of the terms' magnitudes, each addition is off by at most 2^-23 A
(were it to truncate); a term passes at most 32 additions inside an MFMA step,
then one per further step of 32 (each piece of f32 and f16 rows one of its own,
3 at most) and a few across waves: 3 n / 32 + 64 for a sum of n terms.  Then one
rounding to the output type: 2^-8 (bf16) or 2^-11 (f16, 2^-25 among its
subnormals) of the value."""
import numpy as np
import pytest

from oracle import mx4_f64 as mx

pytestmark = pytest.mark.gpu

ROUND = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TYPES = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module")
def qp():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import conv_qpack_weights_amd as qp
    return qp


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def _rows(rng, M, K, dtype, scale=1.0):
    """Random rows of the type, on the device, and the same values in f64."""
    import torch
    x = torch.from_numpy(rng.standard_normal((M, K)) * scale).to(_dt(dtype))
    return x.cuda(), x.double().numpy()


def _matrix(qp, rng, *shape, scales=(118, 130)):
    """A random MX4 of any codes, and its values in f64."""
    import torch
    *lead, K = shape
    G = -(-K // 32)
    codes = rng.integers(0, 256, (*lead, 16 * G)).astype(np.uint8)
    if K % 32:  # the values past K are zeros
        both = np.stack((codes & 15, codes >> 4), axis=-1).reshape(*lead, 32 * G)
        both[..., K:] = 0
        codes = (both[..., 0::2] | (both[..., 1::2] << 4)).astype(np.uint8)
    s = rng.integers(scales[0], scales[1], (*lead, G)).astype(np.uint8)
    return qp.mx4_tensor(torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda(), K), \
        mx.values(codes, s, K)


def _close(got, want, A, terms, dtype, what):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), what
    tol = (3 * terms / 32 + 64) * 2.0 ** -23 * A + ROUND[dtype] * np.abs(want) * 1.01 \
        + (2.0 ** -25 if dtype == "f16" else 0.0)
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%s: %d outputs off, worst by %.3g of its tolerance" % (
        what, bad.sum(), float((np.abs(got - want) / np.maximum(tol, 1e-300)).max()))


# ------------------------------------------------------------ rows to MXFP4 and back
def _hard_rows(dtype):
    """Values on and beside every border, at every exponent of the type."""
    import torch
    t = _dt(dtype)
    edge = [0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0, 7.5]
    lo, hi = {"f32": (-151, 126), "bf16": (-135, 126), "f16": (-27, 14)}[dtype]
    rows = []
    for e in range(lo, hi):
        v = [s * x for x in edge for s in (1.0, -1.0)]
        v = (torch.tensor(v[:32], dtype=torch.float64) * 2.0 ** (e - 2)).to(t)
        up = torch.nextafter(v.float(), torch.full_like(v.float(), 9e30)).to(t)
        rows.append(torch.cat((v, up, v * 0, v.flip(0))))
    return torch.stack(rows)


@pytest.mark.parametrize("rule", ["floor", "ceil"])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_borders(qp, dtype, rule):
    import torch
    x = _hard_rows(dtype)
    # each block's exponent is that of its own largest value: the tied values in it
    # are cut at a few different exponents
    for most in (1.0, 0.25, 4.0):
        y = (x.double() * most).to(x.dtype)
        y = torch.where(torch.isfinite(y), y, torch.zeros_like(y))
        q = qp.qquantize_rows_mx4(y.cuda(), rule=rule)
        codes, scales = mx.quantize(y.double().numpy(), rule == "ceil")
        assert np.array_equal(q.scales.cpu().numpy(), scales)
        assert np.array_equal(q.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("rule", ["floor", "ceil"])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_shapes(qp, dtype, rule):
    rng = np.random.default_rng(7)
    for M, K in [(1, 1), (1, 31), (3, 32), (2, 33), (5, 64), (7, 100), (37, 129), (1, 512),
                 (300, 1100), (2, 8192), (4097, 96), (70000, 40)]:
        print("mx4 quantize", dtype, rule, M, K, flush=True)
        x, ref = _rows(rng, M, K, dtype, 3.0)
        q = qp.qquantize_rows_mx4(x, rule=rule)
        codes, scales = mx.quantize(ref, rule == "ceil")
        assert q.shape == (M, K)
        assert np.array_equal(q.scales.cpu().numpy(), scales)
        assert np.array_equal(q.codes.cpu().numpy(), codes)


def test_quantize_special_values(qp):
    """Infinities and NaN make their own block NaN; zeros of both signs; the
    smallest and largest values."""
    import torch
    x = torch.zeros(9, 96)
    x[1, 40] = float("inf")
    x[2, 40] = float("-inf")
    x[3, 40] = float("nan")
    x[4, 33] = -0.0
    x[5, 95] = 1e-45
    x[6, 32] = 3.4028234e38
    x[7, 63], x[7, 62] = 1.1754944e-38, -5e-39
    x[:4, :32] = 1.5
    x[8] = -6.0
    q = qp.qquantize_rows_mx4(x.cuda())
    codes, scales = mx.quantize(x.double().numpy())
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    y = qp.qdequantize_rows_mx4(q).cpu().numpy()
    want = mx.values(codes, scales, 96).astype(np.float32)
    assert np.array_equal(y, want, equal_nan=True)
    assert np.isnan(y[1:4, 32:64]).all() and np.isfinite(y[1:4, :32]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_strides_and_what_is_left_alone(qp, dtype):
    """Rows of a wider matrix at an odd offset; results into wider rows, whose other
    bytes stay; no rows."""
    import torch
    rng = np.random.default_rng(3)
    big, _ = _rows(rng, 20, 301, dtype)
    x = big[:, 3:3 + 200]
    codes = torch.full((20, 160), 0xa5, dtype=torch.uint8, device="cuda")
    scales = torch.full((20, 12), 0xa5, dtype=torch.uint8, device="cuda")
    out = qp.MX4(codes[:, :112], scales[:, :7], 200)
    q = qp.qquantize_rows_mx4(x, out=out)
    assert q is out
    c, s = mx.quantize(x.double().cpu().numpy())
    assert np.array_equal(codes[:, :112].cpu().numpy(), c)
    assert np.array_equal(scales[:, :7].cpu().numpy(), s)
    assert (codes[:, 112:] == 0xa5).all() and (scales[:, 7:] == 0xa5).all()
    wide = torch.full((20, 222), 9.0, dtype=_dt(dtype), device="cuda")
    qp.qdequantize_rows_mx4(q, dtype=_dt(dtype), out=wide[:, 1:201])
    assert np.array_equal(wide[:, 1:201].double().cpu().numpy(), mx.values(c, s, 200))
    assert (wide[:, :1] == 9).all() and (wide[:, 201:] == 9).all()
    none = qp.qquantize_rows_mx4(x[:0])
    assert none.shape == (0, 200) and qp.qdequantize_rows_mx4(none).shape == (0, 200)
    e = qp.qquantize_rows_mx4(x.contiguous().view(4, 5, 200))
    assert e.shape == (4, 5, 200)
    assert np.array_equal(e.codes.cpu().numpy().reshape(20, -1), c)
    assert np.array_equal(e[2].scales.cpu().numpy(), s[10:15])


@pytest.mark.parametrize("dtype", TYPES)
def test_every_code_and_scale_back(qp, dtype):
    import torch
    codes = np.arange(256, dtype=np.uint8)[None, :].repeat(256, 0)   # 16 blocks
    scales = np.arange(256, dtype=np.uint8)[:, None].repeat(16, 1)
    q = qp.mx4_tensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    got = qp.qdequantize_rows_mx4(q, dtype=_dt(dtype)).cpu()
    want = torch.from_numpy(mx.values(codes, scales, 512)).to(_dt(dtype))  # one rounding
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, 7.0), torch.nan_to_num(want, 7.0))


def test_layouts_that_checkpoints_hold(qp):
    """Odd block counts, offsets and strides are laid out anew; what fits is kept."""
    import torch
    rng = np.random.default_rng(5)
    codes = torch.from_numpy(rng.integers(0, 256, (6, 9, 16 * 5)).astype(np.uint8)).cuda()
    scales = torch.from_numpy(rng.integers(110, 135, (6, 9, 5)).astype(np.uint8)).cuda()
    want = mx.values(codes.cpu().numpy(), scales.cpu().numpy(), 160)
    w = qp.mx4_tensor(codes, scales)
    for e in (0, 5):
        assert np.array_equal(qp.qdequantize_rows_mx4(w[e]).double().cpu().numpy(), want[e])
    assert w.codes.data_ptr() == codes.data_ptr()
    one = qp.mx4_tensor(codes[1, ::2], scales[1, ::2])
    assert np.array_equal(qp.qdequantize_rows_mx4(one).double().cpu().numpy(), want[1, ::2])
    flat = codes.reshape(-1)
    shifted = torch.empty(flat.numel() + 3, dtype=torch.uint8, device="cuda")[3:]
    shifted.copy_(flat)
    odd = qp.mx4_tensor(shifted.view(6, 9, 80)[2], scales[2].t().contiguous().t())
    assert np.array_equal(qp.qdequantize_rows_mx4(odd).double().cpu().numpy(), want[2])


# ------------------------------------------------------------ products and gradients
# K and N off every tile edge; a row up to several tiles
SHAPES = [(1, 1, 1), (1, 16, 32), (1, 70, 129), (2, 64, 128), (5, 130, 1000), (16, 200, 512),
          (17, 48, 640), (33, 100, 257), (64, 64, 96), (130, 257, 390), (257, 300, 1056),
          (600, 513, 288)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_dense_products_and_gradient(qp, dtype, M, N, K):
    import torch
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    print("mx4 products", dtype, M, N, K, flush=True)
    W, w = _matrix(qp, rng, N, K)
    A, a = _matrix(qp, rng, M, K)
    bias = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).cuda()
    b = bias.double().cpu().numpy()
    mag = np.abs(a) @ np.abs(w).T + np.abs(b)
    Y = qp.qgemm_a4w4_mx(A, W, bias, out_dtype=_dt(dtype))
    assert Y.dtype == _dt(dtype)
    _close(Y, a @ w.T + b, mag, K, dtype, "a4w4")
    Y32 = qp.qgemm_a4w4_mx(A, W, bias)
    Yc = qp.qgemm_a4w4_mx(A, W, bias, -0.5, 0.25, out_dtype=_dt(dtype))
    assert torch.equal(Yc, torch.clamp(Y32, -0.5, 0.25).to(_dt(dtype)))

    X, x = _rows(rng, M, K, dtype)
    mag = np.abs(x) @ np.abs(w).T + np.abs(b)
    Y = qp.qgemm_w4_mx(X, W, bias)
    assert Y.dtype == X.dtype
    _close(Y, x @ w.T + b, mag, K, dtype, "w4")
    Y32 = qp.qgemm_w4_mx(X, W, bias, out_dtype=torch.float32)
    _close(Y32, x @ w.T + b, mag, K, "f32", "w4 in f32")
    assert torch.equal(qp.qgemm_w4_mx(X, W, bias, -0.5, 0.25),
                       torch.clamp(Y32, -0.5, 0.25).to(X.dtype))
    _close(qp.qgemm_w4_mx(X, W), x @ w.T, mag, K, dtype, "w4 without bias")

    dY, dy = _rows(rng, M, N, dtype)
    _close(qp.qgemm_w4_mx_dx(dY, W), dy @ w, np.abs(dy) @ np.abs(w), N, dtype, "dx")


@pytest.mark.parametrize("dtype,M,N,K", [
    ("bf16", 1, 4096, 4096), ("f32", 1, 1030, 11008), ("f16", 16, 1024, 4096),
    ("bf16", 300, 512, 2048), ("f16", 1025, 300, 1100), ("bf16", 1024, 768, 2048),
    ("f32", 260, 320, 2048), ("bf16", 2050, 520, 544)])
def test_larger_shapes(qp, dtype, M, N, K):
    rng = np.random.default_rng(M + N + K)
    print("mx4 larger", dtype, M, N, K, flush=True)
    W, w = _matrix(qp, rng, N, K)
    A, a = _matrix(qp, rng, M, K)
    _close(qp.qgemm_a4w4_mx(A, W, out_dtype=_dt(dtype)), a @ w.T, np.abs(a) @ np.abs(w).T, K,
           dtype, "a4w4")
    X, x = _rows(rng, M, K, dtype)
    _close(qp.qgemm_w4_mx(X, W), x @ w.T, np.abs(x) @ np.abs(w).T, K, dtype, "w4")
    dY, dy = _rows(rng, M, N, dtype)
    _close(qp.qgemm_w4_mx_dx(dY, W), dy @ w, np.abs(dy) @ np.abs(w), N, dtype, "dx")


def _counts(kind, E, M, rng):
    if kind == "even":
        c = [M // E] * E
    elif kind == "one":
        c = [0] * E
        c[E // 2] = M - 3
    else:
        cut = np.sort(rng.integers(0, M + 1, E))
        c = np.diff(np.concatenate(([0], cut))).tolist()
        c[0] = 0
    return c


@pytest.mark.parametrize("kind", ["even", "one", "ragged"])
@pytest.mark.parametrize("dtype", TYPES)
def test_experts(qp, dtype, kind):
    """Rows by expert, sorted and through the map; experts without rows; rows past the
    last expert's; slots that are no row."""
    import torch
    for E, M, T, N, K in [(3, 40, 20, 70, 100), (8, 300, 150, 130, 256), (5, 700, 350, 300, 544),
                          (70, 90, 45, 33, 64)]:
        rng = np.random.default_rng(E * 1000 + M)
        print("mx4 experts", dtype, kind, E, M, N, K, flush=True)
        W, w = _matrix(qp, rng, E, N, K)
        c = _counts(kind, E, M, rng)
        off = np.concatenate(([0], np.cumsum(c))).astype(np.int32)
        offsets = torch.from_numpy(off).cuda()
        bias = torch.from_numpy(rng.standard_normal((E, N)).astype(np.float32)).cuda()
        b = bias.double().cpu().numpy()
        rows = rng.integers(0, 2 * T, M).astype(np.int32)
        rows[3], rows[-1] = -1, 2 * T + 5
        src = np.where((rows >= 0) & (rows < 2 * T), rows // 2, -1)
        drows = torch.from_numpy(rows).cuda()

        def expect(x, mapped):
            y, mag = np.zeros((M, N)), np.zeros((M, N))
            for e in range(E):
                for r in range(off[e], off[e + 1]):
                    v = x[src[r]] if mapped and src[r] >= 0 else \
                        np.zeros(K) if mapped else x[r]
                    y[r] = w[e] @ v + b[e]
                    mag[r] = np.abs(w[e]) @ np.abs(v) + np.abs(b[e])
            return y, mag

        A, a = _matrix(qp, rng, M, K)
        want, mag = expect(a, False)
        _close(qp.qgemm_a4w4_mx_experts(A, W, offsets, bias, out_dtype=_dt(dtype)), want, mag, K,
               dtype, "a4w4")
        A, a = _matrix(qp, rng, T, K)
        want, mag = expect(a, True)
        _close(qp.qgemm_a4w4_mx_experts(A, W, offsets, bias, drows, 2, out_dtype=_dt(dtype)), want,
               mag, K, dtype, "a4w4 through the map")
        X, x = _rows(rng, M, K, dtype)
        want, mag = expect(x, False)
        _close(qp.qgemm_w4_mx_experts(X, W, offsets, bias), want, mag, K, dtype, "w4")
        X, x = _rows(rng, T, K, dtype)
        want, mag = expect(x, True)
        _close(qp.qgemm_w4_mx_experts(X, W, offsets, bias, drows, 2), want, mag, K, dtype,
               "w4 through the map")
        dY, dy = _rows(rng, M, N, dtype)
        want, mag = np.zeros((M, K)), np.zeros((M, K))
        for e in range(E):
            s = slice(off[e], off[e + 1])
            want[s], mag[s] = dy[s] @ w[e], np.abs(dy[s]) @ np.abs(w[e])
        _close(qp.qgemm_w4_mx_experts_dx(dY, W, offsets), want, mag, N, dtype, "dx")


def test_offsets_outside_the_rows(qp):
    """Offsets that fall or leave [0, M] are taken at their nearest bounds."""
    import torch
    rng = np.random.default_rng(11)
    W, w = _matrix(qp, rng, 3, 40, 64)
    X, x = _rows(rng, 50, 64, "bf16")
    A = qp.qquantize_rows_mx4(X)
    a = mx.values(A.codes.cpu().numpy(), A.scales.cpu().numpy(), 64)
    dY, dy = _rows(rng, 50, 40, "bf16")
    for off, parts in [([0, 10, 99, 200], [(0, 10), (10, 50), (50, 50)]),
                       ([-5, 20, 20, 30], [(0, 20), (20, 20), (20, 30)])]:
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        y = qp.qgemm_w4_mx_experts(X, W, offsets)
        z = qp.qgemm_a4w4_mx_experts(A, W, offsets)
        d = qp.qgemm_w4_mx_experts_dx(dY, W, offsets)
        end = 0
        for e, (r0, r1) in enumerate(parts):
            s, end = slice(r0, r1), max(end, r1)
            _close(y[s], x[s] @ w[e].T, np.abs(x[s]) @ np.abs(w[e]).T, 64, "bf16", "w4")
            _close(z[s], a[s] @ w[e].T, np.abs(a[s]) @ np.abs(w[e]).T, 64, "f32", "a4w4")
            _close(d[s], dy[s] @ w[e], np.abs(dy[s]) @ np.abs(w[e]), 40, "bf16", "dx")
        assert (y[end:] == 0).all() and (z[end:] == 0).all() and (d[end:] == 0).all()


@pytest.mark.parametrize("M", [2, 300])
def test_nan_blocks_and_infinite_rows_stay_where_they_are(qp, M):
    """A NaN block of the weights reaches its channel alone, a NaN or an infinity of
    a row its row alone; padding bytes behind a row's scales reach nothing."""
    import torch
    rng = np.random.default_rng(M)
    N, K = 150, 330                                     # 11 blocks: one byte behind them
    W, w = _matrix(qp, rng, N, K)
    base = W.scales.as_strided((N, 12), (12, 1))
    base[:, 11] = 255
    W.scales[N - 1, 10] = 255                           # last channel, last block
    W.scales[7, 0] = 255
    ok_n = np.ones(N, bool)
    ok_n[[7, N - 1]] = False
    A, a = _matrix(qp, rng, M, K)
    A.scales.as_strided((M, 12), (12, 1))[:, 11] = 255
    A.scales[M - 1, 10] = 255
    ok_m = np.arange(M) != M - 1
    y = qp.qgemm_a4w4_mx(A, W).cpu()
    assert torch.isnan(y[:, ~ok_n]).all() and torch.isnan(y[M - 1]).all()
    sub = np.ix_(ok_m, ok_n)
    _close(y[sub], (a @ w.T)[sub], (np.abs(a) @ np.abs(w).T)[sub], K, "f32", "a4w4")
    for dtype in TYPES:
        X, x = _rows(rng, M, K, dtype)
        X[M - 1, K - 1] = float("inf")
        y = qp.qgemm_w4_mx(X, W, out_dtype=torch.float32).cpu()
        assert torch.isnan(y[:, ~ok_n]).all()
        bad = ~torch.isfinite(y[M - 1])
        assert (bad | (torch.from_numpy(w[:, K - 1]) == 0)).all()
        _close(y[sub], (x @ w.T)[sub], (np.abs(x) @ np.abs(w).T)[sub], K, "f32", "w4")
        # a channel's NaN block reaches its 32 columns of every row
        dY, dy = _rows(rng, M, N, dtype)
        dY[M - 1, 0] = float("nan")
        d = qp.qgemm_w4_mx_dx(dY, W).float().cpu()
        assert torch.isnan(d[M - 1]).all()
        assert torch.isnan(d[:, :32]).all() and torch.isnan(d[:, 320:]).all()
        cols = np.zeros(K, bool)
        cols[32:320] = True
        sub_d = np.ix_(ok_m, cols)
        _close(d[sub_d], (dy @ w)[sub_d], (np.abs(dy) @ np.abs(w))[sub_d], N, dtype, "dx")


@pytest.mark.parametrize("M", [3, 300])
def test_scales_at_the_ends(qp, M):
    """Scales far from 127, up to the ends of f32, in both operands."""
    rng = np.random.default_rng(M)
    N, K = 70, 200
    W, w = _matrix(qp, rng, N, K, scales=(0, 30))
    A, a = _matrix(qp, rng, M, K, scales=(200, 225))
    _close(qp.qgemm_a4w4_mx(A, W), a @ w.T, np.abs(a) @ np.abs(w).T, K, "f32", "a4w4")
    for dtype, scale in (("f32", 2.0 ** 100), ("bf16", 2.0 ** 100), ("f16", 1000.0)):
        X, x = _rows(rng, M, K, dtype, scale)
        W, w = _matrix(qp, rng, N, K, scales=(20, 30))
        import torch
        _close(qp.qgemm_w4_mx(X, W, out_dtype=torch.float32), x @ w.T, np.abs(x) @ np.abs(w).T, K,
               "f32", "w4")
    W, w = _matrix(qp, rng, N, K, scales=(220, 235))
    X, x = _rows(rng, M, K, "bf16", 2.0 ** -60)
    _close(qp.qgemm_w4_mx(X, W), x @ w.T, np.abs(x) @ np.abs(w).T, K, "bf16", "w4")
    dY, dy = _rows(rng, M, N, "bf16", 2.0 ** -60)
    _close(qp.qgemm_w4_mx_dx(dY, W), dy @ w, np.abs(dy) @ np.abs(w), N, "bf16", "dx")


@pytest.mark.parametrize("M", [5, 270])
def test_strided_operands_and_outputs(qp, M):
    """Rows of wider matrices, weights as rows of wider codes; what lies beside the
    outputs stays."""
    import torch
    rng = np.random.default_rng(M)
    N, K = 90, 160
    big, v = _matrix(qp, rng, N, 512)
    W = qp.MX4(big.codes[:, 64:144], big.scales[:, 4:9], K)
    w = v[:, 128:288]
    for dtype in TYPES:
        wide, _ = _rows(rng, M, K + 9, dtype)
        X = wide[:, 5:5 + K]
        x = X.double().cpu().numpy()
        Y = torch.full((M, N + 7), 9.0, dtype=_dt(dtype), device="cuda")
        qp.qgemm_w4_mx(X, W, out=Y[:, 3:3 + N])
        _close(Y[:, 3:3 + N], x @ w.T, np.abs(x) @ np.abs(w).T, K, dtype, "w4")
        assert (Y[:, :3] == 9).all() and (Y[:, 3 + N:] == 9).all()
        A = qp.qquantize_rows_mx4(X)
        a = mx.values(A.codes.cpu().numpy(), A.scales.cpu().numpy(), K)
        Y.fill_(9.0)
        qp.qgemm_a4w4_mx(A, W, out=Y[:, 3:3 + N])
        _close(Y[:, 3:3 + N], a @ w.T, np.abs(a) @ np.abs(w).T, K, dtype, "a4w4")
        assert (Y[:, :3] == 9).all() and (Y[:, 3 + N:] == 9).all()
        wide, _ = _rows(rng, M, N + 4, dtype)
        dY = wide[:, 1:1 + N]
        dy = dY.double().cpu().numpy()
        D = torch.full((M, K + 5), 9.0, dtype=_dt(dtype), device="cuda")
        qp.qgemm_w4_mx_dx(dY, W, out=D[:, 1:1 + K])
        _close(D[:, 1:1 + K], dy @ w, np.abs(dy) @ np.abs(w), N, dtype, "dx")
        assert (D[:, :1] == 9).all() and (D[:, 1 + K:] == 9).all()


def test_no_rows(qp):
    import torch
    rng = np.random.default_rng(0)
    W, _ = _matrix(qp, rng, 40, 64)
    X = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert qp.qgemm_w4_mx(X, W).shape == (0, 40)
    assert qp.qgemm_a4w4_mx(qp.qquantize_rows_mx4(X), W).shape == (0, 40)
    assert qp.qgemm_w4_mx_dx(X[:, :40], W).shape == (0, 64)


def test_same_bits_on_another_stream_and_replayed(qp):
    """The operators captured into one graph with buffers of their own, replayed
    between eager work, and on a stream of their own: the same bits every time."""
    import torch
    rng = np.random.default_rng(2)
    E, N, K = 4, 200, 288
    W, _ = _matrix(qp, rng, E, N, K)
    for M in (6, 520):
        X, _ = _rows(rng, M, K, "bf16")
        offsets = torch.tensor([0, M // 4, M // 4, M // 2, M], dtype=torch.int32, device="cuda")

        def run():
            A = qp.qquantize_rows_mx4(X)
            Y = qp.qgemm_a4w4_mx_experts(A, W, offsets, out_dtype=torch.bfloat16)
            Z = qp.qgemm_w4_mx_experts(X, W, offsets)
            D = qp.qgemm_w4_mx_experts_dx(Z, W, offsets)
            return [qp.qdequantize_rows_mx4(A), Y, Z, D, qp.qgemm_a4w4_mx(A, W[1]),
                    qp.qgemm_w4_mx(X, W[2]), qp.qgemm_w4_mx_dx(Y, W[3])]

        eager = run()
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(eager, run()))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, other))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = run()
        for turn in range(4):
            X.copy_(torch.randn_like(X) if turn % 2 else X * 0.5)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(run(), held)), turn


def test_gradient_against_differences(qp):
    """dx is what small steps of a row change in <dy, y>."""
    import torch
    rng = np.random.default_rng(9)
    W, _ = _matrix(qp, rng, 60, 96)
    X, _ = _rows(rng, 4, 96, "f32")
    dY, _ = _rows(rng, 4, 60, "f32")
    D = qp.qgemm_w4_mx_dx(dY, W)
    Y = qp.qgemm_w4_mx(X, W).double()
    for k in (0, 31, 32, 95):
        step = X.clone()
        step[:, k] += 0.5
        h = (step[:, k] - X[:, k]).double()
        slope = ((qp.qgemm_w4_mx(step, W).double() - Y) * dY.double()).sum(1) / h
        # linear: only the f32 sums' error is left, 2 sums of magnitude below 2000
        # over a step of one half
        assert torch.allclose(slope, D[:, k].double(), rtol=1e-4, atol=2000 * 96 * 2.0 ** -22)


@pytest.mark.parametrize("M", [4, 140, 520])
@pytest.mark.parametrize("scales", [(104, 112), (103, 112), (133, 141), (133, 142), (100, 140)])
def test_f16_rows_where_weights_stop_being_f16_values(qp, M, scales):
    """Block scales of 2^-23 to 2^13 make every weight an f16, scales beyond do not:
    as exact on both sides."""
    import torch
    rng = np.random.default_rng(M + scales[0])
    for N, K in [(70, 256), (300, 416)]:
        W, w = _matrix(qp, rng, N, K, scales=scales)
        X, x = _rows(rng, M, K, "f16", 0.01)
        _close(qp.qgemm_w4_mx(X, W, out_dtype=torch.float32), x @ w.T, np.abs(x) @ np.abs(w).T, K,
               "f32", "w4")
