"""The weight-only int4 products (qgemm_w4_blockwise, qgemm_w4_experts) and
their gradients to the rows against the formulas in 64 bits.

Tolerances, per output: the sums are f32.  A sum of n terms in any order is
within n * 2^-24 * A of the exact one, A the sum of the terms' magnitudes;
here a term passes at most 32 additions inside an MFMA step, one per further
step and a few across waves, so n = K/32 + 64.  Then one rounding to the
output type: 2^-8 (bf16) or 2^-11 (f16, 2^-25 among its subnormals) of the
value.  The gradient also forms each term to within 2^-15 (2^-22 for f32)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROUND = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module")
def qp():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import conv_qpack_weights_amd as qp
    return qp


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


class Case:
    """Weights of E experts: packed on the device, dense in f64 on the host."""

    def __init__(self, qp, E, N, K, group, kind, seed=0):
        import torch
        rng = np.random.default_rng(seed * 7919 + N * 31 + K)
        G = -(-K // group)
        q = rng.integers(-8, 8, (E, N, K)).astype(np.int8)
        s = rng.uniform(0.001, 0.02, (E, N, G)).astype(np.float32)
        off = rng.uniform(-0.02, 0.02, (E, N, G)).astype(np.float32) if kind == "asym" else None
        if kind == "bf16":
            s = torch.from_numpy(s).to(torch.bfloat16).float().numpy()
        of_k = np.arange(K) // group
        self.W = s[:, :, of_k].astype(np.float64) * q
        if off is not None:
            self.W = self.W + off[:, :, of_k]
        self.E, self.N, self.K, self.group = E, N, K, group
        d = lambda a: None if a is None else torch.from_numpy(a).cuda()
        self.blobs, self.info = qp.pack_s4_experts(d(q), d(s), group,
                                                   "bf16" if kind == "bf16" else "f32", d(off))
        self.bias = rng.standard_normal((E, N)).astype(np.float32)
        self.rng = rng

    def rows(self, M, width, dtype, scale=1.0):
        """Random rows of the type, on the device, and the same values in f64."""
        import torch
        x = torch.from_numpy(self.rng.standard_normal((M, width)) * scale).to(_dt(dtype))
        return x.cuda(), x.double().numpy()


def _close(got, want, A, terms, dtype, what, term_rel=0.0):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    tol = (terms / 32 + 64) * 2.0 ** -24 * A + term_rel * A + ROUND[dtype] * np.abs(want) * 1.01 \
        + (2.0 ** -25 if dtype == "f16" else 0.0)
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%s: %d outputs off, worst by %.3g of its tolerance" % (
        what, bad.sum(), float((np.abs(got - want) / tol).max()))


# every row type, scale kind and group; K and N off every tile edge
SHAPES = [(1, 16, 32), (1, 70, 129), (2, 64, 128), (5, 130, 1000), (16, 200, 512), (17, 48, 640),
          (33, 100, 257), (64, 64, 96), (130, 257, 390)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["f32", "bf16", "asym"])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
def test_dense_product_and_gradient(qp, dtype, kind, group):
    for M, N, K in SHAPES:
        c = Case(qp, 1, N, K, group, kind)
        print("w4", dtype, kind, group, M, N, K, flush=True)
        X, x = c.rows(M, K, dtype)
        W = c.W[0]
        import torch
        bias = torch.from_numpy(c.bias[0]).cuda()
        want = x @ W.T + c.bias[0]
        A = np.abs(x) @ np.abs(W).T + np.abs(c.bias[0])
        if kind == "asym":  # q and the offset are summed apart
            A = A + 2 * np.abs(x) @ np.full((K, 1), 0.18)
        Y = qp.qgemm_w4_blockwise(X, c.blobs[0], c.info, bias)
        assert Y.dtype == X.dtype
        _close(Y, want, A, K, dtype, "y")
        Y32 = qp.qgemm_w4_blockwise(X, c.blobs[0], c.info, bias, out_dtype=torch.float32)
        _close(Y32, want, A, K, "f32", "y in f32")
        lo, hi = -0.5, 0.25
        Yc = qp.qgemm_w4_blockwise(X, c.blobs[0], c.info, bias, lo, hi)
        assert torch.equal(Yc, torch.clamp(Y32, lo, hi).to(X.dtype))
        dY, dy = c.rows(M, N, dtype)
        dX = qp.qgemm_w4_blockwise_dx(dY, c.blobs[0], c.info)
        _close(dX, dy @ W, np.abs(dy) @ np.abs(W), N, dtype, "dx",
               2.0 ** -22 if dtype == "f32" else 2.0 ** -15)


@pytest.mark.parametrize("dtype,M,N,K,group", [
    ("bf16", 1, 4096, 4096, 32), ("bf16", 300, 512, 1024, 32), ("f16", 16, 1024, 4096, 128),
    ("f32", 70, 320, 2048, 64), ("bf16", 1024, 768, 2048, 32), ("bf16", 1025, 300, 1100, 128)])
def test_larger_shapes(qp, dtype, M, N, K, group):
    c = Case(qp, 1, N, K, group, "f32")
    print("w4 larger", dtype, M, N, K, group, flush=True)
    X, x = c.rows(M, K, dtype)
    W = c.W[0]
    _close(qp.qgemm_w4_blockwise(X, c.blobs[0], c.info), x @ W.T, np.abs(x) @ np.abs(W).T, K,
           dtype, "y")
    dY, dy = c.rows(M, N, dtype)
    _close(qp.qgemm_w4_blockwise_dx(dY, c.blobs[0], c.info), dy @ W, np.abs(dy) @ np.abs(W), N,
           dtype, "dx", 2.0 ** -22 if dtype == "f32" else 2.0 ** -15)


# the kernels for many rows: 128-row tiles, cut at every edge
@pytest.mark.parametrize("dtype,kind,group,counts,N,K", [
    ("bf16", "f32", 32, [700, 0, 1300, 129], 1100, 1090),
    ("f16", "f32", 128, [700, 0, 1300, 129], 1100, 1090),
    ("bf16", "asym", 64, [513, 1000], 1030, 1217),
    ("bf16", "bf16", 32, [2100, 1, 1900], 517, 4100),
    ("f32", "f32", 32, [600, 90], 300, 700)])
def test_many_rows(qp, dtype, kind, group, counts, N, K):
    import torch
    E, M = len(counts), sum(counts) + 3
    c = Case(qp, E, N, K, group, kind)
    print("w4 many rows", dtype, kind, group, counts, N, K, flush=True)
    first = np.concatenate([[0], np.cumsum(counts)])
    offsets = torch.tensor(first, dtype=torch.int32).cuda()
    perm = c.rng.permutation(M).astype(np.int32)
    X, x = c.rows(M, K, dtype)
    dY, dy = c.rows(M, N, dtype)
    asym = 0.04 if kind == "asym" else 0.0   # q and the offset are summed apart
    want, A = np.zeros((M, N)), np.zeros((M, N))
    wmap, Amap = np.zeros((M, N)), np.zeros((M, N))
    dwant, dA = np.zeros((M, K)), np.zeros((M, K))
    for e in range(E):
        r = slice(first[e], first[e + 1])
        W, aW = c.W[e], np.abs(c.W[e])
        want[r], A[r] = x[r] @ W.T, np.abs(x[r]) @ (aW + asym).T
        wmap[r], Amap[r] = x[perm[r]] @ W.T, np.abs(x[perm[r]]) @ (aW + asym).T
        dwant[r], dA[r] = dy[r] @ W, np.abs(dy[r]) @ aW
    _close(qp.qgemm_w4_experts(X, c.blobs, c.info, offsets), want, A, K, dtype, "y")
    _close(qp.qgemm_w4_experts(X, c.blobs, c.info, offsets, rows=torch.from_numpy(perm).cuda()),
           wmap, Amap, K, dtype, "y through the map")
    _close(qp.qgemm_w4_experts_dx(dY, c.blobs, c.info, offsets), dwant, dA, N, dtype, "dx",
           2.0 ** -22 if dtype == "f32" else 2.0 ** -15)


COUNTS = [
    [0, 0, 5, 0],              # one expert with rows
    [1, 1, 1, 1],
    [0, 33, 1, 0, 16, 17, 0],
    [129, 0, 64, 300, 15],
    [2] * 70,                  # more experts than lanes in a wave
    [0, 0, 0],                 # no rows at all but those of no expert
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("spare", [0, 7, 40])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "x".join(map(str, c[:7])))
def test_experts(qp, dtype, spare, counts):
    """Rows of experts, experts without rows, rows of no expert (`spare`),
    rows read through a map with entries that name no row."""
    import torch
    E = len(counts)
    N, K = 80, 300
    c = Case(qp, E, N, K, 32, "f32")
    M = sum(counts) + spare
    if M == 0:
        pytest.skip("no rows")
    print("experts", dtype, spare, counts, flush=True)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
    expert = np.repeat(np.arange(E), counts)
    n = expert.size
    X, x = c.rows(M, K, dtype)
    bias = torch.from_numpy(c.bias).cuda()

    def want_of(rows, W):
        w = np.zeros((M, W.shape[1])), np.zeros((M, W.shape[1]))
        for r in range(n):
            w[0][r] = W[expert[r]] @ rows[r]
            w[1][r] = np.abs(W[expert[r]]) @ np.abs(rows[r])
        return w

    want, A = want_of(x, c.W)
    b = np.zeros((M, N))
    b[:n] = c.bias[expert]
    Y = qp.qgemm_w4_experts(X, c.blobs, c.info, offsets, bias)
    _close(Y, want + b, A + np.abs(b), K, dtype, "y")
    assert (Y[n:] == 0).all(), "rows of no expert are zeros"
    # through a map: slots of three choices a token, some outside X
    T = max(1, M // 3)
    slots = c.rng.integers(0, 3 * T, M).astype(np.int32)
    slots[::5] = -1
    slots[1::7] = 3 * T + 2
    Xt, xt = c.rows(T, K, dtype)
    read = np.zeros((M, K))
    ok = (slots >= 0) & (slots < 3 * T)
    read[ok] = xt[slots[ok] // 3]
    want, A = want_of(read, c.W)
    Y = qp.qgemm_w4_experts(Xt, c.blobs, c.info, offsets, bias, rows=torch.from_numpy(slots).cuda(),
                            row_div=3)
    _close(Y, want + b, A + np.abs(b), K, dtype, "y through the map")
    dY, dy = c.rows(M, N, dtype)
    dX = qp.qgemm_w4_experts_dx(dY, c.blobs, c.info, offsets)
    want, A = want_of(dy, np.transpose(c.W, (0, 2, 1)))
    _close(dX, want, A, N, dtype, "dx", 2.0 ** -22 if dtype == "f32" else 2.0 ** -15)
    assert (dX[n:] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_strides_and_alignment(qp, dtype):
    """Rows inside wider buffers, starting at odd elements; what lies between
    them (NaN here) is neither read into the result nor written."""
    import torch
    for M, N, K in [(3, 70, 129), (40, 130, 390)]:
        c = Case(qp, 1, N, K, 32, "f32")
        X, x = c.rows(M, K, dtype)
        for left, right in [(1, 0), (3, 2), (0, 5), (8, 8)]:
            print("strides", dtype, M, N, K, left, right, flush=True)
            wide = torch.full((M, left + K + right), float("nan"), dtype=X.dtype, device="cuda")
            wide[:, left:left + K] = X
            out = torch.full((M, left + N + right), 7.0, dtype=X.dtype, device="cuda")
            Y = qp.qgemm_w4_blockwise(wide[:, left:left + K], c.blobs[0], c.info,
                                      out=out[:, left:left + N])
            assert torch.equal(Y, qp.qgemm_w4_blockwise(X, c.blobs[0], c.info))
            assert (out[:, :left] == 7).all() and (out[:, left + N:] == 7).all()
            dY, _ = c.rows(M, N, dtype)
            widey = torch.full((M, left + N + right), float("nan"), dtype=X.dtype, device="cuda")
            widey[:, left:left + N] = dY
            dout = torch.full((M, left + K + right), 7.0, dtype=X.dtype, device="cuda")
            dX = qp.qgemm_w4_blockwise_dx(widey[:, left:left + N], c.blobs[0], c.info,
                                          out=dout[:, left:left + K])
            assert torch.equal(dX, qp.qgemm_w4_blockwise_dx(dY, c.blobs[0], c.info))
            assert (dout[:, :left] == 7).all() and (dout[:, left + K:] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_non_finite_rows_stay_apart(qp, dtype):
    """A row with an infinity or a NaN gives what its own sum gives; every
    other row is what it is without it."""
    import torch
    M, N, K = 37, 70, 300
    c = Case(qp, 1, N, K, 32, "f32")
    X, x = c.rows(M, K, dtype)
    clean = qp.qgemm_w4_blockwise(X, c.blobs[0], c.info)
    bad = X.clone()
    bad[3, 17] = float("inf")
    bad[20, 299] = float("nan")
    bad[36, 0] = -float("inf")
    Y = qp.qgemm_w4_blockwise(bad, c.blobs[0], c.info)
    keep = [r for r in range(M) if r not in (3, 20, 36)]
    assert torch.equal(Y[keep], clean[keep])
    with np.errstate(invalid="ignore"):
        for r, k, v in [(3, 17, np.inf), (36, 0, -np.inf)]:
            want = v * c.W[0][:, k]       # 0 * inf is NaN, as in the sum
            got = Y[r].double().cpu().numpy()
            assert np.array_equal(np.isnan(got), np.isnan(want))
            assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])
    assert torch.isnan(Y[20]).all()
    dY, _ = c.rows(M, N, dtype)
    clean = qp.qgemm_w4_blockwise_dx(dY, c.blobs[0], c.info)
    dY[3, 17] = float("inf")
    dY[20, 69] = float("nan")
    dX = qp.qgemm_w4_blockwise_dx(dY, c.blobs[0], c.info)
    keep = [r for r in range(M) if r not in (3, 20)]
    assert torch.equal(dX[keep], clean[keep])
    assert not torch.isfinite(dX[3]).any() and torch.isnan(dX[20]).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_gradient_with_one_scale_a_block(qp, dtype, kind):
    """Groups of 128 and 384: by expert, with non-finite rows that stay apart,
    and f32 rows over the exponent range."""
    import torch
    M, N = 75, 330
    for group, K in [(128, 300), (384, 1000)]:
        c = Case(qp, 3, N, K, group, kind, seed=group)
        offsets = torch.tensor([0, 40, 40, 70], dtype=torch.int32, device="cuda")
        dY, dy = c.rows(M, N, dtype)
        if dtype == "f32":
            dY *= torch.logspace(-25, 25, M, device="cuda")[:, None]
            dy = dY.double().cpu().numpy()
        print("one scale a block", dtype, kind, group, flush=True)
        clean = qp.qgemm_w4_experts_dx(dY, c.blobs, c.info, offsets)
        want, A = np.zeros((M, K)), np.zeros((M, K))
        for e, r0, r1 in [(0, 0, 40), (2, 40, 70)]:
            want[r0:r1] = dy[r0:r1] @ c.W[e]
            A[r0:r1] = np.abs(dy[r0:r1]) @ np.abs(c.W[e])
        _close(clean, want, A, N, dtype, "dx", 2.0 ** -22 if dtype == "f32" else 2.0 ** -15)
        dY[3, 17] = float("inf")
        dY[50, N - 1] = float("nan")
        dX = qp.qgemm_w4_experts_dx(dY, c.blobs, c.info, offsets)
        keep = [r for r in range(M) if r not in (3, 50)]
        assert torch.equal(dX[keep], clean[keep])
        assert not torch.isfinite(dX[3]).any() and torch.isnan(dX[50]).all()


def test_large_f32_values_keep_their_accuracy(qp):
    """f32 rows over the whole exponent range, up to the largest finite value."""
    import torch
    N, K = 33, 160
    c = Case(qp, 1, N, K, 32, "f32")
    x = (c.rng.standard_normal((8, K)) * 10.0 ** np.arange(-32, 32, 8)[:, None]).astype(np.float32)
    x = np.concatenate([x, np.zeros((1, K), np.float32)])
    x[8, 5] = np.finfo(np.float32).max
    X = torch.from_numpy(x).cuda()
    W = c.W[0]
    x = x.astype(np.float64)
    _close(qp.qgemm_w4_blockwise(X, c.blobs[0], c.info), x @ W.T, np.abs(x) @ np.abs(W).T, K,
           "f32", "y")


@pytest.mark.parametrize("M", [200, 4096])  # few rows and many
def test_rows_far_apart(qp, M):
    """Mapped rows of a table past 4 GiB."""
    import torch
    N, K, ldx, E = 512, 100, 8192, 2
    c = Case(qp, E, N, K, 32, "f32", seed=M)
    table = torch.empty((1 << 18) + 64, ldx, dtype=torch.bfloat16, device="cuda")
    x_rows = table.shape[0]
    pick = c.rng.choice(x_rows // 2, M, replace=False) * 2   # every other row, the last ones too
    pick[0], pick[-1] = x_rows - 1, 1
    X, x = c.rows(M, K, "bf16")
    where = torch.from_numpy(pick).cuda()
    table[where, :K] = X
    cut = M // 3
    offsets = torch.tensor([0, cut, M], dtype=torch.int32, device="cuda")
    print("rows far apart", M, flush=True)
    Y = qp.qgemm_w4_experts(table[:, :K], c.blobs, c.info, offsets,
                            rows=where.to(torch.int32), row_div=1)
    want = np.concatenate([x[:cut] @ c.W[0].T, x[cut:] @ c.W[1].T])
    mag = np.concatenate([abs(x[:cut]) @ abs(c.W[0]).T, abs(x[cut:]) @ abs(c.W[1]).T])
    tol = (K / 32 + 64) * 2.0 ** -24 * mag + ROUND["bf16"] * np.abs(want) * 1.01
    got = Y.double().cpu().numpy()
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()


def test_empty_and_one(qp):
    import torch
    c = Case(qp, 2, 48, 64, 32, "f32")
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        X = torch.empty((0, 64), dtype=dt, device="cuda")
        off = torch.zeros(3, dtype=torch.int32, device="cuda")
        assert qp.qgemm_w4_blockwise(X, c.blobs[0], c.info).shape == (0, 48)
        assert qp.qgemm_w4_experts(X, c.blobs, c.info, off).shape == (0, 48)
        dY = torch.empty((0, 48), dtype=dt, device="cuda")
        assert qp.qgemm_w4_blockwise_dx(dY, c.blobs[0], c.info).shape == (0, 64)
        assert qp.qgemm_w4_experts_dx(dY, c.blobs, c.info, off).shape == (0, 64)


def test_offsets_out_of_range_stay_in_bounds(qp):
    """Offsets outside [0, M] are taken as the nearest bound."""
    import torch
    c = Case(qp, 3, 48, 64, 32, "f32")
    X, x = c.rows(20, 64, "f32")
    got = qp.qgemm_w4_experts(X, c.blobs, c.info,
                              torch.tensor([0, 8, 1000, 1000], dtype=torch.int32).cuda())
    want = qp.qgemm_w4_experts(X, c.blobs, c.info,
                               torch.tensor([0, 8, 20, 20], dtype=torch.int32).cuda())
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_against_differences(qp, dtype):
    """<dY, Y(X + h V) - Y(X - h V)> / 2h = <dX, V>: the product is linear, so
    the difference is exact but for the f32 sums (outputs in f32)."""
    import torch
    M, N, K = 9, 130, 200
    c = Case(qp, 1, N, K, 32, "asym")
    X, x = c.rows(M, K, dtype)
    dY, dy = c.rows(M, N, dtype)
    V, v = c.rows(M, K, dtype)
    h = 0.5
    Xp, Xm = X + h * V, X - h * V                       # rounded to the type: use what they are
    step = (Xp.double() - Xm.double()).cpu().numpy()
    f32 = torch.float32
    d = (qp.qgemm_w4_blockwise(Xp, c.blobs[0], c.info, out_dtype=f32).double() -
         qp.qgemm_w4_blockwise(Xm, c.blobs[0], c.info, out_dtype=f32).double()).cpu().numpy()
    dX = qp.qgemm_w4_blockwise_dx(dY, c.blobs[0], c.info).double().cpu().numpy()
    lhs, rhs = (dy * d).sum(), (dX * step).sum()
    W = np.abs(c.W[0]) + 0.2
    A = (np.abs(dy) @ W * (np.abs(Xp.double().cpu().numpy()) + np.abs(Xm.double().cpu().numpy()))).sum()
    tol = (2 * (K / 32 + 64) * 2.0 ** -24 + 2.0 ** -15 + ROUND[dtype]) * A
    assert abs(lhs - rhs) <= tol, (lhs, rhs, tol)


def test_other_stream_repeats_and_graph(qp):
    """On a stream that is not the tensors' own, ten times the same bits, and
    replayed in a graph."""
    import torch
    c = Case(qp, 4, 200, 384, 32, "f32")
    off = torch.tensor([0, 40, 40, 41, 90], dtype=torch.int32).cuda()
    X, _ = c.rows(95, 384, "bf16")
    dY, _ = c.rows(95, 200, "bf16")
    y0 = qp.qgemm_w4_experts(X, c.blobs, c.info, off)
    d0 = qp.qgemm_w4_experts_dx(dY, c.blobs, c.info, off)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(10):
            assert torch.equal(qp.qgemm_w4_experts(X, c.blobs, c.info, off), y0)
            assert torch.equal(qp.qgemm_w4_experts_dx(dY, c.blobs, c.info, off), d0)
    side.synchronize()
    Y, D = torch.empty_like(y0), torch.empty_like(d0)
    n = qp.qgemm_w4_dx_ws_size(95, c.info, 4)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qp.qgemm_w4_experts(X, c.blobs, c.info, off, out=Y)
        qp.qgemm_w4_experts_dx(dY, c.blobs, c.info, off, out=D, ws=ws)
    for _ in range(3):
        Y.zero_()
        D.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, y0) and torch.equal(D, d0)
