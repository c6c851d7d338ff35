"""Every kernel of the MXFP4 products and their gradient, with every row type, dense
and by expert, at sizes that cut its tiles, its steps of K and its last block -- and
rows at odd addresses, which the kernels' direct loads cannot take.  The sizes are
held to the kernels they are there for.  Tolerances as in test_gpu_mx4.py, against
64-bit products on the card."""
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


def _matrix(qp, g, *shape):
    """A random MX4, and its values in f64 on the card."""
    import torch
    *lead, K = shape
    G = -(-K // 32)
    codes = torch.randint(0, 256, (*lead, 16 * G), generator=g, dtype=torch.uint8)
    if K % 32:
        both = torch.stack((codes & 15, codes >> 4), -1).reshape(*lead, 32 * G)
        both[..., K:] = 0
        codes = both[..., 0::2] | (both[..., 1::2] << 4)
    scales = torch.randint(118, 130, (*lead, G), generator=g, dtype=torch.uint8)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    grid = torch.cat((grid, -grid))
    v = grid[torch.stack((codes & 15, codes >> 4), -1).long()].reshape(*lead, 32 * G)
    v = v * torch.pow(2.0, scales.double() - 127).repeat_interleave(32, -1)
    return qp.mx4_tensor(codes.cuda(), scales.cuda(), K), v[..., :K].cuda()


def _rows(g, M, K, dtype, odd=False):
    import torch
    x = torch.randn(M, K + 3, generator=g).to(_dt(dtype)).cuda()
    x = x[:, 1:1 + K] if odd else x[:, :K].contiguous()
    return x, x.double()


def _close(got, want, A, terms, dtype, what):
    import torch
    got = got.double()
    assert torch.isfinite(got).all(), what
    tol = (3 * terms / 32 + 64) * 2.0 ** -23 * A + ROUND[dtype] * want.abs() * 1.01 \
        + (2.0 ** -25 if dtype == "f16" else 0.0)
    off = (got - want).abs()
    assert (off <= tol).all(), "%s: %d outputs off, worst by %.3g of its tolerance" % (
        what, int((off > tol).sum()), float((off / tol.clamp_min(1e-300)).max()))


SMALL = [("rows16x16", 5, 300), ("rows16x32", 30, 4010), ("rows16x48", 13, 9000),
         ("rows16x64", 61, 4030)]
PRODUCTS = (
    [("a4w4", t, k, M, N) for t in ("f32", "bf16", "f16") for k, M, N in
     [("rows16x16", 5, 300), ("rows16x32", 45, 4010), ("tile64x64", 250, 4010),
      ("tile128x128", 1100, 4010), ("tile256x256", 4090, 4090)]]
    + [("w4", t, k, M, N) for t in ("bf16", "f16") for k, M, N in SMALL +
       [("tile32x64", 146, 4900), ("tile32x128", 500, 4010), ("tile128x128", 1100, 4010),
        ("tile256x256", 4090, 4090)]]
    + [("w4", t, "rows16x64", 13, 49000) for t in ("bf16", "f16")]  # several rounds
    + [("w4", t, "tile128x128", 1000, 4010) for t in ("bf16", "f16")]  # one to a CU
    + [("w4", "f32", k, M, N) for k, M, N in SMALL + [("tile128x128", 1100, 4010)]])


@pytest.mark.parametrize("product,dtype,kernel,M,N", PRODUCTS)
def test_product_kernels(qp, product, dtype, kernel, M, N):
    import torch
    g = torch.Generator().manual_seed(M + N)
    # whole steps and cut ones; a K below a step; many steps
    for K in (31, 64, 330, 768, 1500):
        if M * N > 8e6 and K not in (330, 768):
            continue
        W, w = _matrix(qp, g, N, K)
        assert qp.qgemm_mx_kernel_name(product, M, W, _dt(dtype)) == kernel
        print("mx4 kernel", product, dtype, kernel, M, N, K, flush=True)
        bias = torch.randn(N, generator=g).cuda()
        for odd in (False, True) if product == "w4" else (False,):
            if product == "a4w4":
                A, a = _matrix(qp, g, M, K)
                got = qp.qgemm_a4w4_mx(A, W, bias, out_dtype=_dt(dtype))
            else:
                A, a = _rows(g, M, K, dtype, odd)
                got = qp.qgemm_w4_mx(A, W, bias)
            _close(got, a @ w.t().contiguous() + bias.double(),
                   a.abs() @ w.abs().t().contiguous() + bias.double().abs(), K, dtype,
                   "K=%d odd=%s" % (K, odd))


@pytest.mark.parametrize("dtype,kernel,M,K", [
    (t, k, M, K) for t in ("f32", "bf16", "f16") for k, M, K in
    [("rows16x128", 5, 300), ("rows16x128", 140, 1500), ("tile128x128", 2100, 4010)]
    + ([] if t == "f32" else [("tile256x256", 4090, 4090)])])
def test_gradient_kernels(qp, dtype, kernel, M, K):
    import torch
    g = torch.Generator().manual_seed(M + K)
    for N in (1, 63, 64, 330, 768, 1500):
        if M * K > 8e6 and N not in (63, 330, 768):
            continue
        W, w = _matrix(qp, g, N, K)
        assert qp.qgemm_mx_kernel_name("w4_dx", M, W, _dt(dtype)).split("/")[0] == kernel
        print("mx4 gradient kernel", dtype, kernel, M, N, K, flush=True)
        for odd in (False, True):
            dY, dy = _rows(g, M, N, dtype, odd)
            _close(qp.qgemm_w4_mx_dx(dY, W), dy @ w, dy.abs() @ w.abs(), N, dtype,
                   "N=%d odd=%s" % (N, odd))


EXPERTS = [  # product, kernel, slots, experts, channels (the gradient's columns)
    ("a4w4", "rows16x16", 40, 8, 200), ("a4w4", "rows16x32", 128, 16, 5500),
    ("a4w4", "tile64x64", 600, 3, 2000), ("a4w4", "tile128x128", 2600, 3, 2000),
    ("a4w4", "tile256x256", 7000, 3, 4000),
    ("w4", "rows16x16", 40, 8, 200), ("w4", "rows16x64", 64, 8, 4000),
    ("w4", "rows16x64", 128, 16, 5500), ("w4", "tile32x128", 256, 16, 5500),
    ("w4", "tile128x128", 2600, 3, 2000), ("w4", "tile128x128", 1200, 3, 2000),
    ("w4", "tile256x256", 7000, 3, 4000),
    ("w4_dx", "rows16x128", 300, 3, 300), ("w4_dx", "tile128x128", 2600, 3, 2000),
    ("w4_dx", "tile256x256", 6000, 3, 2000)]


@pytest.mark.parametrize("product,kernel,S,E,N,dtype", [
    (*c, t) for c in EXPERTS for t in ("bf16", "f16", "f32")
    if t != "f32" or c[0] == "a4w4" or c[1] not in ("tile256x256", "tile32x128")])
def test_kernels_by_expert(qp, product, kernel, S, E, N, dtype):
    """Ragged experts, one of them empty; rows behind the last; products through the
    map, with slots that are no row."""
    import torch
    g = torch.Generator().manual_seed(S + N)
    K = 330
    cut = torch.sort(torch.randint(0, S - 2, (E,), generator=g)).values
    cut[1] = cut[0]
    off = torch.cat((torch.zeros(1, dtype=torch.long), cut))
    offsets = off.int().cuda()
    # (the gradient: N columns, 330 channels)
    W, w = _matrix(qp, g, E, K, N) if product == "w4_dx" else _matrix(qp, g, E, N, K)
    name = qp.qgemm_mx_kernel_name(product, S, W, _dt(dtype)).split("/")[0]
    if dtype != "f32":
        assert name == kernel
    print("mx4 by expert", product, dtype, name, S, E, N, flush=True)
    if product == "w4_dx":
        X, x = _rows(g, S, K, dtype)
        got, terms, cols = qp.qgemm_w4_mx_experts_dx(X, W, offsets), K, N
        src, weights = torch.arange(S), w
    else:
        T = S // 2
        slot = torch.randint(0, 2 * T, (S,), generator=g)
        slot[1], slot[5] = -1, 2 * T
        src = torch.where((slot >= 0) & (slot < 2 * T), slot // 2, torch.full_like(slot, -1))
        through = dict(rows=slot.int().cuda(), row_div=2)
        terms, cols = K, N
        weights = w.transpose(1, 2).contiguous()
        if product == "a4w4":
            A, x = _matrix(qp, g, T, K)
            got = qp.qgemm_a4w4_mx_experts(A, W, offsets, out_dtype=_dt(dtype), **through)
        else:
            X, x = _rows(g, T, K, dtype)
            got = qp.qgemm_w4_mx_experts(X, W, offsets, **through)
    x = torch.cat((x, torch.zeros_like(x[:1])))        # row -1: zeros
    want = torch.zeros(S, cols, dtype=torch.float64, device="cuda")
    A = torch.zeros_like(want)
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        rows = x[src[s].cuda()]
        want[s], A[s] = rows @ weights[e], rows.abs() @ weights[e].abs()
    _close(got, want, A, terms, dtype, "by expert")
    assert (got[int(off[E]):] == 0).all()


@pytest.mark.parametrize("M", [3, 150])
def test_rows_far_apart(qp, M):
    """Rows 8 MiB apart, as far as the description allows: more than 32-bit offsets
    within a tile reach."""
    import torch
    g = torch.Generator().manual_seed(M)
    N, K, far = 40, 330, 1 << 23
    W, w = _matrix(qp, g, N, K)
    A, a = _matrix(qp, g, M, K)

    def spread(m, codes, scales):
        """The matrix with its codes' or scales' rows `far` bytes apart."""
        c, s = m.codes, m.scales
        if codes:
            c = torch.zeros(c.shape[0] * far, dtype=torch.uint8, device="cuda").as_strided(
                c.shape, (far, 1)).copy_(c)
        if scales:
            s = torch.zeros(s.shape[0] * far, dtype=torch.uint8, device="cuda").as_strided(
                s.shape, (far, 1)).copy_(s)
        return qp.MX4(c, s, m.K)

    A_abs = a.abs() @ w.abs().t().contiguous()
    for codes, scales in ((True, False), (False, True)):
        print("mx4 far apart", M, codes, scales, flush=True)
        Wf, Af = spread(W, codes, scales), spread(A, codes, scales)
        for x, y in ((A, Wf), (Af, W)):
            _close(qp.qgemm_a4w4_mx(x, y), a @ w.t().contiguous(), A_abs, K, "f32", "a4w4")
        for dtype in ("f32", "bf16", "f16"):
            X, x = _rows(g, M, K, dtype)
            _close(qp.qgemm_w4_mx(X, Wf), x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous(),
                   K, dtype, "w4")
            dY, dy = _rows(g, M, N, dtype)
            _close(qp.qgemm_w4_mx_dx(dY, Wf), dy @ w, dy.abs() @ w.abs(), N, dtype, "dx")
    X, x = _rows(g, M, K, "bf16")
    wide = torch.zeros(M * (far // 2 + 8), dtype=torch.bfloat16, device="cuda").as_strided(
        (M, K), (far // 2 + 8, 1)).copy_(X)
    _close(qp.qgemm_w4_mx(wide, W), x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous(), K,
           "bf16", "w4")


def test_rows_past_32_bits_through_the_map(qp):
    """Tokens whose rows lie beyond 2^31 bytes, read through the map, and products of as
    many rows in one call's place (sorted rows from far down)."""
    import torch
    g = torch.Generator().manual_seed(1)
    E, N, K, T = 2, 70, 4096, 270000
    W, w = _matrix(qp, g, E, N, K)
    X = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    X[-40:] = torch.randn(40, K, generator=g).to(torch.bfloat16).cuda()
    x = X[-40:].double()
    offsets = torch.tensor([0, 15, 40], dtype=torch.int32, device="cuda")
    rows = torch.arange(T - 40, T, dtype=torch.int32, device="cuda")
    wt = w.transpose(1, 2).contiguous()
    want = torch.cat((x[:15] @ wt[0], x[15:] @ wt[1]))
    A = torch.cat((x[:15].abs() @ wt[0].abs(), x[15:].abs() @ wt[1].abs()))
    _close(qp.qgemm_w4_mx_experts(X, W, offsets, rows=rows), want, A, K, "bf16", "w4")
    q = qp.qquantize_rows_mx4(X)
    back = qp.qdequantize_rows_mx4(qp.MX4(q.codes[-40:], q.scales[-40:], K)).double()
    want = torch.cat((back[:15] @ wt[0], back[15:] @ wt[1]))
    A = torch.cat((back[:15].abs() @ wt[0].abs(), back[15:].abs() @ wt[1].abs()))
    _close(qp.qgemm_a4w4_mx_experts(q, W, offsets, rows=rows), want, A, K, "f32", "a4w4")
    # the same rows at the end of a call of all of them
    Y = qp.qgemm_w4_mx(X, W[0])
    _close(Y[-40:], x @ wt[0], x.abs() @ wt[0].abs(), K, "bf16", "w4 of many rows")
    assert (Y[:-40] == 0).all()


def test_values_below_the_normal_range(qp):
    """bf16 and f32 rows among the subnormal values, brought back by the weights."""
    import torch
    g = torch.Generator().manual_seed(5)
    for M in (4, 600):
        N, K = 4010 if M > 4 else 70, 256
        W, w = _matrix(qp, g, N, K)
        W.scales.add_(80)
        w = w * 2.0 ** 80
        for dtype in ("bf16", "f32"):
            X = (torch.randn(M, K, generator=g) * 2.0 ** -126).to(_dt(dtype)).cuda()
            x = X.double()
            A = x.abs() @ w.abs().t().contiguous()
            # f32 values are cut, not rounded, into bf16 pieces, whose smallest step is
            # 2^-133: what is lost of one is below that
            slack = 0.0 if dtype == "bf16" else 2.0 ** -133 * w.abs().sum(1)
            off = (qp.qgemm_w4_mx(X, W, out_dtype=torch.float32).double()
                   - x @ w.t().contiguous()).abs()
            assert (off <= (3 * K / 32 + 64) * 2.0 ** -23 * A + slack).all(), (dtype, M)


@pytest.mark.parametrize("kernel,M,N", [("tile64x64", 250, 4010), ("tile128x128", 1100, 4010),
                                        ("tile256x256", 4090, 4090)])
def test_tiles_at_every_end_of_a_rows_scales(qp, kernel, M, N):
    """One to sixteen words of scales a row, whole and cut ones, rows apart and not."""
    import torch
    g = torch.Generator().manual_seed(M)
    for K in (385, 416, 512, 520, 640, 770, 900, 1024, 1060, 1290, 1660):
        if M * N > 8e6 and K not in (385, 640, 770, 1290):
            continue
        print("mx4 scales' end", kernel, M, N, K, flush=True)
        W, w = _matrix(qp, g, N, K)
        A, a = _matrix(qp, g, M, K)
        assert qp.qgemm_mx_kernel_name("a4w4", M, W, torch.float32) == kernel
        want, size = a @ w.t().contiguous(), a.abs() @ w.abs().t().contiguous()
        _close(qp.qgemm_a4w4_mx(A, W), want, size, K, "f32", "K=%d" % K)
        G = W.scales.shape[-1]
        apart = torch.full((M, -(-G // 4) * 4 + 8), 255, dtype=torch.uint8, device="cuda")[:, :G]
        B = qp.mx4_tensor(A.codes, apart.copy_(A.scales), K)
        _close(qp.qgemm_a4w4_mx(B, W), want, size, K, "f32", "K=%d apart" % K)


@pytest.mark.parametrize("product,dtype", [("a4w4", "f32"), ("w4", "bf16"), ("w4", "f16"),
                                           ("w4_dx", "bf16"), ("w4_dx", "f16")])
def test_a_last_round_in_half_tiles(qp, product, dtype):
    """19 x 32 tiles of 256 x 256: 76 to each of 8 times 32 CUs, the last 12 in halves,
    some of which have no rows; and few rows of many given."""
    import torch
    g = torch.Generator().manual_seed(5)
    M, N, K = 4700, 8190, 330
    print("mx4 half tiles", product, dtype, flush=True)
    W, w = _matrix(qp, g, K, N) if product == "w4_dx" else _matrix(qp, g, N, K)
    assert qp.qgemm_mx_kernel_name(product, M, W, _dt(dtype)).split("/")[0] == "tile256x256"
    wt = w if product == "w4_dx" else w.t().contiguous()
    if product == "a4w4":
        X, x = _matrix(qp, g, M, K)
    else:
        X, x = _rows(g, M, K, dtype)
    run = {"a4w4": qp.qgemm_a4w4_mx, "w4": qp.qgemm_w4_mx, "w4_dx": qp.qgemm_w4_mx_dx}[product]
    want, size = x @ wt, x.abs() @ wt.abs()
    _close(run(X, W), want, size, K, dtype, "dense")
    one = qp.mx4_tensor(W.codes[None], W.scales[None], W.K)
    assert one.shape[0] == 1
    for rows in (0, 1, 300, 4000):
        offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        run = {"a4w4": qp.qgemm_a4w4_mx_experts, "w4": qp.qgemm_w4_mx_experts,
               "w4_dx": qp.qgemm_w4_mx_experts_dx}[product]
        got = run(X, one, offsets)
        assert not got[rows:].any()
        if rows:
            _close(got[:rows], want[:rows], size[:rows], K, dtype, "%d rows" % rows)


@pytest.mark.parametrize("product,kernel,M,N", [
    ("w4", "rows16x16", 5, 300), ("w4", "rows16x64", 61, 4030), ("w4", "tile32x64", 146, 4900),
    ("w4", "tile32x128", 500, 4010), ("w4", "tile128x128", 1100, 4010),
    ("w4", "tile128x128", 1000, 4010),
    ("w4", "tile256x256", 4090, 4090), ("w4_dx", "rows16x128", 5, 300),
    ("w4_dx", "tile128x128", 2100, 4010), ("w4_dx", "tile256x256", 4090, 4090)])
def test_one_block_that_is_no_f16_values(qp, product, kernel, M, N):
    """f16 rows: a single scale out of f16's reach, in the first block, before the last
    and in a cut one, rows by direct loads and through registers."""
    import torch
    K = 330
    for where in (0, 1, 2):
        g = torch.Generator().manual_seed(M + where)
        # (the gradient: N columns, 330 channels)
        shape = (K, N) if product == "w4_dx" else (N, K)
        W, w = _matrix(qp, g, *shape)
        rows, G = W.scales.shape
        r, b = [(0, 0), (rows // 2, G - 2), (rows - 1, G - 1)][where]
        old = int(W.scales[r, b])
        W.scales[r, b] = 150
        w[r, 32 * b:32 * b + 32] *= 2.0 ** (150 - old)
        assert qp.qgemm_mx_kernel_name(product, M, W, torch.float16).split("/")[0] == kernel
        print("mx4 one block", product, kernel, M, N, where, flush=True)
        for odd in (False, True):
            X, x = _rows(g, M, K, "f16", odd)
            X, x = X * 2.0 ** -14, x * 2.0 ** -14  # (so that f16 gradients stay finite)
            x = X.double()
            if odd:
                X = torch.cat((torch.zeros_like(X[:, :1]), X), 1)[:, 1:]
            if product == "w4_dx":
                got, v = qp.qgemm_w4_mx_dx(X, W), w
                _close(got, x @ v, x.abs() @ v.abs(), K, "f16", "odd=%s" % odd)
            else:
                got, v = qp.qgemm_w4_mx(X, W, out_dtype=torch.float32), w.t().contiguous()
                _close(got, x @ v, x.abs() @ v.abs(), K, "f32", "odd=%s" % odd)


@pytest.mark.parametrize("product,dtype", [("a4w4", "bf16"), ("w4", "f16"), ("w4_dx", "bf16")])
def test_large_tiles_of_many_experts(qp, product, dtype):
    """More experts than a wave has lanes, in 256 x 256 tiles, a last round in halves."""
    import torch
    g = torch.Generator().manual_seed(70)
    E, K, N = 130, 130, 1000
    counts = torch.randint(0, 2000, (E,), generator=g)
    counts[3] = counts[64] = counts[129] = 0
    off = torch.cat((torch.zeros(1, dtype=torch.long), counts.cumsum(0)))
    S = int(off[E]) + 77
    W, w = _matrix(qp, g, E, K, N) if product == "w4_dx" else _matrix(qp, g, E, N, K)
    print("mx4 many experts", product, dtype, S, flush=True)
    assert qp.qgemm_mx_kernel_name(product, S, W, _dt(dtype)).split("/")[0] == "tile256x256"
    offsets = off.int().cuda()
    if product == "a4w4":
        X, x = _matrix(qp, g, S, K)
        got = qp.qgemm_a4w4_mx_experts(X, W, offsets, out_dtype=_dt(dtype))
    else:
        X, x = _rows(g, S, K, dtype)
        got = (qp.qgemm_w4_mx_experts if product == "w4" else qp.qgemm_w4_mx_experts_dx)(
            X, W, offsets)
    want = torch.zeros(S, N, dtype=torch.float64, device="cuda")
    A = torch.zeros_like(want)
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        v = w[e] if product == "w4_dx" else w[e].t().contiguous()
        want[s], A[s] = x[s] @ v, x[s].abs() @ v.abs()
    _close(got, want, A, K, dtype, "many experts")
    assert not got[int(off[E]):].any()


@pytest.mark.parametrize("product,dtype,kernel,M,N", [c for c in PRODUCTS if c[4] < 9000])
def test_bounds_in_every_kernel(qp, product, dtype, kernel, M, N):
    """Bounds on either side and both, after the bias, are a clamp of the result without."""
    import torch
    g = torch.Generator().manual_seed(M)
    K = 330
    W, w = _matrix(qp, g, N, K)
    assert qp.qgemm_mx_kernel_name(product, M, W, _dt(dtype)) == kernel
    print("mx4 bounds", product, dtype, kernel, M, N, flush=True)
    bias = torch.randn(N, generator=g).cuda()
    if product == "a4w4":
        X, run = _matrix(qp, g, M, K)[0], qp.qgemm_a4w4_mx
    else:
        X, run = _rows(g, M, K, dtype)[0], qp.qgemm_w4_mx
    free = run(X, W, bias, out_dtype=torch.float32)
    inf = float("inf")
    for lo, hi in ((-0.5, inf), (-inf, 0.25), (-0.5, 0.25), (0.0, 0.0)):
        got = run(X, W, bias, lo, hi, out_dtype=_dt(dtype))
        assert torch.equal(got, free.clamp(lo, hi).to(_dt(dtype))), (lo, hi)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("product,kernel,M,N", [
    ("a4w4", "rows16x32", 45, 4010), ("a4w4", "tile64x64", 250, 4010),
    ("a4w4", "tile128x128", 1100, 4010), ("a4w4", "tile256x256", 4090, 4090),
    ("w4", "tile32x128", 500, 4010), ("w4", "tile128x128", 1100, 4010),
    ("w4", "tile256x256", 4090, 4090), ("w4_dx", "rows16x128", 5, 300),
    ("w4_dx", "tile128x128", 2100, 4010), ("w4_dx", "tile256x256", 4090, 4090)])
def test_outputs_at_odd_places(qp, product, kernel, M, N, dtype):
    """Rows of the result an odd number of elements apart and from an odd one on: the same
    results, and nothing beside them."""
    import torch
    g = torch.Generator().manual_seed(N)
    K = 330
    W, _ = _matrix(qp, g, K, N) if product == "w4_dx" else _matrix(qp, g, N, K)
    name = qp.qgemm_mx_kernel_name(product, M, W, _dt(dtype)).split("/")[0]
    assert dtype == "f32" or name == kernel
    print("mx4 odd outputs", product, dtype, name, M, N, flush=True)
    X = _matrix(qp, g, M, K)[0] if product == "a4w4" else _rows(g, M, K, dtype)[0]
    run = {"a4w4": qp.qgemm_a4w4_mx, "w4": qp.qgemm_w4_mx, "w4_dx": qp.qgemm_w4_mx_dx}[product]
    kw = {"out_dtype": _dt(dtype)} if product == "a4w4" else {}
    want = run(X, W, **kw)
    wide = torch.full((M + 1, N + 3 - N % 2), 7.0, dtype=_dt(dtype), device="cuda")
    run(X, W, out=wide[:M, 1:1 + N])
    assert torch.equal(wide[:M, 1:1 + N], want)
    assert (wide[M] == 7).all() and (wide[:, 0] == 7).all() and (wide[:, 1 + N:] == 7).all()
