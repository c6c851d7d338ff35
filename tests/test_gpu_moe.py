"""Rows sorted by expert and back (qmoe_sort, qmoe_dispatch, qmoe_combine) and
their gradients against plain formulas in 64 bits.

Integers and copied rows are exact.  A weighted sum of k rows in f32 is within
(k + 1) * 2^-24 of the sum of its terms' magnitudes, a dot product of n terms
within n * 2^-24 (a thread's terms, then a tree: at most n/16 + 16 additions
deep, and n is above that); then one rounding to the row type, 2^-8 (bf16),
2^-11 (f16; 2^-25 among its subnormals) of the value."""
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


def _rows(rng, M, H, dtype):
    import torch
    x = torch.from_numpy(rng.standard_normal((M, H))).to(_dt(dtype))
    return x.cuda(), x.double().numpy()


def _route(rng, T, k, E, mode):
    ids = rng.integers(0, E, (T, k))
    if mode == "some dropped":
        ids[rng.random((T, k)) < 0.3] = -1
        ids[rng.random((T, k)) < 0.1] = E       # past the experts: dropped too
        if T > 2:
            ids[1] = -1                          # a token without experts
    elif mode == "all dropped":
        ids[:] = -1
    elif mode == "one expert":
        ids[:] = E - 1
    return ids


def _plan(ids, E):
    flat = ids.reshape(-1)
    kept = (flat >= 0) & (flat < E)
    order = np.array(sorted(np.flatnonzero(kept), key=lambda s: (flat[s], s)), dtype=np.int64)
    offsets = np.array([(kept & (flat < e)).sum() for e in range(E + 1)])
    ros = np.full(flat.size, -1)
    ros[order] = np.arange(order.size)
    sor = np.full(flat.size, -1)
    sor[:order.size] = order
    return offsets, ros.reshape(ids.shape), sor


def _same(got, want, what):
    assert np.array_equal(got.cpu().numpy(), want), what


def _close(got, want, tol, dtype, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    tol = tol + ROUND[dtype] * np.abs(want) * 1.01 + (2.0 ** -25 if dtype == "f16" else 0.0)
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%s: %d outputs off" % (what, bad.sum())


MODES = ["all kept", "some dropped", "all dropped", "one expert"]
# tokens, choices, experts: below, at and above every switch of the sort
ROUTES = [(1, 1, 1), (1, 8, 512), (3, 2, 5), (32, 2, 8), (33, 2, 64), (17, 16, 65), (1024, 2, 7),
          (2048, 2, 31), (4097, 1, 9), (16400, 1, 40), (262145, 1, 17), (131100, 3, 90),
          (1025, 2, 128), (2048, 1, 1), (700, 3, 512), (4099, 5, 33), (70000, 4, 64),
          (4096, 2, 512), (8192, 1, 3), (2731, 3, 33), (5461, 1, 16)]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T,k,E", ROUTES)
def test_sort(qp, T, k, E, mode):
    import torch
    rng = np.random.default_rng(T * 31 + k + E)
    ids = _route(rng, T, k, E, mode)
    print("sort", T, k, E, mode, flush=True)
    offsets, ros, sor = _plan(ids, E)
    for dt in (torch.int32, torch.int64):
        o, r, s = qp.qmoe_sort(torch.from_numpy(ids).to(dt).cuda(), E)
        _same(o, offsets, "offsets")
        _same(r, ros, "row of slot")
        _same(s, sor, "slot of row")
    wide = torch.full((T, k + 3), 0, dtype=torch.int64)
    wide[:, 1:k + 1] = torch.from_numpy(ids)
    o, r, s = qp.qmoe_sort(wide.cuda()[:, 1:k + 1], E)
    _same(o, offsets, "offsets, strided ids")
    _same(r, ros, "row of slot, strided ids")
    big = torch.from_numpy(np.where(ids < 0, -(1 << 40), np.where(ids >= E, (1 << 32), ids)))
    o, r, s = qp.qmoe_sort(big.cuda(), E)  # 64-bit ids whose low halves look valid
    _same(o, offsets, "offsets, wide ids")
    _same(s, sor, "slot of row, wide ids")


CASES = [(1, 1, 1, 64, "all kept"), (16, 2, 8, 4096, "all kept"), (7, 3, 5, 1, "some dropped"),
         (40, 2, 4, 1101, "some dropped"), (9, 4, 3, 8, "all dropped"), (5, 9, 16, 333, "some dropped"),
         (3, 20, 32, 130, "all kept"), (1500, 2, 64, 257, "some dropped"),
         (2100, 4, 100, 1024, "all kept"), (64, 8, 8, 8200, "one expert"),
         (5000, 3, 17, 5, "some dropped"), (90000, 3, 20, 9, "some dropped"),
         (140001, 2, 6, 4, "some dropped")]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,E,H,mode", CASES)
def test_there_and_back(qp, dtype, T, k, E, H, mode):
    import torch
    rng = np.random.default_rng(T + 13 * H)
    ids = _route(rng, T, k, E, mode)
    offsets, ros, sor = _plan(ids, E)
    S, n = T * k, offsets[-1]
    print("dispatch and back", dtype, T, k, E, H, mode, flush=True)
    X, x = _rows(rng, T, H, dtype)
    Xs, o, r, s = qp.qmoe_dispatch(X, torch.from_numpy(ids).cuda(), E)
    _same(o, offsets, "offsets")
    _same(r, ros, "row of slot")
    _same(s, sor, "slot of row")
    want = np.zeros((S, H))
    want[:n] = x[sor[:n] // k]
    _same(Xs.double(), want, "sorted rows")

    Z, z = _rows(rng, S, H, dtype)
    weights = rng.uniform(0, 1, (T, k)).astype(np.float32)
    w64 = weights.astype(np.float64)
    token, row = sor[:n] // k, np.arange(n)
    # what dropped slots and rows without a slot hold has no effect
    wt = torch.from_numpy(weights)
    wt[torch.from_numpy(ros < 0)] = float("nan")
    Zn = Z.clone()
    Zn[n:] = float("nan")
    wt = wt.cuda()
    want, mag = np.zeros((T, H)), np.zeros((T, H))
    np.add.at(want, token, z[row] * w64.reshape(-1)[sor[:n], None])
    np.add.at(mag, token, np.abs(z[row]) * w64.reshape(-1)[sor[:n], None])
    _close(qp.qmoe_combine(Zn, r, wt), want, (k + 1) * 2.0 ** -24 * mag, dtype, "combined rows")
    want, mag = np.zeros((T, H)), np.zeros((T, H))
    np.add.at(want, token, z[row])
    np.add.at(mag, token, np.abs(z[row]))
    _close(qp.qmoe_dispatch_grad(Zn, r), want, (k + 1) * 2.0 ** -24 * mag, dtype, "dX")

    dY, dy = _rows(rng, T, H, dtype)
    dZ, dw = qp.qmoe_combine_grad(dY, Zn, r, s, wt)
    want = np.zeros((S, H))
    want[:n] = dy[token] * w64.reshape(-1)[sor[:n], None]
    _close(dZ, want, 2.0 ** -24 * np.abs(want), dtype, "dZ")
    assert (dZ[n:] == 0).all()
    want, mag = np.zeros(S), np.zeros(S)
    want[sor[:n]] = (dy[token] * z[row]).sum(axis=1)
    mag[sor[:n]] = np.abs(dy[token] * z[row]).sum(axis=1)
    _close(dw.reshape(-1), want, (H + 1) * 2.0 ** -24 * mag, "f32", "dweights")
    assert (dw.cpu().numpy()[ros < 0] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [20, 2000])
def test_strides(qp, dtype, T):
    """Rows inside wider buffers at odd starts; the gaps are left alone."""
    import torch
    rng = np.random.default_rng(T)
    k, E, H = 2, 9, 203
    ids = torch.from_numpy(_route(rng, T, k, E, "some dropped")).cuda()
    X, _ = _rows(rng, T, H, dtype)
    Z, _ = _rows(rng, T * k, H, dtype)
    w = torch.from_numpy(rng.uniform(0, 1, (T, k)).astype(np.float32)).cuda()
    base = qp.qmoe_dispatch(X, ids, E)
    y0 = qp.qmoe_combine(Z, base[2], w)
    g0 = qp.qmoe_dispatch_grad(Z, base[2])
    d0 = qp.qmoe_combine_grad(X, Z, base[2], base[3], w)

    def wide(t, left, right):
        b = torch.full((t.shape[0], left + t.shape[1] + right), float("nan"), dtype=t.dtype,
                       device="cuda")
        b[:, left:left + t.shape[1]] = t
        return b[:, left:left + t.shape[1]]

    def room(M, left, right, dt):
        b = torch.full((M, left + H + right), 7.0, dtype=dt, device="cuda")
        return b, b[:, left:left + H]

    for left, right in [(1, 0), (0, 3), (5, 8)]:
        print("moe strides", dtype, T, left, right, flush=True)
        b, out = room(T * k, left, right, X.dtype)
        got = qp.qmoe_dispatch(wide(X, left, right), ids, E, out=out)
        assert all(torch.equal(a, c) for a, c in zip(got, base))
        assert (b[:, :left] == 7).all() and (b[:, left + H:] == 7).all()
        ww = wide(w, 1, 2)
        b, out = room(T, left, right, X.dtype)
        assert torch.equal(qp.qmoe_combine(wide(Z, left, right), base[2], ww, out=out), y0)
        assert (b[:, :left] == 7).all() and (b[:, left + H:] == 7).all()
        b, out = room(T, left, right, X.dtype)
        assert torch.equal(qp.qmoe_dispatch_grad(wide(Z, left, right), base[2], out=out), g0)
        b, out = room(T * k, left, right, X.dtype)
        got = qp.qmoe_combine_grad(wide(X, left, right), wide(Z, left, right), base[2], base[3],
                                   ww, out=out)
        assert torch.equal(got[0], d0[0]) and torch.equal(got[1], d0[1])
        assert (b[:, :left] == 7).all() and (b[:, left + H:] == 7).all()


def test_no_tokens(qp):
    import torch
    ids = torch.empty((0, 2), dtype=torch.int64, device="cuda")
    Xs, o, r, s = qp.qmoe_dispatch(torch.empty((0, 64), device="cuda"), ids, 5)
    assert Xs.shape == (0, 64) and o.tolist() == [0] * 6 and r.shape == (0, 2) and s.numel() == 0
    assert qp.qmoe_sort(ids, 512)[0].tolist() == [0] * 513
    w = torch.empty((0, 2), device="cuda")
    assert qp.qmoe_combine(Xs, r, w).shape == (0, 64)
    assert qp.qmoe_dispatch_grad(Xs, r).shape == (0, 64)
    assert qp.qmoe_combine_grad(Xs, Xs, r, s, w)[1].shape == (0, 2)


def test_infinities_reach_only_their_tokens(qp):
    import torch
    rng = np.random.default_rng(4)
    T, k, E, H = 50, 2, 6, 130
    ids = torch.from_numpy(_route(rng, T, k, E, "all kept")).cuda()
    _, _, r, s = qp.qmoe_dispatch(torch.zeros((T, H), device="cuda"), ids, E)
    Z, _ = _rows(rng, T * k, H, "bf16")
    w = torch.from_numpy(rng.uniform(0.1, 1, (T, k)).astype(np.float32)).cuda()
    y0 = qp.qmoe_combine(Z, r, w)
    Z[int(r[7, 1]), 3] = float("inf")
    Z[int(r[9, 0]), 129] = float("nan")
    y = qp.qmoe_combine(Z, r, w)
    assert y[7, 3] == float("inf") and torch.isnan(y[9, 129])
    y[7, 3], y[9, 129] = y0[7, 3], y0[9, 129]
    assert torch.equal(y, y0)


def test_combine_gradient_against_differences(qp):
    """The combination is linear in Z and in the weights, so central
    differences are exact but for the f32 sums."""
    import torch
    rng = np.random.default_rng(8)
    T, k, E, H = 30, 3, 5, 96
    ids = torch.from_numpy(_route(rng, T, k, E, "some dropped")).cuda()
    X, _ = _rows(rng, T, H, "f32")
    Xs, _, r, s = qp.qmoe_dispatch(X, ids, E)
    Z, z = _rows(rng, T * k, H, "f32")
    w = torch.from_numpy(rng.uniform(0.1, 1, (T, k)).astype(np.float32)).cuda()
    dY, dy = _rows(rng, T, H, "f32")
    V, v = _rows(rng, T * k, H, "f32")
    U = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    dZ, dw = qp.qmoe_combine_grad(dY, Z, r, s, w)

    def f(z_, w_):
        return (qp.qmoe_combine(z_, r, w_).double() * dY.double()).sum()

    scale = 16 * 2.0 ** -24 * float((qp.qmoe_combine(Z.abs() + V.abs(), r, w.abs() + U.abs())
                                     * dY.abs()).double().sum())
    dif = (f(Z + V, w) - f(Z - V, w)) / 2
    assert abs(float(dif - (dZ.double() * V.double()).sum())) <= scale
    dif = (f(Z, w + U) - f(Z, w - U)) / 2
    assert abs(float(dif - (dw.double() * U.double()).sum())) <= (H + 16) / 16 * scale
    # dispatch: <dXs, Xs(X)> = <dX, X>
    dX = qp.qmoe_dispatch_grad(Z, r)
    n = int((s >= 0).sum())
    lhs = (Xs[:n].double() * Z[:n].double()).sum()
    assert abs(float(lhs - (dX.double() * X.double()).sum())) <= \
        8 * 2.0 ** -24 * float((Xs[:n].abs() * Z[:n].abs()).double().sum())


def test_other_stream_repeats_and_graph(qp):
    import torch
    rng = np.random.default_rng(3)
    for T, k, E, H in [(20, 2, 8, 256), (3000, 2, 40, 200)]:
        print("moe stream and graph", T, flush=True)
        ids = torch.from_numpy(_route(rng, T, k, E, "some dropped")).cuda()
        X, _ = _rows(rng, T, H, "bf16")
        Z, _ = _rows(rng, T * k, H, "bf16")
        w = torch.from_numpy(rng.uniform(0, 1, (T, k)).astype(np.float32)).cuda()

        def all_of():
            d = qp.qmoe_dispatch(X, ids, E)
            return [*d, qp.qmoe_combine(Z, d[2], w), qp.qmoe_dispatch_grad(Z, d[2]),
                    *qp.qmoe_combine_grad(X, Z, d[2], d[3], w)]

        first = all_of()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(10):
                assert all(torch.equal(a, b) for a, b in zip(all_of(), first))
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = all_of()
        for _ in range(3):
            for o in outs:
                o.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, first))
