"""Row maps with entries outside [0, T*top_k): they count as dropped."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qp():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import conv_qpack_weights_amd as qp
    return qp


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("T,k,H", [(3, 2, 5), (20, 2, 64), (40, 9, 1101)])
def test_rows_whose_slot_is_out_of_range_get_zeros(qp, dtype, T, k, H):
    """dZ of a row without a slot is zero, whichever value says so."""
    import torch
    rng = np.random.default_rng(T)
    print("combine gradient, slots out of range", dtype, T, k, H, flush=True)
    ids = rng.integers(0, 4, (T, k))
    ids[rng.random((T, k)) < 0.4] = -1
    ids[0, 0] = -1
    d = lambda a: torch.from_numpy(a).cuda()
    S = T * k
    t = getattr(torch, dtype)
    Z, dY = d(rng.standard_normal((S, H))).to(t), d(rng.standard_normal((T, H))).to(t)
    w = d(rng.uniform(0.1, 1, (T, k)).astype(np.float32))
    _, ros, sor = qp.qmoe_sort(d(ids), 4)
    dZ, dw = qp.qmoe_combine_grad(dY, Z, ros, sor, w)
    bare = sor < 0
    assert bool(bare.any()) and bool((dZ[bare] == 0).all())
    for value in (S, S + 1, 2 ** 31 - 1, -1, -(2 ** 31)):
        out = torch.full_like(Z, float("nan"))
        other = torch.where(bare, torch.full_like(sor, value), sor)
        maps = torch.where(ros < 0, torch.full_like(ros, value), ros)
        got, gw = qp.qmoe_combine_grad(dY, Z, maps, other, w, out=out)
        assert torch.equal(got, dZ) and torch.equal(gw, dw), value
        assert torch.equal(qp.qmoe_combine(Z, maps, w), qp.qmoe_combine(Z, ros, w)), value
        assert torch.equal(qp.qmoe_dispatch_grad(Z, maps), qp.qmoe_dispatch_grad(Z, ros)), value


@pytest.mark.parametrize("S", [63, 64, 65, 127, 128, 129, 255, 511, 512, 513, 1023, 1024, 1025, 4095,
                               4096, 4097, 8191, 8192, 8193])
@pytest.mark.parametrize("E", [1, 3, 64, 512])
def test_every_switch_of_the_sort(qp, S, E):
    """The sort alone and with rows, around the slot counts where its kernels
    change: offsets, maps and rows from a stable sort."""
    import torch
    rng = np.random.default_rng(S + E)
    print("sort around a switch", S, E, flush=True)
    for k in (1, 3) if S % 3 == 0 else (1,):
        T = S // k
        ids = rng.integers(0, E, (T, k))
        ids[rng.random((T, k)) < 0.2] = -1
        flat = ids.reshape(-1)
        order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
        n = int((flat >= 0).sum())
        offsets = np.searchsorted(flat[order][:n], np.arange(E + 1))
        ros, sor = np.full(S, -1), np.full(S, -1)
        sor[:n] = order[:n]
        ros[order[:n]] = np.arange(n)
        d = torch.from_numpy(ids).cuda()
        for H, dtype in ((5, torch.float32), (130, torch.bfloat16)):
            X = torch.from_numpy(rng.standard_normal((T, H))).to(dtype).cuda()
            out = torch.full((S, H), float("nan"), dtype=dtype, device="cuda")
            Xs, *maps = qp.qmoe_dispatch(X, d, E, out=out)
            for got in (maps, qp.qmoe_sort(d, E)):
                assert np.array_equal(got[0].cpu().numpy(), offsets)
                assert np.array_equal(got[1].cpu().numpy().reshape(-1), ros)
                assert np.array_equal(got[2].cpu().numpy(), sor)
            want = torch.zeros_like(Xs)
            want[:n] = X[torch.from_numpy(sor[:n] // k).cuda()]
            assert torch.equal(Xs, want)
