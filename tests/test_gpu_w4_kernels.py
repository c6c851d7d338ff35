"""Every kernel of the weight-only int4 products and of their gradients, with
every row type, scale kind and class of groups that it is built for, dense and
by expert, against the formulas in 64 bits.

FORWARD and GRADIENT hold sizes that take each kernel; that they do is checked
on the host too (test_w4_kernel_choice.py), so that other estimates of the
kernels' times cannot leave one without a test.  K ends inside a group, a 64-K
unit and a 128-K block; the few-rows kernels' waves have one and two blocks.

Tolerances, per output: the sums are f32.  A sum of n terms in any order is
within n * 2^-24 * A of the exact one, A the sum of the terms' magnitudes (of q
and of the offset, which are summed apart); a term passes at most 32 additions
inside an MFMA step, one per further step and a few across waves, so
n = terms/32 + 64.  Then one rounding to the output type: 2^-8 (bf16), 2^-11
(f16, 2^-25 among its subnormals) of the value.  The gradient also forms each
term to within 2^-15 (2^-22 for f32 rows)."""
import pytest

pytestmark = pytest.mark.gpu

ROUND = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
# kernel: (M, N, K) dense, (M, N, K) by expert (three of them)
FORWARD = {
    "rows1x1": ((9, 70, 1162), (9, 70, 1162)),
    "rows1x2": ((520, 70, 1162), (9, 2067, 1162)),
    "rows1x3": ((9, 8211, 1162), (9, 3300, 1162)),
    "rows1x4": ((1500, 70, 1162), (9, 4101, 1162)),
    "rows2x3": ((2050, 70, 1162), (2050, 70, 1162)),
    "rows2x4": ((33, 6165, 1162), (40, 4101, 1162)),
    "tile4x8": ((100, 14003, 450), (335, 4101, 450)),
    "tile8x8": ((4004, 517, 450), (400, 5013, 450)),
}
GRADIENT = {
    "rows1/1": ((9, 517, 100), (9, 517, 100)),
    "rows1/2": ((9, 2067, 8201), (9, 2067, 4101)),
    "rows1/4": ((9, 1101, 100), (9, 1101, 100)),
    "rows1/8": ((9, 2067, 100), (9, 2067, 100)),
    "rows2/1": ((33, 517, 12003), (40, 517, 8201)),
    "rows2/2": ((21, 3300, 12003), (40, 3300, 4101)),
    "rows2/4": ((21, 2067, 4101), (40, 2067, 2060)),
    "rows2/8": ((21, 2067, 2060), (40, 2067, 1101)),
    "rows4/1": ((100, 517, 8201), (100, 517, 8201)),
    "rows4/2": ((64, 3300, 8201), (257, 3300, 2060)),
    "rows4/4": ((2050, 2067, 100), (2050, 2067, 100)),
    "rows4/8": ((257, 2067, 450), (100, 2067, 1101)),
    "tile": ((335, 517, 12003), (257, 517, 12003)),
}
TYPES = ["f32", "bf16", "f16"]
KINDS = ["f32", "bf16", "asym"]


def forward_kernel(name, dtype):
    """f32 rows have no 128-row tile: their three pieces fill the LDS with 64."""
    return "tile4x8" if dtype == "f32" and name == "tile8x8" else name


@pytest.fixture(scope="module")
def qp():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import conv_qpack_weights_amd as qp
    return qp


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


class Weights:
    """E experts' int4 weights packed, and in f64 on the device: W the values,
    A their magnitudes, q's and the offset's apart."""

    def __init__(self, qp, E, N, K, group, kind, seed):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        G = -(-K // group)
        q = torch.randint(-8, 8, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
        uniform = lambda lo, hi: lo + (hi - lo) * torch.rand(E, N, G, generator=g, device="cuda")
        s = uniform(0.001, 0.02)
        off = uniform(-0.02, 0.02) if kind == "asym" else None
        if kind == "bf16":
            s = s.to(torch.bfloat16).float()
        of_k = torch.arange(K, device="cuda") // group
        self.W = s.double()[:, :, of_k] * q.double()
        self.A = self.W.abs()
        if off is not None:
            o = off.double()[:, :, of_k]
            self.W = self.W + o
            self.A = self.A + o.abs()
        self.blobs, self.info = qp.pack_s4_experts(q, s, group, "bf16" if kind == "bf16" else "f32",
                                                   off)
        self.g = g

    def rows(self, M, width, dtype):
        import torch
        return torch.randn(M, width, generator=self.g, device="cuda").to(_dt(dtype))


def _close(got, want, A, terms, dtype, what, term_rel=0.0):
    got = got.double()
    assert bool(got.isfinite().all()), what
    tol = ((terms / 32 + 64) * 2.0 ** -24 + term_rel) * A + ROUND[dtype] * want.abs() * 1.01 + \
        (2.0 ** -25 if dtype == "f16" else 0.0)
    off = (got - want).abs()
    bad = off > tol
    assert not bool(bad.any()), "%s: %d outputs off, worst by %.3g of its tolerance" % (
        what, int(bad.sum()), float((off / tol)[bad].max()))


def _split(M):
    """Rows of three experts, the second without any, and three of no expert."""
    a = (M - 3) * 2 // 5
    return [0, a, a, M - 3]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group", [32, 64, 128, 256])
def test_forward(qp, dtype, kind, group):
    import torch
    for name, sizes in FORWARD.items():
        for E, (M, N, K) in zip((1, 3), sizes):
            print("w4 kernel", name, dtype, kind, group, E, M, N, K, flush=True)
            c = Weights(qp, E, N, K, group, kind, seed=M * 31 + N + group)
            assert qp.qgemm_w4_kernel_name(M, c.info, _dt(dtype), E) == forward_kernel(name, dtype)
            X = c.rows(M, K, dtype)
            bias = torch.randn(E, N, generator=c.g, device="cuda")
            if E == 1:
                want = torch.mm(X.double(), c.W[0].t().contiguous()) + bias[0].double()
                A = torch.mm(X.double().abs(), c.A[0].t().contiguous()) + bias[0].abs().double()
                Y = qp.qgemm_w4_blockwise(X, c.blobs[0], c.info, bias[0])
                _close(Y, want, A, K, dtype, "y")
                continue
            first = _split(M)
            offsets = torch.tensor(first, dtype=torch.int32, device="cuda")
            perm = torch.randperm(M, generator=c.g, device="cuda")
            for rows in (None, perm.to(torch.int32)):
                src = X if rows is None else X[perm]
                want = torch.zeros(M, N, dtype=torch.float64, device="cuda")
                A = torch.zeros_like(want)
                for e in range(E):
                    r = slice(first[e], first[e + 1])
                    x = src[r].double()
                    want[r] = torch.mm(x, c.W[e].t().contiguous()) + bias[e].double()
                    A[r] = torch.mm(x.abs(), c.A[e].t().contiguous()) + bias[e].abs().double()
                Y = qp.qgemm_w4_experts(X, c.blobs, c.info, offsets, bias, rows=rows)
                _close(Y, want, A, K, dtype, "y" if rows is None else "y through the map")
                assert bool((Y[first[-1]:] == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group", [32, 64, 128, 256])
def test_gradient(qp, dtype, kind, group):
    import torch
    rel = 2.0 ** -22 if dtype == "f32" else 2.0 ** -15
    for name, sizes in GRADIENT.items():
        if name == "tile" and dtype != "bf16":
            continue
        for E, (M, N, K) in zip((1, 3), sizes):
            print("w4 gradient kernel", name, dtype, kind, group, E, M, N, K, flush=True)
            c = Weights(qp, E, N, K, group, kind, seed=M * 31 + N + group)
            assert qp.qgemm_w4_kernel_name(M, c.info, _dt(dtype), E, gradient=True) == name
            dY = c.rows(M, N, dtype)
            if E == 1:
                dX = qp.qgemm_w4_blockwise_dx(dY, c.blobs[0], c.info)
                _close(dX, torch.mm(dY.double(), c.W[0]), torch.mm(dY.double().abs(), c.A[0]), N,
                       dtype, "dx", rel)
                continue
            first = _split(M)
            offsets = torch.tensor(first, dtype=torch.int32, device="cuda")
            want = torch.zeros(M, K, dtype=torch.float64, device="cuda")
            A = torch.zeros_like(want)
            for e in range(E):
                r = slice(first[e], first[e + 1])
                dy = dY[r].double()
                want[r], A[r] = torch.mm(dy, c.W[e]), torch.mm(dy.abs(), c.A[e])
            dX = qp.qgemm_w4_experts_dx(dY, c.blobs, c.info, offsets)
            _close(dX, want, A, N, dtype, "dx", rel)
            assert bool((dX[first[-1]:] == 0).all())
