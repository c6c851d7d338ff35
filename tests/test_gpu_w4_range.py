"""The int4 products and their gradients over the range of values that their
header states, against the formulas in 64 bits.

Tolerances as in test_gpu_w4_kernels.py: (terms/32 + 64) * 2^-24 of the sum of
the terms' magnitudes, the output's rounding, 2^-22 a term for f32 gradients.
What lies below a type's smallest steps is added: f32 rows enter as three bf16
pieces, whose smallest step is 2^-133, so a value misses less than that; f32
sums of sixteenths step by 2^-149, 2^-145 of the result, a term each."""
import pytest

from test_gpu_w4_kernels import FORWARD, GRADIENT, Weights, _close, _dt, qp  # noqa: F401

pytestmark = pytest.mark.gpu

FEW_AND_MANY = ["rows1x1", "rows2x4", "tile4x8", "tile8x8"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "asym"])
@pytest.mark.parametrize("group", [32, 128, 256])
def test_large_rows(qp, dtype, kind, group):  # noqa: F811
    """Every element near 2^121: 128 of them times q/16 stay below 2^128."""
    import torch
    for name in FEW_AND_MANY:
        M, N, K = FORWARD[name][0]
        print("w4 large rows", name, dtype, kind, group, flush=True)
        c = Weights(qp, 1, N, K, group, kind, seed=group)
        x = 0.5 + 0.5 * torch.rand(M, K, generator=c.g, device="cuda")
        sign = torch.where(torch.rand(M, K, generator=c.g, device="cuda") < 0.5, -1.0, 1.0)
        X = (x * sign * 2.0 ** 121).to(_dt(dtype))
        X[0] = X[0].abs()                       # one row all of one sign
        _close(qp.qgemm_w4_blockwise(X, c.blobs[0], c.info),
               torch.mm(X.double(), c.W[0].t().contiguous()),
               torch.mm(X.double().abs(), c.A[0].t().contiguous()), K, dtype, "y")


@pytest.mark.parametrize("dtype,exponents", [("f32", [-100, -109, -115, -126, -140]),
                                             ("bf16", [-110, -118, -126, -132]),
                                             ("f16", [-12, -16, -22])])
@pytest.mark.parametrize("kind", ["f32", "asym"])
@pytest.mark.parametrize("group", [32, 128])
def test_small_rows(qp, dtype, exponents, kind, group):  # noqa: F811
    """Rows down to the types' subnormal values, outputs in f32."""
    import torch
    for name in FEW_AND_MANY:
        M, N, K = FORWARD[name][0]
        c = Weights(qp, 1, N, K, group, kind, seed=group + 1)
        for e in exponents:
            print("w4 small rows", name, dtype, kind, group, e, flush=True)
            X = torch.randn(M, K, generator=c.g, device="cuda", dtype=torch.float64)
            X = (X * 2.0 ** e).to(_dt(dtype))
            A = torch.mm(X.double().abs(), c.A[0].t().contiguous())
            want = torch.mm(X.double(), c.W[0].t().contiguous())
            got = qp.qgemm_w4_blockwise(X, c.blobs[0], c.info, out_dtype=torch.float32).double()
            tol = (K / 32 + 64) * 2.0 ** -24 * A + K * 2.0 ** -145
            if dtype == "f32":
                tol = tol + 2.0 ** -133 * c.A[0].sum(dim=1)
            assert not bool(((got - want).abs() > tol).any())


@pytest.mark.parametrize("kind", ["f32", "bf16", "asym"])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
def test_gradient_of_the_largest_values(qp, kind, group):  # noqa: F811
    """Finite f32 values of dY up to the largest: rounded to bf16 they would be
    infinities."""
    import torch
    big = torch.finfo(torch.float32).max
    for name in ("rows1/1", "rows1/8", "rows2/8", "rows4/8"):
        for E, (M, N, K) in zip((1, 3), GRADIENT[name]):
            print("w4 gradient of large values", name, kind, group, E, flush=True)
            c = Weights(qp, E, N, K, group, kind, seed=group + 2)
            dY = c.rows(M, N, "f32")
            dY[0, 5] = big
            dY[1, N - 1] = -big
            dY[2, 0], dY[2, N // 2] = 3.3961e38, -3.3980e38
            dY[M - 4, 40] = 3.39e38                         # rounds to the largest bf16
            if E == 1:
                dX = qp.qgemm_w4_blockwise_dx(dY, c.blobs[0], c.info)
                first = [0, M]
            else:
                first = [0, 2, 2, M]
                dX = qp.qgemm_w4_experts_dx(dY, c.blobs, c.info, torch.tensor(
                    first, dtype=torch.int32, device="cuda"))
            for e in range(E):
                r = slice(first[e], first[e + 1])
                dy = dY[r].double()
                if dy.shape[0]:
                    _close(dX[r], torch.mm(dy, c.W[e]), torch.mm(dy.abs(), c.A[e]), N, "f32",
                           "dx", 2.0 ** -22)
