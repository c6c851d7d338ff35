"""MXFP4 rows that 32-bit offsets do not reach -- tokens through a map beyond 2^31 bytes,
rows 8 MiB apart -- in products of many rows: the same results as from rows that lie
together, as far as 2^31 outputs and more.  Tolerances as in test_gpu_mx4.py."""
import pytest

import mx4_card as card

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qp():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import conv_qpack_weights_amd as qp
    return qp


def _apart(qp, m, ldc, lds):
    """The matrix with its rows that many bytes apart, NaN's scale between them."""
    import torch
    rows, G = m.scales.shape
    room = lambda ld: torch.full((rows * ld,), 255, dtype=torch.uint8, device="cuda")
    c = room(ldc).as_strided((rows, 16 * G), (ldc, 1)).copy_(m.codes)
    s = room(lds).as_strided((rows, G), (lds, 1)).copy_(m.scales)
    return qp.MX4(c, s, m.K)


# one to eight stages of K, whole and cut, few and many words of scales
@pytest.mark.parametrize("K", [31, 256, 330, 416, 770, 1500, 2048])
@pytest.mark.parametrize("kernel,M,N", [("tile64x64", 600, 2000), ("tile128x128", 2600, 2000)])
def test_rows_through_the_map(qp, kernel, M, N, K):
    import torch
    g = torch.Generator().manual_seed(M + K)
    T = 300
    ldc = 1 << 23 if K == 330 else ((1 << 31) // T + 16) // 16 * 16
    W, w = card.matrix(qp, g, 3, N, K)
    A, a = card.matrix(qp, g, T, K)
    assert qp.qgemm_mx_kernel_name("a4w4", M, W, torch.float32) == kernel
    far = _apart(qp, A, ldc, 2048)
    off = torch.tensor([0, M // 5, M // 5, M - 9])
    offsets = off.int().cuda()
    rows = torch.randint(0, 2 * T, (M,), generator=g)
    rows[3], rows[M // 2], rows[7] = -1, 2 * T, 2 * T - 1
    src = torch.where((rows >= 0) & (rows < 2 * T), rows // 2, torch.full_like(rows, T)).cuda()
    print("mx4 far rows", kernel, M, N, K, flush=True)
    bias = torch.randn(3, N, generator=g).cuda()
    got = qp.qgemm_a4w4_mx_experts(far, W, offsets, bias, rows.int().cuda(), 2)
    x = torch.cat((a, torch.zeros_like(a[:1])))[src]
    for e in range(3):
        s = slice(int(off[e]), int(off[e + 1]))
        b = bias[e].double()
        card.close(got[s], x[s] @ card.t(w[e]) + b,
               x[s].abs() @ card.t(w[e]).abs() + b.abs(), K, "f32", "expert %d" % e)
    assert (got[M - 9:] == 0).all()


@pytest.mark.parametrize("K", [96, 770])
def test_rows_far_apart_in_tiles(qp, K):
    """Dense rows as far apart as a description may have them."""
    import torch
    g = torch.Generator().manual_seed(K)
    M, N, far = 300, 4010, 1 << 23
    W, w = card.matrix(qp, g, N, K)
    A, a = card.matrix(qp, g, M, K)
    assert qp.qgemm_mx_kernel_name("a4w4", M, W, torch.float32).startswith("tile")
    want, size = a @ card.t(w), a.abs() @ card.t(w).abs()
    for ldc, lds in ((far, 64), (-(-K // 32) * 16, far)):
        print("mx4 far apart in tiles", K, ldc, lds, flush=True)
        card.close(qp.qgemm_a4w4_mx(_apart(qp, A, ldc, lds), W), want, size, K, "f32", "far")


def test_more_outputs_than_a_launch_of_small_tiles(qp):
    """2^20 rows by 2064 channels through the map: refused before."""
    import torch
    g = torch.Generator().manual_seed(9)
    M, N, K, T = 1 << 20, 2064, 64, 2100
    W, w = card.matrix(qp, g, 1, N, K)
    A, a = card.matrix(qp, g, T, K)
    far = _apart(qp, A, 1 << 20, 64)
    rows = torch.randint(0, T, (M,), generator=g).cuda()
    rows[:T] = torch.arange(T, device="cuda")
    offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    print("mx4 far rows, many outputs", flush=True)
    got = qp.qgemm_a4w4_mx_experts(far, W, offsets, rows=rows.int(), out_dtype=torch.float32)
    card.close(got[:T], a @ card.t(w[0]), a.abs() @ card.t(w[0]).abs(), K, "f32", "first rows")
    for r in range(0, M, 1 << 17):
        s = slice(r, r + (1 << 17))
        assert torch.equal(got[s], got[rows[s]]), r
