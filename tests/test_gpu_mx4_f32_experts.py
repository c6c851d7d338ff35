"""f32 rows by expert in every kernel that they take, sizes held to their kernels."""
import pytest

import mx4_card as card

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qp():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import conv_qpack_weights_amd as qp
    return qp


# slots, experts, channels (the gradient's columns), and the kernel they take with f32 rows
F32 = [("w4", "rows16x16", 40, 8, 200), ("w4", "rows16x32", 40, 8, 800),
       ("w4", "rows16x48", 30, 4, 4100), ("w4", "rows16x64", 128, 16, 5500),
       ("w4", "tile128x128", 1200, 3, 2000), ("w4_dx", "rows16x128", 300, 3, 300),
       ("w4_dx", "tile128x128", 2600, 3, 2000)]


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("product,kernel,S,E,N", F32)
def test_f32_rows_by_expert(qp, product, kernel, S, E, N, odd):
    """Every kernel of f32 rows by expert: ragged experts, one of them empty, rows behind
    the last, slots that are no row."""
    import torch
    g = torch.Generator().manual_seed(S + N)
    K = 330
    cut = torch.sort(torch.randint(0, S - 2, (E,), generator=g)).values
    cut[1] = cut[0]
    off = torch.cat((torch.zeros(1, dtype=torch.long), cut))
    W, w = card.matrix(qp, g, E, K, N) if product == "w4_dx" else card.matrix(qp, g, E, N, K)
    assert qp.qgemm_mx_kernel_name(product, S, W, torch.float32).split("/")[0] == kernel
    print("mx4 f32 by expert", product, kernel, S, E, N, odd, flush=True)
    if product == "w4_dx":
        X, x = card.rows(torch.randn(S, K + 3, generator=g), "f32", odd)
        got, weights = qp.qgemm_w4_mx_experts_dx(X, W, off.int().cuda()), w
        src = torch.arange(S)
    else:
        T = S // 2
        X, x = card.rows(torch.randn(T, K + 3, generator=g), "f32", odd)
        slot = torch.randint(0, 2 * T, (S,), generator=g)
        slot[1], slot[5] = -1, 2 * T
        src = torch.where((slot >= 0) & (slot < 2 * T), slot // 2, torch.full_like(slot, T))
        got = qp.qgemm_w4_mx_experts(X, W, off.int().cuda(), rows=slot.int().cuda(), row_div=2)
        weights = card.t(w)
    x = torch.cat((x, torch.zeros_like(x[:1])))
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        r = x[src[s].cuda()]
        card.close(got[s], r @ weights[e], r.abs() @ weights[e].abs(), K, "f32", "expert %d" % e)
    assert (got[int(off[E]):] == 0).all()
