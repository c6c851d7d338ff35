"""One workspace of the MXFP4 gradients for calls of any number of rows: the size for the
most of them, with nothing written behind it."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qp():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import conv_qpack_weights_amd as qp
    return qp


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("N,K,E", [(1037, 1100, 1), (600, 130, 3)])
def test_one_workspace_for_all(qp, N, K, E, dtype):
    import torch
    g = torch.Generator().manual_seed(N)
    w = torch.randn(E, N, K, generator=g).cuda()
    W = qp.qquantize_rows_mx4(w)
    most = 2100
    n = qp.qgemm_w4_mx_dx_ws_size(most, W if E > 1 else W[0])
    assert n > 0
    room = torch.full((n + 256,), 0xa5, dtype=torch.uint8, device="cuda")
    ws = room[:n]
    X = torch.randn(most, N, generator=g).to(getattr(torch, dtype)).cuda()
    for M in (most, 1, 7, 15, 16, 31, 47, 100, 239, 300, most):
        print("mx4 workspace", dtype, N, K, E, M, flush=True)
        if E == 1:
            got = qp.qgemm_w4_mx_dx(X[:M], W[0], ws=ws)
            own = qp.qgemm_w4_mx_dx(X[:M], W[0])
        else:
            off = torch.tensor([0, M // 3, M // 2, M], dtype=torch.int32, device="cuda")
            got = qp.qgemm_w4_mx_experts_dx(X[:M], W, off, ws=ws)
            own = qp.qgemm_w4_mx_experts_dx(X[:M], W, off)
        assert torch.equal(got, own)
        assert (room[n:] == 0xa5).all()
    # calls of many rows need none
    if E == 1:
        assert "/" not in qp.qgemm_mx_kernel_name("w4_dx", most, W[0], torch.float32) or \
            qp.qgemm_mx_kernel_name("w4_dx", most, W[0], torch.float32).endswith("/1")
        none = torch.empty(0, dtype=torch.uint8, device="cuda")
        assert torch.equal(qp.qgemm_w4_mx_dx(X, W[0], ws=none), qp.qgemm_w4_mx_dx(X, W[0]))
