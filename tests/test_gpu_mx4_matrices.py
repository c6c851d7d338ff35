"""MXFP4 matrices whose tensors move, on the GPU: the operators read where they are."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qp():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    import conv_qpack_weights_amd as qp
    return qp


def test_weights_of_a_module_that_moves(qp):
    """Made from parameters on the host, used on the card; then new tensors with other
    values at other places, and values loaded into them."""
    import torch
    g = torch.Generator().manual_seed(3)
    m = torch.nn.Module()
    made = lambda E: (torch.randint(0, 256, (E, 70, 96), generator=g, dtype=torch.uint8),
                      torch.randint(118, 130, (E, 70, 8), generator=g, dtype=torch.uint8)[..., :6])
    codes, scales = made(3)
    m.codes = torch.nn.Parameter(codes, requires_grad=False)
    m.scales = torch.nn.Parameter(scales, requires_grad=False)
    W = qp.mx4_tensor(m.codes, m.scales, 192)
    assert W.codes is m.codes
    X = torch.randn(9, 192, generator=g).bfloat16().cuda()
    A = qp.qquantize_rows_mx4(X)
    dY = torch.randn(9, 70, generator=g).bfloat16().cuda()
    offsets = torch.tensor([0, 4, 4, 9], dtype=torch.int32, device="cuda")

    def run(w):
        return [qp.qgemm_w4_mx_experts(X, w, offsets), qp.qgemm_a4w4_mx_experts(A, w, offsets),
                qp.qgemm_w4_mx_experts_dx(dY, w, offsets), qp.qgemm_w4_mx(X, w[2]),
                qp.qgemm_a4w4_mx(A, w[1]), qp.qgemm_w4_mx_dx(dY, w[0]), qp.qdequantize_rows_mx4(w[1])]

    def same():
        fresh = qp.mx4_tensor(m.codes.clone(), m.scales.clone(), 192)
        assert all(torch.equal(a, b) for a, b in zip(run(W), run(fresh)))

    with pytest.raises(AssertionError, match="on (the|one) GPU"):
        run(W)
    # (to() of scales in rows of whole words loses the padding)
    card = torch.zeros(3, 70, 8, dtype=torch.uint8, device="cuda")[..., :6].copy_(scales)
    m.codes.data, m.scales.data = codes.cuda(), card
    W = qp.MX4(m.codes, m.scales, 192)
    same()
    codes, scales = made(3)
    m.codes.data = codes.cuda()
    m.scales.data = torch.zeros(3, 70, 8, dtype=torch.uint8, device="cuda")[..., :6].copy_(scales)
    same()
    m.codes.copy_(made(3)[0])
    same()
    m._apply(lambda t: t.clone() if t.dim() == 3 and t.is_contiguous() else t)
    same()
