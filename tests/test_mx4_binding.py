"""The binding's MXFP4 matrix (MX4) on the host: what its constructor refuses, and that
what the library is told of a matrix is where its tensors are.  No GPU needed."""
import pytest
import torch


@pytest.fixture(scope="module")
def qp():
    import conv_qpack_weights_amd as qp
    return qp


def _u(*s):
    return torch.zeros(*s, dtype=torch.uint8)


@pytest.mark.parametrize("codes,scales,K,needle", [
    (_u(4, 64), _u(400, 4), 128, "alike"),                   # rows of codes that are not there
    (_u(2, 4, 64), _u(4, 4), 128, "alike"), (_u(64), _u(4), 128, "alike"),
    (_u(4, 48), _u(4, 4), 128, "16 bytes a block"), (_u(4, 64), _u(4, 3), 96, "16 bytes a block"),
    (_u(4, 0), _u(4, 0), 1, "block"),
    (_u(4, 64).int(), _u(4, 4), 128, "uint8"), (_u(4, 64), _u(4, 4).to(torch.int8), 128, "uint8"),
    (_u(4, 64), _u(4, 4), 129, "does not fit"), (_u(4, 64), _u(4, 4), 96, "does not fit"),
    (_u(4, 64), _u(4, 4), 0, "does not fit"),
    (_u(64, 4).t(), _u(4, 4), 128, "side by side"), (_u(4, 64), _u(4, 4).t(), 128, "side by side"),
    (_u(1, 64).expand(4, 64), _u(4, 4), 128, "overlap"),
    (_u(4, 64), _u(1, 4).expand(4, 4), 128, "overlap"),
    (_u(4, 80), _u(4, 5), 160, "overlap"),                   # words of one row's scales in the next
    (_u(4, 80), _u(35).as_strided((4, 5), (8, 1), 4), 160, "last word"),
    (_u(1, 80), _u(1, 5), 160, "last word"),
    (_u(3, 1, 80), _u(3, 1, 5), 160, "last word"),
    (_u(3, 2, 80), _u(47).as_strided((3, 2, 5), (16, 8, 1)), 160, "last word")])
def test_matrices_that_are_not_there(qp, codes, scales, K, needle):
    with pytest.raises(AssertionError, match=needle):
        qp.MX4(codes, scales, K)


def test_matrices_of_wider_buffers(qp):
    """Rows of wider codes and scales, the last one's padding at the buffer's very end."""
    codes, scales = _u(4, 160), _u(4, 12)
    m = qp.MX4(codes[:, 16:96], scales[:, 4:9], 150)
    d = m.desc
    assert (d.rows, d.K, d.ld_codes, d.ld_scales, d.matrices) == (4, 150, 160, 12, 1)
    assert (d.codes, d.scales) == (codes.data_ptr() + 16, scales.data_ptr() + 4)
    e = qp.MX4(_u(3, 2, 80), _u(48).as_strided((3, 2, 5), (16, 8, 1)), 160)
    d = e.desc
    assert (d.matrices, d.codes_stride, d.scales_stride, d.ld_scales) == (3, 160, 16, 8)
    one = e[2]
    assert one.shape == (2, 160) and one.desc.scales == d.scales + 32
    assert qp.MX4(_u(1, 80), _u(1, 8)[:, :5], 160).desc.ld_scales == 8
    assert qp.MX4(_u(0, 80), _u(0, 5), 160).desc.rows == 0
    assert qp.MX4(_u(3, 0, 80), _u(3, 0, 5), 160).desc.matrices == 3
    assert qp.MX4(_u(2, 16), _u(8).as_strided((2, 1), (4, 1)), 1).desc.ld_scales == 4
