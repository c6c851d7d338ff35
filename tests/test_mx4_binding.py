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


def _where(d):
    return (d.codes, d.scales, d.rows, d.K, d.ld_codes, d.ld_scales, d.matrices, d.codes_stride,
            d.scales_stride)


def _moved(m):
    """A new tensor for every parameter, as module.to() of another place makes."""
    m._apply(lambda t: t.clone())
    return m


class Layer(torch.nn.Module):
    def __init__(self, E=3, N=48, G=4):
        super().__init__()
        self.codes = torch.nn.Parameter(_u(E, N, 16 * G), requires_grad=False)
        self.scales = torch.nn.Parameter(_u(E, N, G), requires_grad=False)


def test_a_modules_parameters_move_under_their_matrix(qp):
    m = Layer()
    W = qp.mx4_tensor(m.codes, m.scales)
    old, kept = _where(W.desc), (m.codes.data, m.scales.data)
    _moved(m)
    assert m.codes.data_ptr() != old[0] and m.scales.data_ptr() != old[1]
    assert _where(W.desc) == (m.codes.data_ptr(), m.scales.data_ptr(), *old[2:])
    one = W[1]
    assert one.desc.codes == m.codes.data_ptr() + 48 * 64
    # a single matrix keeps the place it was taken from, which its tensors hold
    _moved(m)
    assert one.desc.codes == one.codes.data_ptr() != m.codes.data_ptr() + 48 * 64
    # other shapes and strides, at another address and at the same one
    m.codes.data, m.scales.data = _u(2, 48, 64), _u(2, 48, 4)
    assert W.shape == (2, 48, 128) and W.desc.matrices == 2
    wide, more = _u(2, 48, 96), _u(2, 48, 8)
    m.codes.data, m.scales.data = wide[..., :64], more[..., :4]
    assert _where(W.desc) == (wide.data_ptr(), more.data_ptr(), 48, 128, 96, 8, 2, 48 * 96, 48 * 8)
    m.codes.data, m.scales.data = wide[:1, :, :64], more[:1, :, :4]
    assert W.desc.matrices == 1 and W.desc.codes == wide.data_ptr()
    m.codes.data, m.scales.data = wide.view(2, 96, 48)[:, :48], more.view(2, 96, 4)[:, :48]
    with pytest.raises(AssertionError, match="16 bytes a block"):
        W.desc


def test_a_move_that_loses_the_padding_is_refused(qp):
    """Scales of 5 blocks in rows of 8 bytes, copied without what is behind them."""
    m = Layer(G=5)
    m.scales = torch.nn.Parameter(_u(3, 48, 8)[..., :5], requires_grad=False)
    W = qp.MX4(m.codes, m.scales, 160)
    assert W.desc.ld_scales == 8
    m.scales.data = m.scales.data.contiguous()
    for _ in range(2):
        with pytest.raises(AssertionError, match="mx4_tensor"):
            W.desc
    W = qp.mx4_tensor(m.codes, m.scales)
    assert W.desc.ld_scales == 8


def test_the_librarys_own_matrices_are_followed_once_given_away(qp, monkeypatch):
    """Rows that the library made keep their place; tensors asked for may be moved."""
    made = qp.MX4._new(torch.zeros(1), (3,), 5, 150)
    d = made.desc
    assert (d.rows, d.K, d.ld_codes, d.ld_scales, d.matrices, d.codes_stride, d.scales_stride) == \
        (5, 150, 80, 8, 3, 400, 40)
    assert made.shape == (3, 5, 150) and made.codes.shape == (3, 5, 80) and \
        made.scales.shape == (3, 5, 5) and made.scales.stride() == (40, 8, 1)
    assert _where(qp.MX4(made.codes, made.scales, 150).desc) == _where(made.desc)
    made.codes.data = made.codes.data.clone()
    assert made.desc.codes == made.codes.data_ptr() != d.codes
    # one row or none: as the constructor describes them
    for lead, rows in (((), 1), ((), 0), ((2,), 1), ((), 7)):
        m = qp.MX4._new(torch.zeros(1), lead, rows, 70)
        a, b = _where(m.desc), _where(qp.MX4(m.codes, m.scales, 70).desc)
        assert a == b
    with pytest.raises(AttributeError):
        made.codes = _u(3, 5, 80)


@pytest.mark.parametrize("e", [0, 2, -1])
def test_an_experts_matrix(qp, e):
    W = qp.mx4_tensor(_u(3, 6, 80), _u(3, 6, 5), 150)
    one, same = W[e], qp.MX4(W.codes[e], W.scales[e], 150)
    assert _where(one.desc) == _where(same.desc) and one.shape == (6, 150)
    assert one.codes.data_ptr() == W.codes[e].data_ptr()
    two = W[1:]
    assert two.desc.matrices == 2 and two.desc.codes == W.desc.codes + W.desc.codes_stride
    with pytest.raises(IndexError):
        W[3]
    single = qp.mx4_tensor(_u(3, 1, 80), _u(3, 1, 5), 150)
    assert _where(single[e].desc) == _where(qp.MX4(single.codes[e], single.scales[e], 150).desc)


def test_copies_follow_their_tensors(qp):
    """A copy shares the tensors of a matrix that the library made; a deep one has its own,
    the padding behind the rows with them."""
    import copy
    made = qp.MX4._new(torch.zeros(1), (3,), 5, 150)
    made_codes = made._codes
    other = copy.copy(made)
    assert other.codes is made_codes and _where(other.desc) == _where(made.desc)
    made_codes.data = made_codes.data.clone()
    assert other.desc.codes == made.desc.codes == made_codes.data_ptr()
    deep = copy.deepcopy(made)
    d = deep.desc
    assert (d.codes, d.scales) == (deep.codes.data_ptr(), deep.scales.data_ptr())
    assert d.codes != made.desc.codes and _where(d)[2:] == _where(made.desc)[2:]
