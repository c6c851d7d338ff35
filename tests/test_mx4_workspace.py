"""The workspace of the MXFP4 gradients (host only): a size for M rows serves every call
of fewer, of any type."""
import ctypes as C

import pytest

P = 0x10000        # never dereferenced


@pytest.fixture(scope="module")
def qp():
    import conv_qpack_weights_amd as qp
    return qp


def _desc(qp, N, K, E):
    G = -(-K // 32)
    ldc, lds = 16 * G, -(-G // 4) * 4
    return qp.Mx4Desc(P, P, N, K, ldc, lds, E, N * ldc, N * lds)


def _size(qp, M, d):
    n = C.c_size_t()
    assert qp.lib().qgemm_w4_mx_dx_ws_size(M, C.byref(d), C.byref(n)) == qp.QP_OK
    return n.value


def _splits(qp, M, d, dtype):
    name = C.create_string_buffer(32)
    assert qp.lib().qgemm_mx_kernel_name(qp.QP_MX_W4_DX, M, C.byref(d), dtype, name, 32) == qp.QP_OK
    name = name.value.decode()
    return int(name.split("/")[1]) if "/" in name else 1


@pytest.mark.parametrize("N,K,E", [(4096, 4096, 1), (11008, 4096, 1), (4096, 128, 1), (1037, 1100, 1),
                                   (257, 4096, 1), (512, 100, 1), (4096, 4096, 8), (700, 64, 70),
                                   (4096, 33, 3), (8192, 128, 16), (2000, 256, 300)])
def test_a_size_serves_all_fewer_rows(qp, N, K, E):
    d, last, reached = _desc(qp, N, K, E), 0, 0
    assert _size(qp, 0, d) == 0
    for M in list(range(1, 300)) + list(range(300, 9000, 37)):
        size = _size(qp, M, d)
        assert last <= size <= 4 << 20, M
        last = size
        for dtype in (qp.QP_F32, qp.QP_BF16, qp.QP_F16):
            splits = _splits(qp, M, d, dtype)
            need = 4 * splits * M * K if splits > 1 else 0
            assert need <= size, (M, dtype)
            reached = max(reached, need)
    assert reached > 0.9 * last                               # and is no more than some need


def test_no_room_where_no_call_splits(qp):
    for N, K, E in [(256, 4096, 1), (4096, 128 * 512, 1), (64, 64, 4)]:
        d = _desc(qp, N, K, E)
        assert all(_size(qp, M, d) == 0 for M in (1, 16, 300, 5000))
