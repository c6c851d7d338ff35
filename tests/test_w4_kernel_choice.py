"""Which kernel the int4 products take, on the host: the sizes that the GPU tests
use for each kernel do select it, and every kernel has such sizes."""
import ctypes as C

import pytest
import torch

from test_gpu_w4_kernels import FORWARD, GRADIENT, KINDS, TYPES, _dt, forward_kernel
from test_w4_moe_binding import _info


@pytest.fixture(scope="module")
def qp():
    import conv_qpack_weights_amd as qp
    return qp


@pytest.mark.parametrize("dtype", TYPES)
def test_the_sizes_of_the_kernel_tests_select_their_kernels(qp, dtype):
    for name, sizes in FORWARD.items():
        for E, (M, N, K) in zip((1, 3), sizes):
            assert qp.qgemm_w4_kernel_name(M, _info(qp, N, K), _dt(dtype), E) == \
                forward_kernel(name, dtype)
    for name, sizes in GRADIENT.items():
        for E, (M, N, K) in zip((1, 3), sizes):
            if name != "tile" or dtype == "bf16":
                assert qp.qgemm_w4_kernel_name(M, _info(qp, N, K), _dt(dtype), E,
                                               gradient=True) == name


def test_every_kernel_that_any_size_selects_is_among_them(qp):
    sizes = [1, 7, 16, 17, 40, 64, 100, 128, 300, 700, 1024, 2048, 5000, 16384]
    for E in (1, 2, 8, 64):
        for M in sizes:
            for N in (1, 64, 500, 1024, 4096, 11008, 40000):
                for dtype in (torch.float32, torch.bfloat16, torch.float16):
                    i = _info(qp, N, 64)
                    assert qp.qgemm_w4_kernel_name(M, i, dtype, E) in FORWARD
                    for K in (100, 1024, 4096, 11008):
                        name = qp.qgemm_w4_kernel_name(M, _info(qp, N, K), dtype, E, gradient=True)
                        assert name in GRADIENT, name


def test_refusals(qp):
    i = _info(qp)
    room = C.create_string_buffer(32)
    call = lambda M=4, w=i, dt=qp.QP_BF16, E=1, name=room, n=32: qp.lib().qgemm_w4_kernel_name(
        M, None if w is None else C.byref(w), dt, E, 0, name, n)
    assert call() == qp.QP_OK
    for kw in (dict(M=0), dict(M=(1 << 30) + 1), dict(w=None), dict(dt=qp.QP_S8), dict(E=0),
               dict(name=None), dict(n=15)):
        assert call(**kw) == qp.QP_EINVAL and "qgemm_w4_kernel_name" in qp.last_error()
