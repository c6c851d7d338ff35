"""Which kernel the MXFP4 products take (host only): the sizes each is there for."""
import pytest


@pytest.fixture(scope="module")
def qp():
    import conv_qpack_weights_amd as qp
    return qp


def _weights(qp, N, K, E=1):
    import torch
    # (nothing is read: the description alone is asked for)
    w = qp.MX4(torch.empty(1, 1, 16, dtype=torch.uint8), torch.empty(1, 1, 4, dtype=torch.uint8)[..., :1],
               32)
    w.K = K
    d, G = w.desc, -(-K // 32)
    d.rows, d.K, d.matrices = N, K, E
    d.ld_codes, d.ld_scales = 16 * G, -(-G // 4) * 4
    d.codes_stride, d.scales_stride = N * d.ld_codes, N * d.ld_scales
    return w


# product, row type, M, N, K, experts, kernel
CHOICES = [
    ("a4w4", "bf16", 1, 4096, 4096, 1, "rows16x16"),
    ("a4w4", "bf16", 64, 4096, 4096, 1, "rows16x32"),
    ("a4w4", "bf16", 128, 11008, 4096, 16, "rows16x32"),
    ("a4w4", "bf16", 256, 4096, 4096, 1, "tile64x64"),
    ("a4w4", "bf16", 512, 11008, 4096, 1, "tile128x128"),
    ("a4w4", "bf16", 8192, 8192, 8192, 1, "tile256x256"),
    ("w4", "bf16", 1, 4096, 4096, 1, "rows16x16"),
    ("w4", "f16", 32, 4096, 4096, 1, "rows16x32"),
    ("w4", "bf16", 16, 11008, 4096, 1, "rows16x48"),
    ("w4", "f16", 64, 4096, 4096, 1, "rows16x64"),
    ("w4", "f16", 146, 4900, 4096, 1, "tile32x64"),
    ("w4", "bf16", 512, 4096, 4096, 1, "tile32x128"),
    ("w4", "bf16", 1024, 4096, 4096, 1, "tile128x128"),
    ("w4", "f16", 8192, 11008, 4096, 1, "tile256x256"),
    ("w4", "bf16", 128, 11008, 4096, 16, "rows16x64"),
    ("w4", "bf16", 256, 11008, 4096, 16, "tile32x128"),
    ("w4", "bf16", 8192, 11008, 4096, 8, "tile256x256"),
    ("w4", "f32", 1, 4096, 4096, 1, "rows16x16"),
    ("w4", "f32", 32, 4096, 4096, 1, "rows16x32"),
    ("w4", "f32", 16, 11008, 4096, 1, "rows16x48"),
    ("w4", "f32", 64, 4096, 4096, 1, "rows16x64"),
    ("w4", "f32", 4096, 4096, 4096, 1, "tile128x128"),
    ("w4_dx", "bf16", 16, 4096, 4096, 1, "rows16x128/8"),
    ("w4_dx", "f16", 256, 4096, 4096, 1, "rows16x128/1"),
    ("w4_dx", "bf16", 1024, 4096, 4096, 1, "tile128x128"),
    ("w4_dx", "f16", 4096, 4096, 4096, 1, "tile256x256"),
    ("w4_dx", "f32", 256, 4096, 4096, 1, "rows16x128/1"),
    ("w4_dx", "f32", 4096, 4096, 4096, 1, "tile128x128"),
]


@pytest.mark.parametrize("product,dtype,M,N,K,E,kernel", CHOICES)
def test_sizes_take_their_kernels(qp, product, dtype, M, N, K, E, kernel):
    import torch
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    assert qp.qgemm_mx_kernel_name(product, M, _weights(qp, N, K, E), dt) == kernel


def test_refusals(qp):
    import ctypes as C
    w = _weights(qp, 64, 64)
    name = C.create_string_buffer(32)
    call = lambda product=1, M=4, dtype=qp.QP_F32, buf=name, n=32: qp.lib().qgemm_mx_kernel_name(
        product, M, C.byref(w.desc), dtype, buf, n)
    assert call() == qp.QP_OK
    for kw, needle in [(dict(product=3), "product"), (dict(M=0), "row"), (dict(dtype=qp.QP_S8), "rows"),
                       (dict(buf=None), "room"), (dict(n=8), "room")]:
        assert call(**kw) == qp.QP_EINVAL and needle in qp.last_error()
