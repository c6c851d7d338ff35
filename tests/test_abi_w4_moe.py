"""What the float operators over int4 blobs and experts (qgemm_w4_*, qmoe_*)
refuse on the host, before any launch: a status, a message, no GPU needed."""
import ctypes as C

import pytest

P = 0x10000        # never dereferenced: every call below fails validation first
INF = float("inf")


@pytest.fixture(scope="module")
def qp():
    import conv_qpack_weights_amd as qp
    return qp


def _info(qp, N=70, K=129, group=32, fmt=2):
    """The description qpack_weights gives for such weights."""
    scheme = {2: qp.QP_BLOCKWISE, 3: qp.QP_BLOCKWISE_BF16, 4: qp.QP_BLOCKWISE_ASYM}[fmt]
    i = qp.PackedInfo()
    i.format, i.scheme, i.N, i.K, i.group = fmt, scheme, N, K, group
    up = lambda a, b: -(-a // b) * b
    i.Npad, i.Kpad = up(N, 64), up(K, max(group, 128))
    i.data_off, i.data_bytes = 256, i.Npad * i.Kpad // 2
    i.scale_off = 256 + up(i.data_bytes, 256)
    sb = up(4 * (2 if fmt == 3 else 4) * i.Npad * (-(-(i.Kpad // group) // 4)), 256)
    i.sum_off = i.scale_off + sb
    i.total_bytes = i.sum_off + up(4 * i.Npad, 256)
    if fmt == 4:
        i.zp_off = i.total_bytes
        i.total_bytes += sb
    return i


def _refused(qp, status, code, needle):
    assert status == code, (status, qp.last_error())
    assert needle in qp.last_error(), qp.last_error()


def _dense(qp, info, X=P, dtype=None, M=4, K=129, ldx=129, W=P, lo=-INF, hi=INF, Y=P, ydt=None,
           ldy=70):
    dtype = qp.QP_BF16 if dtype is None else dtype
    return qp.lib().qgemm_w4_blockwise(X, dtype, M, K, ldx, C.byref(info) if info else None, W,
                                       None, lo, hi, Y, dtype if ydt is None else ydt, ldy, None)


def test_dense_product_refusals(qp):
    i = _info(qp)
    for kw, code, needle in [
            (dict(M=-1), qp.QP_EINVAL, "negative"),
            (dict(M=1 << 31), qp.QP_EUNSUPPORTED, "rows"),
            (dict(M=(1 << 30) + 1), qp.QP_EUNSUPPORTED, "rows"),
            (dict(K=128), qp.QP_EINVAL, "K=128"),
            (dict(ldx=128), qp.QP_EINVAL, "stride of X"),
            (dict(ldy=69), qp.QP_EINVAL, "stride of Y"),
            (dict(X=None), qp.QP_EINVAL, "X is null"),
            (dict(Y=None), qp.QP_EINVAL, "Y is null"),
            (dict(W=None), qp.QP_EINVAL, "null"),
            (dict(W=P + 16), qp.QP_EALIGN, "256-byte"),
            (dict(X=P + 1), qp.QP_EALIGN, "X is not aligned"),
            (dict(dtype=qp.QP_S8), qp.QP_EINVAL, "QP_F32"),
            (dict(dtype=qp.QP_F16, ydt=qp.QP_BF16), qp.QP_EUNSUPPORTED, "rows' type"),
            (dict(dtype=qp.QP_F32, ydt=qp.QP_BF16), qp.QP_EUNSUPPORTED, "rows' type"),
            (dict(lo=1.0, hi=0.0), qp.QP_EINVAL, "reversed"),
            (dict(lo=float("nan")), qp.QP_EINVAL, "NaN")]:
        _refused(qp, _dense(qp, i, **kw), code, needle)
    _refused(qp, _dense(qp, None), qp.QP_EINVAL, "int4 blob")
    i8 = _info(qp)
    i8.format = 1
    _refused(qp, _dense(qp, i8), qp.QP_EINVAL, "int4 blob")
    assert _dense(qp, i, M=0, X=None, Y=None) == qp.QP_OK  # nothing to do


def test_more_threads_than_a_launch_has_are_refused(qp):
    i = _info(qp, N=65536, K=129)
    _refused(qp, _dense(qp, i, M=1 << 30, ldy=65536), qp.QP_EUNSUPPORTED, "2^32 threads")
    j = _info(qp, N=32, K=1 << 16)
    _refused(qp, qp.lib().qgemm_w4_blockwise_dx(P, qp.QP_BF16, 1 << 28, 32, C.byref(j), P, P,
                                                1 << 16, None, 0, None), qp.QP_EUNSUPPORTED,
             "2^32 threads")


@pytest.mark.parametrize("fmt", [2, 3, 4])
@pytest.mark.parametrize("field", ["Npad", "Kpad", "data_off", "scale_off", "zp_off",
                                   "total_bytes"])
def test_a_description_that_does_not_fit_its_shape_is_refused(qp, fmt, field):
    i = _info(qp, fmt=fmt)
    setattr(i, field, getattr(i, field) + 256)
    _refused(qp, _dense(qp, i), qp.QP_EINVAL, "description")
    _refused(qp, qp.lib().qgemm_w4_blockwise_dx(P, qp.QP_BF16, 4, 70, C.byref(i), P, P, 129, None,
                                                0, None), qp.QP_EINVAL, "description")


def _experts(qp, info, X=P, x_rows=8, K=129, ldx=129, rows=None, row_div=1, M=8, W=P, stride=None,
             E=4, offsets=P, Y=P, ldy=70):
    return qp.lib().qgemm_w4_experts(X, qp.QP_BF16, x_rows, K, ldx, rows, row_div, M,
                                     C.byref(info), W, info.total_bytes if stride is None else
                                     stride, E, offsets, None, -INF, INF, Y, qp.QP_BF16, ldy, None)


def test_experts_product_refusals(qp):
    i = _info(qp)
    for kw, code, needle in [
            (dict(M=-1), qp.QP_EINVAL, "negative"),
            (dict(x_rows=-1), qp.QP_EINVAL, "negative"),
            (dict(x_rows=7), qp.QP_EINVAL, "fewer than M"),
            (dict(rows=P, x_rows=0), qp.QP_EINVAL, "no rows"),
            (dict(rows=P, row_div=0), qp.QP_EINVAL, "row_div"),
            (dict(E=0), qp.QP_EINVAL, "expert"),
            (dict(E=65537), qp.QP_EUNSUPPORTED, "experts"),
            (dict(stride=i.total_bytes - 256), qp.QP_EINVAL, "total_bytes"),
            (dict(stride=i.total_bytes + 8), qp.QP_EINVAL, "multiple of 256"),
            (dict(offsets=None), qp.QP_EINVAL, "offsets"),
            (dict(K=130), qp.QP_EINVAL, "K=130"),
            (dict(ldy=1), qp.QP_EINVAL, "stride of Y")]:
        _refused(qp, _experts(qp, i, **kw), code, needle)
    assert _experts(qp, i, M=0, x_rows=0, X=None, Y=None) == qp.QP_OK


def test_gradient_refusals(qp):
    L = qp.lib()
    i = _info(qp, N=4096, K=4096)
    need = C.c_size_t()
    assert L.qgemm_w4_dx_ws_size(16, C.byref(i), 1, C.byref(need)) == qp.QP_OK
    assert need.value > 0                    # few rows: the channels are split
    call = lambda ws, n, **kw: L.qgemm_w4_blockwise_dx(
        kw.get("dY", P), kw.get("dtype", qp.QP_BF16), kw.get("M", 16), kw.get("lddy", 4096),
        C.byref(i), P, kw.get("dX", P), kw.get("lddx", 4096), ws, n, None)
    _refused(qp, call(P, need.value - 1), qp.QP_ESIZE, "workspace")
    _refused(qp, call(None, need.value), qp.QP_EALIGN, "workspace")
    _refused(qp, call(P + 16, need.value), qp.QP_EALIGN, "workspace")
    _refused(qp, call(P, need.value, lddy=4095), qp.QP_EINVAL, "stride of dY")
    _refused(qp, call(P, need.value, lddx=4095), qp.QP_EINVAL, "stride of dX")
    _refused(qp, call(P, need.value, dY=None), qp.QP_EINVAL, "dY is null")
    _refused(qp, call(P, need.value, dtype=qp.QP_S32), qp.QP_EINVAL, "QP_F32")
    _refused(qp, call(P, need.value, M=-1), qp.QP_EINVAL, "negative")
    _refused(qp, L.qgemm_w4_experts_dx(P, qp.QP_BF16, 16, 4096, C.byref(i), P, i.total_bytes, 4,
                                       None, P, 4096, None, 0, None), qp.QP_EINVAL, "offsets")
    _refused(qp, L.qgemm_w4_dx_ws_size(-1, C.byref(i), 1, C.byref(need)), qp.QP_EINVAL, "bad")
    _refused(qp, L.qgemm_w4_dx_ws_size(4, C.byref(i), 0, C.byref(need)), qp.QP_EINVAL, "bad")
    assert L.qgemm_w4_dx_ws_size(0, C.byref(i), 1, C.byref(need)) == qp.QP_OK and need.value == 0


def test_sort_and_dispatch_refusals(qp):
    L = qp.lib()
    sort = lambda **kw: L.qmoe_sort(
        kw.get("ids", P), kw.get("dt", qp.QP_S32), kw.get("T", 8), kw.get("k", 2),
        kw.get("ld", 2), kw.get("E", 4), kw.get("o", P), kw.get("r", P), kw.get("s", P),
        kw.get("ws", None), kw.get("n", 0), None)
    for kw, code, needle in [
            (dict(T=-1), qp.QP_EINVAL, "T >= 0"),
            (dict(k=0), qp.QP_EINVAL, "top_k"),
            (dict(k=1025, ld=1025), qp.QP_EUNSUPPORTED, "1024"),
            (dict(T=1 << 30), qp.QP_EUNSUPPORTED, "2^30"),
            (dict(dt=qp.QP_F32), qp.QP_EINVAL, "QP_S64"),
            (dict(ld=1), qp.QP_EINVAL, "ldids"),
            (dict(E=0), qp.QP_EINVAL, "expert"),
            (dict(E=513), qp.QP_EUNSUPPORTED, "512"),
            (dict(ids=None), qp.QP_EINVAL, "null"),
            (dict(o=None), qp.QP_EINVAL, "null"),
            (dict(r=None), qp.QP_EINVAL, "null"),
            (dict(s=None), qp.QP_EINVAL, "null"),
            (dict(ids=P + 4, dt=qp.QP_S64), qp.QP_EALIGN, "ids"),
            (dict(T=5000), qp.QP_ESIZE, "workspace"),
            (dict(T=5000, n=1 << 30), qp.QP_EALIGN, "workspace")]:
        _refused(qp, sort(**kw), code, needle)
    assert qp.qmoe_sort_ws_size(8, 2, 4) == 0 and qp.qmoe_sort_ws_size(5000, 2, 4) > 0

    disp = lambda **kw: L.qmoe_dispatch(
        kw.get("X", P), kw.get("dt", qp.QP_BF16), kw.get("H", 64), kw.get("ldx", 64), P, qp.QP_S32,
        8, 2, 2, 4, kw.get("Xs", P), kw.get("ldxs", 64), P, P, P, None, 0, None)
    for kw, code, needle in [
            (dict(dt=qp.QP_S8), qp.QP_EINVAL, "QP_F32"),
            (dict(H=0), qp.QP_EINVAL, "row length"),
            (dict(ldx=63), qp.QP_EINVAL, "X needs"),
            (dict(ldxs=63), qp.QP_EINVAL, "Xs needs"),
            (dict(H=(1 << 24) + 1, ldx=1 << 25, ldxs=1 << 25), qp.QP_EUNSUPPORTED, "2^24"),
            (dict(X=None), qp.QP_EINVAL, "X is null"),
            (dict(Xs=P + 1), qp.QP_EALIGN, "Xs is not aligned")]:
        _refused(qp, disp(**kw), code, needle)


def test_combine_and_gradient_refusals(qp):
    L = qp.lib()
    comb = lambda **kw: L.qmoe_combine(
        kw.get("Z", P), kw.get("dt", qp.QP_F16), kw.get("T", 8), kw.get("k", 2), 64,
        kw.get("ldz", 64), kw.get("r", P), kw.get("w", P), kw.get("ldw", 2), kw.get("Y", P),
        kw.get("ldy", 64), None)
    for kw, code, needle in [
            (dict(dt=qp.QP_S64), qp.QP_EINVAL, "QP_F32"), (dict(T=-1), qp.QP_EINVAL, "T >= 0"),
            (dict(ldz=63), qp.QP_EINVAL, "Z needs"), (dict(ldy=63), qp.QP_EINVAL, "Y needs"),
            (dict(Z=None), qp.QP_EINVAL, "Z is null"), (dict(r=None), qp.QP_EINVAL, "null"),
            (dict(w=None), qp.QP_EINVAL, "null"), (dict(ldw=1), qp.QP_EINVAL, "stride"),
            (dict(Z=P + 1), qp.QP_EALIGN, "Z is not aligned")]:
        _refused(qp, comb(**kw), code, needle)
    grad = lambda **kw: L.qmoe_combine_grad(
        kw.get("dY", P), 64, P, 64, qp.QP_F16, 8, 2, 64, P, kw.get("s", P), P, kw.get("ldw", 2),
        kw.get("dZ", P), 64, kw.get("dw", P), kw.get("lddw", 2), None)
    for kw, code, needle in [
            (dict(dY=None), qp.QP_EINVAL, "dY is null"), (dict(dZ=None), qp.QP_EINVAL, "dZ is null"),
            (dict(s=None), qp.QP_EINVAL, "null"), (dict(dw=None), qp.QP_EINVAL, "null"),
            (dict(ldw=1), qp.QP_EINVAL, "stride"), (dict(lddw=1), qp.QP_EINVAL, "stride")]:
        _refused(qp, grad(**kw), code, needle)
    _refused(qp, L.qmoe_dispatch_grad(P, qp.QP_F16, 8, 2, 64, 64, None, P, 64, None), qp.QP_EINVAL,
             "null")
    _refused(qp, L.qmoe_dispatch_grad(P, qp.QP_F16, 8, 2, 64, 63, P, P, 64, None), qp.QP_EINVAL,
             "dXs needs")


def test_the_binding_checks_its_tensors(qp):
    """Types, shapes and strides are looked at before anything is allocated."""
    import torch
    i = _info(qp, 48, 64)
    blob = torch.zeros(i.total_bytes, dtype=torch.uint8)
    with pytest.raises(AssertionError):
        qp.qgemm_w4_blockwise(torch.zeros(4, 64, dtype=torch.int32), blob, i)
    with pytest.raises(AssertionError):
        qp.qgemm_w4_blockwise(torch.zeros(64, 4).t(), blob, i)
    with pytest.raises(AssertionError):
        qp.qgemm_w4_blockwise(torch.zeros(4, 64), blob, i, out=torch.zeros(4, 47))
    with pytest.raises(AssertionError):
        qp.qgemm_w4_blockwise(torch.zeros(4, 64), blob, i, bias=torch.zeros(47))
    with pytest.raises(AssertionError):
        qp.qgemm_w4_experts(torch.zeros(4, 64), blob.view(1, -1), i,
                            torch.zeros(3, dtype=torch.int32))
    with pytest.raises(AssertionError):
        qp.qgemm_w4_experts(torch.zeros(4, 64), blob.view(1, -1), i,
                            torch.zeros(2, dtype=torch.int64))
    with pytest.raises(AssertionError):
        qp.qgemm_w4_blockwise_dx(torch.zeros(4, 47), blob, i)
    with pytest.raises(AssertionError):
        qp.qmoe_sort(torch.zeros(4, 2, dtype=torch.int16), 4)
    with pytest.raises(AssertionError):
        qp.qmoe_dispatch(torch.zeros(3, 64), torch.zeros(4, 2, dtype=torch.int32), 4)
    with pytest.raises(AssertionError):
        qp.qmoe_combine(torch.zeros(8, 64), torch.zeros(4, 2, dtype=torch.int32),
                        torch.zeros(4, 2, dtype=torch.float16))
    with pytest.raises(AssertionError):
        qp.qmoe_combine(torch.zeros(7, 64), torch.zeros(4, 2, dtype=torch.int32),
                        torch.zeros(4, 2))
