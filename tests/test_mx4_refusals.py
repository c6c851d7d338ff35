"""What the MXFP4 operators refuse on the host: the C entry points with a status and
a message, the binding before anything reaches the library.  No GPU needed."""
import ctypes as C

import pytest
import torch

P = 0x10000        # never dereferenced: every call below fails validation first
INF = float("inf")


@pytest.fixture(scope="module")
def qp():
    import conv_qpack_weights_amd as qp
    return qp


def _desc(qp, rows=70, K=100, codes=P, scales=P, ldc=None, lds=None, matrices=1, cs=None, ss=None):
    d = qp.Mx4Desc()
    G = -(-K // 32)
    d.codes, d.scales, d.rows, d.K = codes, scales, rows, K
    d.ld_codes = 16 * G if ldc is None else ldc
    d.ld_scales = -(-G // 4) * 4 if lds is None else lds
    d.matrices = matrices
    d.codes_stride = d.ld_codes * rows if cs is None else cs
    d.scales_stride = d.ld_scales * rows if ss is None else ss
    return d


def _refused(qp, status, code, needle):
    assert status == code, (status, qp.last_error())
    assert needle in qp.last_error(), qp.last_error()


BAD_MATRIX = [
    (dict(rows=-1), "QP_EINVAL", "rows"), (dict(K=0), "QP_EINVAL", "K=0"),
    (dict(K=(1 << 22) + 1), "QP_EUNSUPPORTED", "2^22"),
    (dict(rows=(1 << 30) + 1), "QP_EUNSUPPORTED", "2^30"),
    (dict(ldc=48), "QP_EINVAL", "codes' stride"), (dict(lds=3), "QP_EINVAL", "scales' stride"),
    (dict(ldc=(1 << 23) + 16), "QP_EUNSUPPORTED", "2^23"),
    (dict(codes=None), "QP_EINVAL", "null"), (dict(scales=None), "QP_EINVAL", "null"),
    (dict(codes=P + 8), "QP_EALIGN", "16 bytes"), (dict(ldc=72), "QP_EALIGN", "16 bytes"),
    (dict(scales=P + 2), "QP_EALIGN", "4 bytes"), (dict(lds=6), "QP_EALIGN", "4 bytes"),
    (dict(matrices=0), "QP_EINVAL", "at least one"),
    (dict(matrices=65537), "QP_EUNSUPPORTED", "65536"),
    (dict(matrices=2, cs=8), "QP_EALIGN", "16 bytes"),
    (dict(matrices=2, ss=2), "QP_EALIGN", "4 bytes"),
    (dict(matrices=2, cs=-16), "QP_EINVAL", "negative"),
]


@pytest.mark.parametrize("kw,code,needle", BAD_MATRIX)
def test_matrices_that_are_refused(qp, kw, code, needle):
    L, ok, bad = qp.lib(), _desc(qp), _desc(qp, **kw)
    code = getattr(qp, code)
    B, K = C.byref, bad.K
    lo = dict(clamp=(-INF, INF))["clamp"]
    _refused(qp, L.qgemm_w4_mx(P, qp.QP_BF16, 4, K, 1 << 23, B(bad), None, *lo, P, qp.QP_BF16,
                               1 << 31, None), code, needle)
    _refused(qp, L.qgemm_w4_mx_experts(P, qp.QP_BF16, 4, K, 1 << 23, None, 1, 4, B(bad), P, None, *lo,
                                       P, qp.QP_BF16, 1 << 31, None), code, needle)
    _refused(qp, L.qgemm_w4_mx_dx(P, qp.QP_BF16, 4, 1 << 31, B(bad), P, 1 << 23, None, 0, None),
             code, needle)
    _refused(qp, L.qgemm_w4_mx_experts_dx(P, qp.QP_BF16, 4, 1 << 31, B(bad), P, P, 1 << 23, None, 0,
                                          None), code, needle)
    n = C.c_size_t()
    _refused(qp, L.qgemm_w4_mx_dx_ws_size(4, B(bad), B(n)), code, needle)
    for a, w in ((bad, ok), (ok, bad)):
        _refused(qp, L.qgemm_a4w4_mx(B(a), B(w), None, *lo, P, qp.QP_F32, 1 << 31, None), code, needle)
        _refused(qp, L.qgemm_a4w4_mx_experts(B(a), None, 1, 4, B(w), P, None, *lo, P, qp.QP_F32,
                                             1 << 31, None), code, needle)
    _refused(qp, L.qdequantize_rows_mx4(B(bad), P, qp.QP_F32, 1 << 23, None), code, needle)
    if bad.matrices == 1:
        _refused(qp, L.qquantize_rows_mx4(P, qp.QP_F32, bad.rows, bad.K, 1 << 23, 0, bad.codes,
                                          bad.ld_codes, bad.scales, bad.ld_scales, None), code, needle)


def test_product_refusals(qp):
    L, B = qp.lib(), C.byref
    w = _desc(qp)

    def w4(X=P, dtype=None, M=4, K=100, ldx=100, w=w, lo=-INF, hi=INF, Y=P, ydt=None, ldy=70):
        dtype = qp.QP_BF16 if dtype is None else dtype
        return L.qgemm_w4_mx(X, dtype, M, K, ldx, B(w) if w else None, None, lo, hi, Y,
                             dtype if ydt is None else ydt, ldy, None)

    for kw, code, needle in [
            (dict(M=-1), qp.QP_EINVAL, "negative"),
            (dict(M=(1 << 30) + 1), qp.QP_EUNSUPPORTED, "rows"),
            (dict(K=128, ldx=128), qp.QP_EINVAL, "K=128"),
            (dict(ldx=99), qp.QP_EINVAL, "stride of X"), (dict(ldy=69), qp.QP_EINVAL, "stride of Y"),
            (dict(X=None), qp.QP_EINVAL, "X is null"), (dict(Y=None), qp.QP_EINVAL, "Y is null"),
            (dict(X=P + 1), qp.QP_EALIGN, "X is not aligned"),
            (dict(Y=P + 1), qp.QP_EALIGN, "Y is not aligned"), (dict(w=None), qp.QP_EINVAL, "null"),
            (dict(dtype=qp.QP_S8), qp.QP_EINVAL, "X must be"),
            (dict(ydt=qp.QP_F16), qp.QP_EUNSUPPORTED, "f32"),
            (dict(lo=1.0, hi=0.0), qp.QP_EINVAL, "clamp"),
            (dict(lo=float("nan")), qp.QP_EINVAL, "clamp"),
            (dict(w=_desc(qp, rows=0)), qp.QP_EINVAL, "no rows"),
            (dict(w=_desc(qp, matrices=2)), qp.QP_EINVAL, "one matrix")]:
        _refused(qp, w4(**kw), code, needle)

    def a4(a=_desc(qp, rows=4), w=w, lo=-INF, hi=INF, Y=P, ydt=qp.QP_BF16, ldy=70):
        return L.qgemm_a4w4_mx(B(a), B(w), None, lo, hi, Y, ydt, ldy, None)

    for kw, code, needle in [
            (dict(a=_desc(qp, rows=4, K=96)), qp.QP_EINVAL, "K=96"),
            (dict(a=_desc(qp, rows=4, matrices=2)), qp.QP_EINVAL, "one matrix"),
            (dict(w=_desc(qp, matrices=2)), qp.QP_EINVAL, "one matrix"),
            (dict(ldy=69), qp.QP_EINVAL, "stride of Y"), (dict(Y=None), qp.QP_EINVAL, "Y is null"),
            (dict(ydt=qp.QP_S32), qp.QP_EINVAL, "Y must be"),
            (dict(lo=2.0, hi=1.0), qp.QP_EINVAL, "clamp")]:
        _refused(qp, a4(**kw), code, needle)

    we = _desc(qp, matrices=3)

    def experts(x_rows=4, rows=None, div=1, M=4, off=P):
        s = [L.qgemm_w4_mx_experts(P, qp.QP_BF16, x_rows, 100, 100, rows, div, M, B(we), off, None,
                                   -INF, INF, P, qp.QP_BF16, 70, None)]
        e = [qp.last_error()]
        s.append(L.qgemm_a4w4_mx_experts(B(_desc(qp, rows=max(x_rows, 0))), rows, div, M, B(we), off,
                                         None, -INF, INF, P, qp.QP_BF16, 70, None))
        return list(zip(s, e + [qp.last_error()]))

    for kw, needle in [(dict(off=None), "offsets is null"), (dict(x_rows=3), "fewer"),
                       (dict(rows=P, div=0), "row_div"), (dict(rows=P, div=1 << 31), "row_div"),
                       (dict(rows=P, x_rows=0), "no rows"), (dict(M=-1), "negative")]:
        for status, message in experts(**kw):
            assert status == qp.QP_EINVAL and needle in message, (kw, message)


def test_gradient_and_quantizer_refusals(qp):
    L, B = qp.lib(), C.byref
    w = _desc(qp, rows=4096, K=4096)
    n = C.c_size_t()
    assert L.qgemm_w4_mx_dx_ws_size(16, B(w), B(n)) == qp.QP_OK
    need = n.value
    assert need > 0

    def dx(dY=P, dtype=qp.QP_BF16, M=16, lddy=4096, w=w, dX=P, lddx=4096, ws=P, bytes_=need):
        return L.qgemm_w4_mx_dx(dY, dtype, M, lddy, B(w), dX, lddx, ws, bytes_, None)

    for kw, code, needle in [
            (dict(M=-1), qp.QP_EINVAL, "negative"), (dict(lddy=4095), qp.QP_EINVAL, "stride of dY"),
            (dict(lddx=4095), qp.QP_EINVAL, "stride of dX"), (dict(dY=None), qp.QP_EINVAL, "dY is null"),
            (dict(dX=None), qp.QP_EINVAL, "dX is null"), (dict(dtype=9), qp.QP_EINVAL, "dY must be"),
            (dict(bytes_=need - 1), qp.QP_ESIZE, "workspace"), (dict(ws=None), qp.QP_EALIGN, "workspace"),
            (dict(ws=P + 128), qp.QP_EALIGN, "workspace"),
            (dict(w=_desc(qp, rows=4096, K=4096, matrices=2)), qp.QP_EINVAL, "offsets")]:
        _refused(qp, dx(**kw), code, needle)
    _refused(qp, L.qgemm_w4_mx_experts_dx(P, qp.QP_BF16, 4, 4096, B(w), None, P, 4096, P, 1 << 40,
                                          None), qp.QP_EINVAL, "offsets")
    _refused(qp, L.qgemm_w4_mx_dx_ws_size(4, B(w), None), qp.QP_EINVAL, "null")
    _refused(qp, L.qgemm_w4_mx_dx_ws_size(-1, B(w), B(n)), qp.QP_EINVAL, "negative")

    def q(X=P, dtype=qp.QP_F32, ldx=100, rule=0):
        return L.qquantize_rows_mx4(X, dtype, 4, 100, ldx, rule, P, 64, P, 4, None)

    for kw, code, needle in [
            (dict(rule=2), qp.QP_EINVAL, "rule"), (dict(X=None), qp.QP_EINVAL, "X is null"),
            (dict(dtype=qp.QP_S8), qp.QP_EINVAL, "X must be"), (dict(ldx=99), qp.QP_EINVAL, "stride"),
            (dict(X=P + 2), qp.QP_EALIGN, "X is not aligned")]:
        _refused(qp, q(**kw), code, needle)
    a = _desc(qp, matrices=2)
    _refused(qp, L.qdequantize_rows_mx4(B(a), P, qp.QP_F32, 100, None), qp.QP_EINVAL, "one matrix")
    a = _desc(qp)
    _refused(qp, L.qdequantize_rows_mx4(B(a), P, qp.QP_F32, 99, None), qp.QP_EINVAL, "stride of Y")
    _refused(qp, L.qdequantize_rows_mx4(B(a), P, qp.QP_S8, 100, None), qp.QP_EINVAL, "Y must be")


# ------------------------------------------------------------ the binding
class OnCard(torch.Tensor):
    """A host tensor that gives card 0 as its place."""

    def get_device(self):
        return 0


def _card(t):
    return t.as_subclass(OnCard)


@pytest.fixture
def no_launch(qp, monkeypatch):
    """The library's entry points replaced: a call that gets as far is noted."""
    reached = []

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_ws_size"):
                return getattr(real, name)
            return lambda *a: reached.append(name) or qp.QP_OK

    real = qp._lib
    monkeypatch.setattr(qp, "_lib", Lib())
    monkeypatch.setattr(qp, "_stream_of", lambda t: None)
    monkeypatch.setattr(qp, "_several_gpus", lambda: False)
    return reached


def _calls(qp):
    """Every operator with arguments that fit: {name: (function, its tensors, the rest)}."""
    b = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    f = lambda *s: torch.zeros(*s)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    w = dict(Wc=b(48, 64), Ws=b(48, 4))
    we = dict(Wc=b(3, 48, 64), Ws=b(3, 48, 4))
    m = lambda t, p: qp.MX4(t[p + "c"], t[p + "s"], 128)
    return {
        "quantize": (lambda t: qp.qquantize_rows_mx4(t["X"], out=m(t, "O")),
                     dict(X=f(5, 128), Oc=b(5, 64), Os=b(5, 4))),
        "dequantize": (lambda t: qp.qdequantize_rows_mx4(m(t, "A"), out=t["out"]),
                       dict(Ac=b(5, 64), As=b(5, 4), out=f(5, 128))),
        "a4w4": (lambda t: qp.qgemm_a4w4_mx(m(t, "A"), m(t, "W"), t["bias"], out=t["out"]),
                 dict(Ac=b(5, 64), As=b(5, 4), **w, bias=f(48), out=f(5, 48))),
        "a4w4_experts": (lambda t: qp.qgemm_a4w4_mx_experts(m(t, "A"), m(t, "W"), t["off"], t["bias"],
                                                            t["rows"], out=t["out"]),
                         dict(Ac=b(5, 64), As=b(5, 4), **we, off=i(4), bias=f(3, 48), rows=i(7),
                              out=f(7, 48))),
        "w4": (lambda t: qp.qgemm_w4_mx(t["X"], m(t, "W"), t["bias"], out=t["out"]),
               dict(X=f(5, 128), **w, bias=f(48), out=f(5, 48))),
        "w4_experts": (lambda t: qp.qgemm_w4_mx_experts(t["X"], m(t, "W"), t["off"], t["bias"],
                                                        t["rows"], out=t["out"]),
                       dict(X=f(5, 128), **we, off=i(4), bias=f(3, 48), rows=i(7), out=f(7, 48))),
        "dx": (lambda t: qp.qgemm_w4_mx_dx(t["dY"], m(t, "W"), out=t["out"], ws=t["ws"]),
               dict(dY=f(5, 48), **w, out=f(5, 128), ws=b(1 << 20))),
        "experts_dx": (lambda t: qp.qgemm_w4_mx_experts_dx(t["dY"], m(t, "W"), t["off"], out=t["out"],
                                                           ws=t["ws"]),
                       dict(dY=f(5, 48), **we, off=i(4), out=f(5, 128), ws=b(1 << 20))),
    }


@pytest.mark.parametrize("name", ["quantize", "dequantize", "a4w4", "a4w4_experts", "w4",
                                  "w4_experts", "dx", "experts_dx"])
def test_every_tensor_must_be_on_the_gpu(qp, no_launch, name):
    call, tensors = _calls(qp)[name]
    card = {n: _card(t) for n, t in tensors.items()}
    call(card)
    assert len(no_launch) == 1
    for n in tensors:
        with pytest.raises(AssertionError, match="on (the|one) GPU"):
            call({**card, n: tensors[n]})
    assert len(no_launch) == 1


def test_shapes_and_types_that_the_binding_refuses(qp, no_launch):
    for name, change, needle in [
            ("quantize", dict(X=torch.zeros(5, 96)), "X's shape"),
            ("quantize", dict(X=torch.zeros(5, 128, dtype=torch.float64)), "rows must be"),
            ("dequantize", dict(out=torch.zeros(5, 127)), "shape"),
            ("a4w4", dict(out=torch.zeros(5, 47)), "shape"),
            ("a4w4", dict(bias=torch.zeros(47)), "bias"),
            ("a4w4", dict(bias=torch.zeros(48, dtype=torch.float64)), "float32"),
            ("a4w4", dict(Wc=torch.zeros(3, 48, 64, dtype=torch.uint8),
                          Ws=torch.zeros(3, 48, 4, dtype=torch.uint8)), "one matrix"),
            ("a4w4_experts", dict(off=torch.zeros(3, dtype=torch.int32)), "experts \\+ 1"),
            ("a4w4_experts", dict(off=torch.zeros(4, dtype=torch.int64)), "int32"),
            ("a4w4_experts", dict(rows=torch.zeros(7, dtype=torch.int64)), "int32"),
            ("a4w4_experts", dict(bias=torch.zeros(48)), "experts x N"),
            ("w4", dict(X=torch.zeros(128, 5).t()), "unit column stride"),
            ("w4_experts", dict(Wc=torch.zeros(48, 64, dtype=torch.uint8),
                                Ws=torch.zeros(48, 4, dtype=torch.uint8)), "matrix an expert"),
            ("w4_experts", dict(out=torch.zeros(5, 48)), "shape"),
            ("dx", dict(dY=torch.zeros(5, 47)), "N columns"),
            ("dx", dict(out=torch.zeros(5, 128, dtype=torch.float16)), "dY's type"),
            ("experts_dx", dict(off=torch.zeros(5, dtype=torch.int32)), "experts \\+ 1")]:
        call, tensors = _calls(qp)[name]
        with pytest.raises(AssertionError, match=needle):
            call({n: _card(t) for n, t in {**tensors, **change}.items()})
    assert not no_launch
    with pytest.raises(AssertionError, match="rule"):
        qp.qquantize_rows_mx4(_card(torch.zeros(2, 32)), rule="even")
    with pytest.raises(AssertionError, match="MX4"):
        qp.qgemm_w4_mx(_card(torch.zeros(2, 32)), torch.zeros(2, 16, dtype=torch.uint8))


def test_checkpoint_layouts_that_do_not_fit(qp):
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    for c, s, K, needle in [(u(4, 32), u(4, 3), None, "16 bytes a block"),
                            (u(4, 32), u(5, 2), None, "alike"), (u(32), u(2), None, "alike"),
                            (u(4, 32), u(4, 2), 32, "does not fit"),
                            (u(4, 32), u(4, 2), 65, "does not fit"), (u(4, 0), u(4, 0), None, "block"),
                            (u(4, 32).int(), u(4, 2), None, "uint8")]:
        with pytest.raises(AssertionError, match=needle):
            qp.mx4_tensor(c, s, K)
    m = qp.mx4_tensor(u(4, 48), u(4, 3), 70)
    assert m.shape == (4, 70) and m.desc.ld_scales == 4 and m.desc.ld_codes == 48
    row = qp.mx4_tensor(u(1, 48)[:, :], u(1, 3))
    assert row.desc.ld_codes == 48 and row.desc.ld_scales == 4
    with pytest.raises(AssertionError, match="one matrix"):
        m[0]
