"""What the binding of the float operators over int4 blobs and experts looks at
before anything reaches the library: where its tensors are and how large their
buffers.  No GPU needed: a tensor that says it is on card 0 stands for one that
is, and every call here is refused before its address is used."""
import pytest
import torch


class OnCard(torch.Tensor):
    """A host tensor that gives card 0 as its place."""

    def get_device(self):
        return 0


def _card(t):
    return t.as_subclass(OnCard)


@pytest.fixture(scope="module")
def qp():
    import conv_qpack_weights_amd as qp
    return qp


@pytest.fixture
def no_launch(qp, monkeypatch):
    """The library's entry points replaced: a call that gets as far is a failure."""
    reached = []

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_ws_size"):
                return getattr(real, name)
            return lambda *a: reached.append(name) or qp.QP_OK

    real = qp._lib
    monkeypatch.setattr(qp, "_lib", Lib())
    monkeypatch.setattr(qp, "_stream_of", lambda t: None)
    return reached


def _info(qp, N=48, K=64):
    """The description of f32-scaled int4 weights in groups of 32."""
    i = qp.PackedInfo()
    up = lambda a, b: -(-a // b) * b
    i.format, i.scheme, i.N, i.K, i.group = 2, qp.QP_BLOCKWISE, N, K, 32
    i.Npad, i.Kpad = up(N, 64), up(K, 128)
    i.data_off, i.data_bytes = 256, i.Npad * i.Kpad // 2
    i.scale_off = 256 + up(i.data_bytes, 256)
    i.sum_off = i.scale_off + up(16 * i.Npad * (-(-(i.Kpad // 32) // 4)), 256)
    i.total_bytes = i.sum_off + up(4 * i.Npad, 256)
    return i


def _calls(qp, i):
    """Every operator with arguments that fit: {name: (function, tensors by name)}."""
    ints = lambda *shape: torch.zeros(*shape, dtype=torch.int32)
    bytes_ = lambda *shape: torch.zeros(*shape, dtype=torch.uint8)
    n = i.total_bytes
    f = lambda *shape: torch.zeros(*shape)
    return {
        "qgemm_w4_blockwise": (
            lambda X, blob, bias, out: qp.qgemm_w4_blockwise(X, blob, i, bias, out=out),
            dict(X=f(4, 64), blob=bytes_(n), bias=f(48), out=f(4, 48))),
        "qgemm_w4_experts": (
            lambda X, blobs, offsets, bias, rows, out: qp.qgemm_w4_experts(
                X, blobs, i, offsets, bias, rows=rows, out=out),
            dict(X=f(4, 64), blobs=bytes_(2, n), offsets=ints(3), bias=f(2, 48), rows=ints(4),
                 out=f(4, 48))),
        "qgemm_w4_blockwise_dx": (
            lambda dY, blob, out, ws: qp.qgemm_w4_blockwise_dx(dY, blob, i, out=out, ws=ws),
            dict(dY=f(4, 48), blob=bytes_(n), out=f(4, 64), ws=bytes_(4096))),
        "qgemm_w4_experts_dx": (
            lambda dY, blobs, offsets, out, ws: qp.qgemm_w4_experts_dx(
                dY, blobs, i, offsets, out=out, ws=ws),
            dict(dY=f(4, 48), blobs=bytes_(2, n), offsets=ints(3), out=f(4, 64),
                 ws=bytes_(4096))),
        "qmoe_sort": (lambda ids, ws: qp.qmoe_sort(ids, 3, ws=ws),
                      dict(ids=ints(4, 2), ws=bytes_(256))),
        "qmoe_dispatch": (lambda X, ids, out, ws: qp.qmoe_dispatch(X, ids, 3, out=out, ws=ws),
                          dict(X=f(4, 64), ids=ints(4, 2), out=f(8, 64), ws=bytes_(256))),
        "qmoe_dispatch_grad": (
            lambda dXs, ros, out: qp.qmoe_dispatch_grad(dXs, ros, out=out),
            dict(dXs=f(8, 64), ros=ints(4, 2), out=f(4, 64))),
        "qmoe_combine": (
            lambda Z, ros, weights, out: qp.qmoe_combine(Z, ros, weights, out=out),
            dict(Z=f(8, 64), ros=ints(4, 2), weights=f(4, 2), out=f(4, 64))),
        "qmoe_combine_grad": (
            lambda dY, Z, ros, sor, weights, out, out_weights: qp.qmoe_combine_grad(
                dY, Z, ros, sor, weights, out=out, out_weights=out_weights),
            dict(dY=f(4, 64), Z=f(8, 64), ros=ints(4, 2), sor=ints(8), weights=f(4, 2),
                 out=f(8, 64), out_weights=f(4, 2))),
    }


NAMES = ["qgemm_w4_blockwise", "qgemm_w4_experts", "qgemm_w4_blockwise_dx", "qgemm_w4_experts_dx",
         "qmoe_sort", "qmoe_dispatch", "qmoe_dispatch_grad", "qmoe_combine", "qmoe_combine_grad"]


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_elsewhere_is_refused(qp, no_launch, name):
    call, tensors = _calls(qp, _info(qp))[name]
    on_card = {k: _card(t) for k, t in tensors.items()}
    call(**on_card)
    assert no_launch == [name]               # the arguments fit as they are
    for k in tensors:
        with pytest.raises(AssertionError, match="GPU"):
            call(**dict(on_card, **{k: tensors[k]}))
    with pytest.raises(AssertionError, match="on the GPU"):
        call(**tensors)                      # all of them on the host
    assert no_launch == [name]


@pytest.mark.parametrize("name", [n for n in NAMES if n.startswith("qgemm")])
def test_a_blob_shorter_than_its_description_is_refused(qp, no_launch, name):
    call, tensors = _calls(qp, _info(qp))[name]
    on_card = {k: _card(t) for k, t in tensors.items()}
    key = "blobs" if "experts" in name else "blob"
    blob = tensors[key]
    short = blob[..., :-1].contiguous()
    with pytest.raises(AssertionError, match="holds"):
        call(**dict(on_card, **{key: _card(short)}))
    if key == "blobs":                       # one expert's, too
        with pytest.raises(AssertionError, match="holds"):
            call(**dict(on_card, blobs=_card(short[:1]), offsets=on_card["offsets"][:2],
                        **({"bias": on_card["bias"][:1]} if "bias" in tensors else {})))
    else:
        apart = torch.zeros(2 * blob.numel(), dtype=torch.uint8)[::2]
        with pytest.raises(AssertionError, match="contiguous"):
            call(**dict(on_card, blob=_card(apart)))
        with pytest.raises(AssertionError, match="uint8"):
            call(**dict(on_card, blob=_card(torch.zeros(blob.numel()))))
    assert no_launch == []


@pytest.mark.parametrize("name", ["qgemm_w4_blockwise_dx", "qgemm_w4_experts_dx", "qmoe_sort",
                                  "qmoe_dispatch"])
def test_a_workspace_with_gaps_is_refused(qp, no_launch, name):
    call, tensors = _calls(qp, _info(qp))[name]
    on_card = {k: _card(t) for k, t in tensors.items()}
    gaps = torch.zeros(2 * tensors["ws"].numel(), dtype=torch.uint8)[::2]
    with pytest.raises(AssertionError, match="contiguous"):
        call(**dict(on_card, ws=_card(gaps)))
    assert no_launch == []


# ---------------------------------------------------------------- packing int4 weights
@pytest.fixture
def packed(qp, monkeypatch):
    """What pack_s4 hands to the packer: the values at the scales' address."""
    import ctypes as C
    import numpy as np
    seen = []

    def pack(w, desc, k_axis, n_axis, into=None):
        groups = -(-w.shape[1] // desc.group_size) * (2 if desc.scheme == qp.QP_BLOCKWISE_ASYM else 1)
        at = (C.c_float * (w.shape[0] * groups)).from_address(desc.scales)
        seen.append(np.array(at).reshape(w.shape[0], groups))
        return (torch.zeros(256, dtype=torch.uint8), None) if into is None else into

    monkeypatch.setattr(qp, "qpack_weights", pack)
    monkeypatch.setattr(qp, "_alloc_bytes", lambda n, device: torch.empty(n, dtype=torch.uint8))
    return seen


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16, torch.float64])
@pytest.mark.parametrize("layout", ["plain", "transposed", "every other"])
@pytest.mark.parametrize("kind", ["f32", "bf16", "asym"])
def test_scales_of_any_float_type_and_layout(qp, packed, dtype, layout, kind):
    """The packer reads f32 values one behind the other: bf16 scales, or a view
    with strides, have to be laid out that way first."""
    E, N, K, group = 3, 5, 100, 32
    G = 4
    g = torch.Generator().manual_seed(1)

    def make():
        v = (0.5 + torch.rand(E, N, G, generator=g)).to(torch.bfloat16).to(dtype)
        if layout == "transposed":
            t = v.transpose(1, 2).contiguous().transpose(1, 2)
        elif layout == "every other":
            t = torch.zeros(E, N, 2 * G, dtype=v.dtype)[:, :, ::2]
            t.copy_(v)
        else:
            t = v
        return t, v.double()

    scales, s = make()
    offsets, o = make() if kind == "asym" else (None, None)
    w = torch.zeros(E, N, K, dtype=torch.int8)
    card = lambda t: None if t is None else _card(t)
    qp.pack_s4(card(w[0]), card(scales[0]), group, "bf16" if kind == "bf16" else "f32",
               card(None if offsets is None else offsets[0]))
    qp.pack_s4_experts(card(w), card(scales), group, "bf16" if kind == "bf16" else "f32",
                       card(offsets))
    want = s if o is None else torch.stack((o, s), dim=-1).flatten(2)
    assert len(packed) == 1 + E
    for got, e in zip(packed, [0, *range(E)]):
        assert (torch.from_numpy(got).double() == want[e]).all()


def test_scales_that_do_not_fit_are_refused(qp, packed):
    w, s = _card(torch.zeros(2, 5, 100, dtype=torch.int8)), _card(torch.ones(2, 5, 4))
    for bad in (s[0, :, :3], s[0, :4], s[0].to(torch.int32)):
        with pytest.raises(AssertionError, match="scales"):
            qp.pack_s4(w[0], bad)
        with pytest.raises(AssertionError, match="offsets"):
            qp.pack_s4(w[0], s[0], offsets=bad)
    for bad in (s[:1], s[0], s[:, :, :3], s[:, :4]):
        with pytest.raises(AssertionError):
            qp.pack_s4_experts(w, bad)
        with pytest.raises(AssertionError):
            qp.pack_s4_experts(w, s, offsets=bad)
    with pytest.raises(AssertionError, match="byte"):
        qp.pack_s4(_card(torch.zeros(5, 100, dtype=torch.int32)), s[0])
    host = torch.ones(5, 4)
    with pytest.raises(AssertionError, match="GPU"):
        qp.pack_s4(w[0], host)
    with pytest.raises(AssertionError, match="GPU"):
        qp.pack_s4(w[0], s[0], offsets=host)
    with pytest.raises(AssertionError, match="GPU"):
        qp.pack_s4(torch.zeros(5, 100, dtype=torch.int8), s[0])
    assert packed == []


def test_sorts_of_up_to_8192_slots_need_no_workspace(qp):
    for T, k, E in ((1, 1, 1), (2048, 2, 8), (4096, 2, 512), (8192, 1, 512)):
        assert qp.qmoe_sort_ws_size(T, k, E) == 0
    assert qp.qmoe_sort_ws_size(4097, 2, 8) > 0
