"""What is measured of microscaled 4-bit floating point (MXFP4): the cases, their
inputs, the operators in plain form and through the library, and the same
results in 64 bits.

An MXFP4 matrix holds e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives) in blocks of 32 along its rows, each block times a power of two
2^(scale - 127) (scale 255: the block is NaN).  Two values a byte, the first in
the low bits.  K need not be a multiple of 32; the values that fill the last
block are zeros.

  quantize  rows to MXFP4 and the values read back (what training with
            quantized rows, or a check of a checkpoint, does).  A block's
            exponent is that of its largest magnitude less 2 ("floor": values
            above 6 become 6), or the least one that lets no value pass 6
            ("ceil").  Values round to the nearest, ties to the even code.
            Outputs: the values, the scales.
  a4w4      y[r] = a[r] W_e^T + bias, both MXFP4, for the rows r of expert e
            (one expert: the ordinary product).
  w4        the same with rows in floating point, not quantized.
  w4_dx     its gradient to the rows: dx[r] = dy[r] W_e.

With experts, rows are sorted by expert (offsets: the experts' first rows); T
tokens choose k experts each, and "map" reads the rows through slot_of_row / k
instead of from sorted copies.
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _quantize(dtype, M, K, rule="floor", **kw):
    return dict(op="quantize", dtype=dtype, M=M, K=K, rule=rule, **kw)


def _product(op, dtype, T, N, K, E=1, k=1, map=False, bias=False, **kw):
    return dict(op=op, dtype=dtype, T=T, N=N, K=K, E=E, k=k, map=map, bias=bias, **kw)


def listed():
    return [
        # the rows of one decoding step of 16 sequences
        _quantize("bf16", 16, 4096, name="quantize_step"),
        # a long prompt's rows, and an odd row length in f32 without clipping
        _quantize("bf16", 8192, 4096, name="quantize_prompt"),
        _quantize("f32", 1037, 1100, rule="ceil", name="quantize_odd"),
        # one token with quantized rows: an ordinary layer
        _product("a4w4", "bf16", 1, 4096, 4096, bias=True, name="a4w4_token"),
        # a large square product, as training with quantized operands runs it
        _product("a4w4", "bf16", 8192, 8192, 8192, name="a4w4_square"),
        # a prompt over 8 experts: the tokens are quantized once and read through the map
        _product("a4w4", "f16", 4096, 11008, 4096, E=8, k=2, map=True, name="a4w4_experts_prompt"),
        # one token over weights alone
        _product("w4", "bf16", 1, 11008, 4096, name="w4_token"),
        # odd sizes in f32, the last block cut short
        _product("w4", "f32", 131, 1037, 1100, bias=True, name="w4_odd"),
        # decoding 64 sequences over 16 experts
        _product("w4", "f16", 64, 11008, 4096, E=16, k=2, map=True, name="w4_experts_step"),
        # a prompt over 8 experts, sorted rows
        _product("w4", "bf16", 4096, 11008, 4096, E=8, k=2, name="w4_experts_prompt"),
        # training adapters under frozen experts
        _product("w4_dx", "bf16", 2048, 4096, 4096, E=8, k=2, name="w4_dx_experts"),
        # a few odd rows
        _product("w4_dx", "f16", 37, 1037, 1100, name="w4_dx_odd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "a4w4", "a4w4", "w4", "w4", "w4_dx"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op == "quantize":
        K = _log(rng, 32, 16384)
        if rng.random() < 0.7:
            K = (K + 31) // 32 * 32
        M = max(1, min(_log(rng, 1, 32768), (1 << 26) // K))
        return _quantize(dtype, M, K, rule=rng.choice(["floor", "ceil"]))
    N, K = _log(rng, 64, 11008), _log(rng, 64, 11008)
    if rng.random() < 0.7:
        N, K = (N + 31) // 32 * 32, (K + 31) // 32 * 32
    E = 1 if rng.random() < 0.5 else _log(rng, 2, 16)
    k = 1 if E == 1 else rng.randint(1, min(4, E))
    most = {"a4w4": 8192 ** 3, "w4": 8192 * 11008 * 4096 // 4, "w4_dx": 4096 ** 3}[op]
    T = max(1, min(_log(rng, 1, 8192), most // (k * N * K)))
    return _product(op, dtype, T, N, K, E=E, k=k, bias=op != "w4_dx" and rng.random() < 0.5,
                    map=op != "w4_dx" and E > 1 and rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(g, M, K):
    """Rows as a layer meets them: some columns a good deal larger than others, a
    spread between rows."""
    col = torch.exp(0.5 * _randn(g, 1, K))
    return _randn(g, M, K) * col * torch.exp(0.5 * _randn(g, M, 1))


def _blocks(x):
    M, K = x.shape
    G = (K + 31) // 32
    if K % 32:
        x = torch.nn.functional.pad(x, (0, G * 32 - K))
    return x.view(M, G, 32)


def _scaled(v, e):
    """v 2^e for whole e: two factors, as 2^e alone may lie outside f32."""
    h = torch.div(e, 2, rounding_mode="floor")
    two = [((n + 127) << 23).to(torch.int32).view(torch.float32) for n in (h, e - h)]
    return v * two[0] * two[1]


def _encode(x, rule):
    """Codes (one a byte) [M, 32 G] and scales [M, G] of f32 rows, in plain torch."""
    b = _blocks(x)
    big = b.abs().amax(dim=2)
    m, p = torch.frexp(big)
    e = p - 3
    if rule == "ceil":
        e = e + (m > 0.75).to(e.dtype)
    e = torch.where(big == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    a = _scaled(b.abs(), -e[:, :, None])
    small = torch.round(a * 2)                       # steps of 0.5 up to 2: codes 0 .. 4
    middle = torch.round(a) + 2                      # steps of 1 from 2 to 4: codes 4 .. 6
    large = torch.round(a * 0.5) + 4                 # steps of 2 from 4 on: codes 6, 7
    code = torch.where(a < 2, small, torch.where(a < 4, middle, large)).clamp(max=7)
    code = code.to(torch.uint8) + 8 * torch.signbit(b).to(torch.uint8)
    return code.view(x.shape[0], -1), (e + 127).to(torch.uint8)


def _packed(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()


def _decode(codes, scales):
    """The values of packed codes [M, 16 G] and scales [M, G], in f32."""
    grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float32, device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), dim=2).to(torch.int64)
    e = scales.to(torch.int32) - 127
    v = _scaled(grid[both].view(codes.shape[0], -1, 32), e[:, :, None])
    return v.view(codes.shape[0], -1)


def _route(g, T, k, E):
    """Rows of a router whose experts differ in popularity, sorted by expert:
    offsets and the slot of every row."""
    score = _randn(g, T, E) + 0.5 * _randn(g, E)
    ids = torch.topk(score, k, dim=1).indices.reshape(-1)
    key, order = torch.sort(ids, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device="cuda"))
    return offsets.to(torch.int32), order.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPE[case["dtype"]]
    st = {"case": case}
    if case["op"] == "quantize":
        st["x"] = _rows(g, case["M"], case["K"]).to(dt)
        return st
    T, N, K, E, k = (case[n] for n in ("T", "N", "K", "E", "k"))
    G = (K + 31) // 32
    codes = torch.empty((E, N, 16 * G), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, N, G), dtype=torch.uint8, device="cuda")
    for e in range(E):
        w = _randn(g, N, K) * torch.exp(0.5 * _randn(g, N, 1)) / math.sqrt(K)
        c, s = _encode(w, "floor")
        codes[e], scales[e] = _packed(c), s
    st["bias"] = _randn(g, E, N) if case["bias"] else None
    if E > 1:
        st["offsets"], st["slot_of_row"] = _route(g, T, k, E)
    rows = T if case["map"] else T * k
    x = _randn(g, rows, N).to(dt) if case["op"] == "w4_dx" else _rows(g, rows, K)
    if case["op"] == "a4w4":
        c, s = _encode(x, "floor")
        st["a"] = (_packed(c), s)
    else:
        st["x"] = x.to(dt)
    if own:
        import conv_qpack_weights_amd as qp
        st["w"] = qp.mx4_tensor(codes, scales, K) if E > 1 else qp.mx4_tensor(codes[0], scales[0], K)
        if case["op"] == "a4w4":
            st["a"] = qp.mx4_tensor(*st["a"], K)
    else:
        st["w"] = (codes, scales)
        st["counts"] = [T * k] if E == 1 else torch.diff(st["offsets"]).tolist()
    return st


# -------------------------------------------------------------- one pass
def _run_own(st, case):
    import conv_qpack_weights_amd as qp
    op, dt = case["op"], DTYPE[case["dtype"]]
    if op == "quantize":
        q = qp.qquantize_rows_mx4(st["x"], rule=case["rule"])
        return [qp.qdequantize_rows_mx4(q, dtype=dt), q.scales]
    if op == "w4_dx":
        if case["E"] == 1:
            return [qp.qgemm_w4_mx_dx(st["x"], st["w"])]
        return [qp.qgemm_w4_mx_experts_dx(st["x"], st["w"], st["offsets"])]
    through = dict(rows=st["slot_of_row"], row_div=case["k"]) if case["map"] else {}
    if op == "a4w4":
        if case["E"] == 1:
            bias = None if st["bias"] is None else st["bias"][0]
            return [qp.qgemm_a4w4_mx(st["a"], st["w"], bias, out_dtype=dt)]
        return [qp.qgemm_a4w4_mx_experts(st["a"], st["w"], st["offsets"], st["bias"], out_dtype=dt,
                                         **through)]
    if case["E"] == 1:
        bias = None if st["bias"] is None else st["bias"][0]
        return [qp.qgemm_w4_mx(st["x"], st["w"], bias)]
    return [qp.qgemm_w4_mx_experts(st["x"], st["w"], st["offsets"], st["bias"], **through)]


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    op, dt = case["op"], DTYPE[case["dtype"]]
    if op == "quantize":
        code, scales = _encode(state["x"].float(), case["rule"])
        return [_decode(_packed(code), scales)[:, :case["K"]].to(dt), scales]
    K = case["K"]
    x = _decode(*state["a"])[:, :K] if op == "a4w4" else state["x"].float()
    if case["map"]:
        x = x[torch.div(state["slot_of_row"].long(), case["k"], rounding_mode="floor")]
    out, at = [], 0
    for e, c in enumerate(state["counts"]):
        if c == 0:
            continue
        w = _decode(state["w"][0][e], state["w"][1][e])[:, :K]
        rows = x[at:at + c]
        at += c
        y = rows @ w if op == "w4_dx" else rows @ w.t()
        if state["bias"] is not None:
            y = y + state["bias"][e]
        out.append(y.to(dt))
    return [torch.cat(out)]


# ------------------------------------------------------------------- work
def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "quantize":
        M, K = case["M"], case["K"]
        G = (K + 31) // 32
        return {"bytes": 2 * M * K * es + 17 * M * G, "flops": 4 * M * K}
    T, N, K, E, k = (case[n] for n in ("T", "N", "K", "E", "k"))
    S, row = T * k, 17 * ((K + 31) // 32)
    # experts that some row is sent to, were all equally popular
    active = E * (1 - (1 - k / E) ** T) if E > 1 else 1
    b = active * N * row
    rows_in = T if case["map"] else S
    if case["op"] == "a4w4":
        b += rows_in * row + S * N * es
    elif case["op"] == "w4":
        b += (rows_in * K + S * N) * es
    else:
        b += S * (N + K) * es
    if case["bias"]:
        b += 4 * active * N
    return {"bytes": int(b), "flops": 2 * S * N * K}


# ---------------------------------------------------- from the definitions
def _two64(e):
    """2^e in 64 bits, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _value64(codes, scales, K):
    """What codes and scales stand for, bit by bit, in 64 bits: sign, two
    exponent bits, one bit of mantissa."""
    G = scales.shape[1]
    v = torch.empty((codes.shape[0], 32 * G), dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = (codes >> (4 * half)).to(torch.int64) & 15
        exp, man = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(exp == 0, man / 2, (1 + man / 2) * _two64(exp - 1))
        v[:, half::2] = torch.where(c >= 8, -mag, mag)
    two = _two64(scales.long() - 127).repeat_interleave(32, dim=1)
    return (v * two)[:, :K]


def _quantize64(x, rule):
    """The nearest grid point of every value, by comparing it with the points
    half way; a value on one goes to the even code."""
    K = x.shape[1]
    b = _blocks(x.double())
    big = b.abs().amax(dim=2)
    e = torch.where(big > 0, torch.floor(torch.log2(big.clamp_min(1e-300))) - 2, -127.0)
    if rule == "ceil":
        e = torch.where(big > 6 * _two64(e), e + 1, e)
    e = e.clamp(-127, 127)
    a = b.abs() / _two64(e)[:, :, None]
    code = torch.zeros_like(a, dtype=torch.int64)
    for lower in range(7):
        half = (GRID[lower] + GRID[lower + 1]) / 2
        code += ((a > half) | ((a == half) & (lower % 2 == 1))).long()
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    v = torch.copysign(grid[code], b) * _two64(e)[:, :, None]
    return v.view(x.shape[0], -1)[:, :K], (e + 127).to(torch.uint8)


def exact(case, seed):
    """The outputs of `run` from the definitions, in 64 bits."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "quantize":
        return list(_quantize64(st["x"], case["rule"]))
    op, K, N, E = case["op"], case["K"], case["N"], case["E"]
    S = case["T"] * case["k"]
    x = _value64(*st["a"], K) if op == "a4w4" else st["x"].double()
    first = [0, S] if E == 1 else st["offsets"].tolist()
    y = torch.zeros(S, K if op == "w4_dx" else N, dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = first[e], first[e + 1]
        if a == b:
            continue
        rows = torch.arange(a, b, device="cuda")
        if case["map"]:
            rows = st["slot_of_row"][a:b].long() // case["k"]
        W = _value64(st["w"][0][e], st["w"][1][e], K)
        y[a:b] = torch.mm(x[rows], W if op == "w4_dx" else W.t().contiguous())
        if st["bias"] is not None:
            y[a:b] += st["bias"][e].double()
    return [y]
