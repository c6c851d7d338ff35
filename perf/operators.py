"""What is measured of the 4-bit expert layer: the cases, their inputs, the
operators in plain form and through the library, and the same results in 64
bits.

A layer of experts with packed 4-bit weights runs, for T tokens of which each
goes to top_k of E experts (a slot is one (token, choice) pair; slot
s = token*top_k + choice; a negative expert id is a dropped slot):

  dispatch   rows sorted by expert, stable in the slot order; each sorted row
             is a copy of its token's row (rows left over by dropped slots
             are zero).  Outputs: the sorted rows, the experts' first rows,
             the row of every slot (-1: dropped), the slot of every row.
             Its gradient sums a token's sorted-row gradients.
  combine    y[t] = sum_j weight[t,j] * z[row(t,j)] over the slots that are
             not dropped.  Its gradient: dz[row] = weight*dy[t] (zero for
             rows without a slot) and dweight[t,j] = <dy[t], z[row]> (zero
             for dropped slots).
  w4         y[r] = x[r] W_e^T + bias for the rows r of expert e, with
             W[n,k] = scale[n, k/group]*q[n,k] (+ offset[n, k/group]),
             q in [-8, 7].  One expert is the ordinary product.  "map": the
             rows are read through the slot of every row, slot/top_k being
             the row of x, instead of from sorted copies.
  w4_dx      its gradient to the rows: dx[r] = dy[r] W_e.
"""
import math

import numpy as np
import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def _moe(op, dtype, T, k, E, H, drop=False, ids="s32", **kw):
    return dict(op=op, dtype=dtype, T=T, k=k, E=E, H=H, drop=drop, ids=ids, **kw)


def _w4(op, dtype, T, N, K, group=32, scales="f32", E=1, k=1, map=False, bias=False, **kw):
    return dict(op=op, dtype=dtype, T=T, k=k, E=E, N=N, K=K, group=group, scales=scales, map=map,
                bias=bias, **kw)


def listed():
    return [
        # one decoding step of 16 sequences: latency of the sort and the copy
        dict(_moe("dispatch", "bf16", 16, 2, 8, 4096), name="dispatch_step"),
        # a long prompt (or a batch of prompts) over many small experts
        dict(_moe("dispatch", "bf16", 8192, 8, 128, 4096, ids="s64"), name="dispatch_prompt"),
        # training with padding tokens (dropped slots), an odd row length
        dict(_moe("dispatch_grad", "f32", 4099, 4, 32, 1101, drop=True), name="dispatch_grad_odd"),
        # the same prompt on its way back
        dict(_moe("combine", "f16", 8192, 8, 128, 4096), name="combine_prompt"),
        # training: both gradients of the weighted sum, padding tokens dropped
        dict(_moe("combine_grad", "bf16", 4096, 8, 64, 4096, drop=True), name="combine_grad_train"),
        # one sequence, one token: an ordinary layer's product
        dict(_w4("w4", "bf16", 1, 4096, 4096), name="w4_token"),
        # a decoding batch of 16, coarse groups, bias
        dict(_w4("w4", "f16", 16, 11008, 4096, group=128, bias=True), name="w4_batch16"),
        # odd sizes in f32, asymmetric weights, the last group cut short
        dict(_w4("w4", "f32", 131, 1037, 1100, group=64, scales="asym", bias=True), name="w4_odd"),
        # decoding 64 sequences over 16 experts, rows read through the map
        dict(_w4("w4", "bf16", 64, 11008, 4096, E=16, k=2, map=True), name="w4_experts_step"),
        # a prompt over 8 experts, sorted rows
        dict(_w4("w4", "bf16", 4096, 11008, 4096, E=8, k=2), name="w4_experts_prompt"),
        # training adapters under frozen 4-bit experts
        dict(_w4("w4_dx", "bf16", 2048, 4096, 4096, E=8, k=2), name="w4_dx_experts"),
        # a few odd rows, bf16 scales
        dict(_w4("w4_dx", "f16", 37, 1037, 1100, scales="bf16"), name="w4_dx_odd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "w4", "w4", "w4_dx"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op not in ("w4", "w4_dx"):
        E = _log(rng, 2, 256)
        k = rng.randint(1, min(8, E))
        H = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            H = (H + 63) // 64 * 64
        T = _log(rng, 1, 32768)
        T = max(1, min(T, 8192 * 8 * 4096 // 2 // (k * H)))
        return _moe(op, dtype, T, k, E, H, drop=rng.random() < 0.4, ids=rng.choice(["s32", "s64"]))
    group = rng.choice([32, 32, 64, 128, 256])
    scales = rng.choice(["f32", "f32", "bf16", "asym"])
    N, K = _log(rng, 64, 11008), _log(rng, 64, 11008)
    if rng.random() < 0.7:
        N, K = (N + 63) // 64 * 64, (K + 63) // 64 * 64
    E = 1 if rng.random() < 0.4 else _log(rng, 2, 16)
    k = 1 if E == 1 else rng.randint(1, min(4, E))
    T = _log(rng, 1, 4096)
    most = (8192 if op == "w4" else 4096) * 4096 * 4096 / (4 if dtype == "f32" else 1)
    T = max(1, min(T, int(most / (k * N * K))))
    return _w4(op, dtype, T, N, K, group=group, scales=scales, E=E, k=k,
               map=op == "w4" and E > 1 and rng.random() < 0.5,
               bias=op == "w4" and rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _route(g, T, k, E, drop):
    """Expert ids and weights of a router whose experts differ in popularity;
    with `drop`, one token in sixteen is padding and one choice in sixteen
    was cut off."""
    score = _randn(g, T, E) + 0.5 * _randn(g, E)
    top, ids = torch.topk(score, k, dim=1)
    weights = torch.softmax(top, dim=1).contiguous()
    if drop:
        pad = torch.rand(T, 1, generator=g, device="cuda") < 1 / 16
        cut = torch.rand(T, k, generator=g, device="cuda") < 1 / 16
        ids = torch.where(pad | cut, torch.full_like(ids, -1), ids)
    return ids, weights


def _plan(ids, E):
    """Offsets, row of every slot, slot of every row: a stable sort in plain
    torch operations."""
    flat = ids.reshape(-1).to(torch.int64)
    S = flat.numel()
    kept = flat >= 0
    key = torch.where(kept, flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    row = torch.empty_like(order)
    row[order] = torch.arange(S, device=flat.device)
    row_of_slot = torch.where(kept, row, torch.full_like(row, -1))
    bounds = torch.arange(E + 1, device=flat.device)
    offsets = (key[None, :] < bounds[:, None]).sum(dim=1) if S * E < 1 << 24 else \
        torch.searchsorted(key[order].contiguous(), bounds)
    slot_of_row = torch.where(torch.arange(S, device=flat.device) < offsets[E], order,
                              torch.full_like(order, -1))
    return (offsets.to(torch.int32), row_of_slot.to(torch.int32).reshape(ids.shape),
            slot_of_row.to(torch.int32))


def _groups(case):
    return (case["K"] + case["group"] - 1) // case["group"]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPE[case["dtype"]]
    st = {"case": case}
    T, k, E = case["T"], case["k"], case["E"]
    if case["op"] in ("w4", "w4_dx"):
        N, K, G = case["N"], case["K"], _groups(case)
        q = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
        for e in range(E):
            q[e] = torch.clamp(torch.round(2.6 * _randn(g, N, K)), -8, 7).to(torch.int8)
        s = (0.5 + torch.rand(E, N, G, generator=g, device="cuda")) * (0.4 / math.sqrt(K))
        off = None
        if case["scales"] == "asym":
            off = s * (torch.rand(E, N, G, generator=g, device="cuda") * 2 - 1)
        if case["scales"] == "bf16":
            s = s.to(torch.bfloat16).float()
        st["bias"] = _randn(g, E, N) if case["bias"] else None
        if E > 1:
            ids, _ = _route(g, T, k, E, False)
            st["offsets"], _, st["slot_of_row"] = _plan(ids, E)
        S = T * k
        width = K if case["op"] == "w4" else N
        st["x"] = _randn(g, T if case["map"] else S, width).to(dt)
        if own:
            import conv_qpack_weights_amd as qp
            kind = "bf16" if case["scales"] == "bf16" else "f32"
            if E == 1:
                st["blob"], st["info"] = qp.pack_s4(q[0], s[0], case["group"], kind,
                                                    None if off is None else off[0])
            else:
                st["blob"], st["info"] = qp.pack_s4_experts(q, s, case["group"], kind, off)
        else:
            st.update(q=q, s=s, off=off)
            st["counts"] = [S] if E == 1 else torch.diff(st["offsets"]).tolist()
        return st
    ids, weights = _route(g, T, k, E, case["drop"])
    ids = ids.to(torch.int32 if case["ids"] == "s32" else torch.int64)
    st.update(ids=ids, weights=weights)
    st["offsets"], st["row_of_slot"], st["slot_of_row"] = _plan(ids, E)
    H = case["H"]
    if case["op"] == "dispatch":
        st["x"] = _randn(g, T, H).to(dt)
    elif case["op"] == "dispatch_grad":
        st["dxs"] = _randn(g, T * k, H).to(dt)
    else:
        st["z"] = _randn(g, T * k, H).to(dt)
        if case["op"] == "combine_grad":
            st["dy"] = _randn(g, T, H).to(dt)
    return st


# -------------------------------------------------------------- one pass
def _run_own(st, case):
    import conv_qpack_weights_amd as qp
    op = case["op"]
    if op == "dispatch":
        return list(qp.qmoe_dispatch(st["x"], st["ids"], case["E"]))
    if op == "dispatch_grad":
        return [qp.qmoe_dispatch_grad(st["dxs"], st["row_of_slot"])]
    if op == "combine":
        return [qp.qmoe_combine(st["z"], st["row_of_slot"], st["weights"])]
    if op == "combine_grad":
        return list(qp.qmoe_combine_grad(st["dy"], st["z"], st["row_of_slot"], st["slot_of_row"],
                                         st["weights"]))
    if op == "w4":
        if case["E"] == 1:
            bias = None if st["bias"] is None else st["bias"][0]
            return [qp.qgemm_w4_blockwise(st["x"], st["blob"], st["info"], bias)]
        if case["map"]:
            return [qp.qgemm_w4_experts(st["x"], st["blob"], st["info"], st["offsets"], st["bias"],
                                        rows=st["slot_of_row"], row_div=case["k"])]
        return [qp.qgemm_w4_experts(st["x"], st["blob"], st["info"], st["offsets"], st["bias"])]
    if case["E"] == 1:
        return [qp.qgemm_w4_blockwise_dx(st["x"], st["blob"], st["info"])]
    return [qp.qgemm_w4_experts_dx(st["x"], st["blob"], st["info"], st["offsets"])]


def _weights32(st, case, e):
    """W of expert e in f32."""
    N, K, G, group = case["N"], case["K"], _groups(case), case["group"]
    w = st["q"][e].float()
    s = st["s"][e].repeat_interleave(group, dim=1)[:, :K]
    w = w * s
    if st["off"] is not None:
        w = w + st["off"][e].repeat_interleave(group, dim=1)[:, :K]
    return w


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    op, dt = case["op"], DTYPE[case["dtype"]]
    T, k, E = case["T"], case["k"], case["E"]
    if op in ("w4", "w4_dx"):
        x = state["x"]
        if case["map"]:
            x = x[torch.div(state["slot_of_row"].long(), k, rounding_mode="floor")]
        out, at = [], 0
        for e, c in enumerate(state["counts"]):
            if c == 0:
                continue
            w = _weights32(state, case, e)
            rows = x[at:at + c].float()
            at += c
            y = rows @ w.t() if op == "w4" else rows @ w
            if state["bias"] is not None:
                y = y + state["bias"][e]
            out.append(y.to(dt))
        return [torch.cat(out)]
    if op == "dispatch":
        offsets, row_of_slot, slot_of_row = _plan(state["ids"], E)
        kept = slot_of_row >= 0
        token = torch.div(slot_of_row.long().clamp(min=0), k, rounding_mode="floor")
        xs = torch.where(kept[:, None], state["x"][token], torch.zeros((), dtype=dt, device="cuda"))
        return [xs, offsets, row_of_slot, slot_of_row]
    ros = state["row_of_slot"].long()
    kept = ros >= 0
    if op == "dispatch_grad":
        acc = torch.zeros(T, case["H"], dtype=torch.float32, device="cuda")
        for j in range(k):
            acc += torch.where(kept[:, j, None], state["dxs"][ros[:, j].clamp(min=0)].float(), 0.0)
        return [acc.to(dt)]
    if op == "combine":
        acc = torch.zeros(T, case["H"], dtype=torch.float32, device="cuda")
        for j in range(k):
            row = state["z"][ros[:, j].clamp(min=0)].float()
            acc += torch.where(kept[:, j, None], row * state["weights"][:, j, None], 0.0)
        return [acc.to(dt)]
    dy = state["dy"].float()
    dz = torch.zeros(T * k, case["H"], dtype=dt, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float32, device="cuda")
    for j in range(k):
        row = ros[:, j].clamp(min=0)
        dw[:, j] = torch.where(kept[:, j], (dy * state["z"][row].float()).sum(dim=1), 0.0)
        mine = torch.nonzero(kept[:, j]).squeeze(1)
        dz[ros[mine, j]] = (dy[mine] * state["weights"][mine, j, None]).to(dt)
    return [dz, dw]


# ------------------------------------------------------------------- work
def work(case):
    es = BYTES[case["dtype"]]
    T, k, E = case["T"], case["k"], case["E"]
    S = T * k
    if case["op"] in ("w4", "w4_dx"):
        N, K = case["N"], case["K"]
        # experts that some row is sent to, were all equally popular
        active = E * (1 - (1 - k / E) ** T) if E > 1 else 1
        per_group = {"f32": 4, "bf16": 2, "asym": 8}[case["scales"]]
        w = active * (N * K / 2 + N * _groups(case) * per_group)
        rows_in = T if case["map"] else S
        b = w + (rows_in * K + S * N if case["op"] == "w4" else S * (N + K)) * es
        if case["bias"]:
            b += 4 * active * N
        return {"bytes": int(b), "flops": 2 * S * N * K}
    H = case["H"]
    idb = 4 if case["ids"] == "s32" else 8
    if case["op"] == "dispatch":
        return {"bytes": (T + S) * H * es + S * (idb + 8) + 4 * (E + 1), "flops": 0}
    if case["op"] == "dispatch_grad":
        return {"bytes": (T + S) * H * es + 4 * S, "flops": S * H}
    if case["op"] == "combine":
        return {"bytes": (T + S) * H * es + 8 * S, "flops": 2 * S * H}
    return {"bytes": (T + 2 * S) * H * es + 16 * S, "flops": 3 * S * H}


# ---------------------------------------------------- from the definitions
def _sorted_slots(ids):
    """Slots of every expert in slot order, by counting on the host."""
    flat = ids.reshape(-1).cpu().numpy().astype(np.int64)
    kept = np.flatnonzero(flat >= 0)
    return flat, kept[np.lexsort((kept, flat[kept]))]


def exact(case, seed):
    """The outputs of `run` from the definitions, in 64 bits."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, T, k, E = case["op"], case["T"], case["k"], case["E"]
    S = T * k
    if op in ("w4", "w4_dx"):
        N, K, group = case["N"], case["K"], case["group"]
        of_k = torch.arange(K, device="cuda") // group
        first = [0, S] if E == 1 else st["offsets"].tolist()
        src = torch.arange(S, device="cuda")
        if case["map"]:
            src = st["slot_of_row"].long() // k
        y = torch.zeros(S, N if op == "w4" else K, dtype=torch.float64, device="cuda")
        for e in range(E):
            a, b = first[e], first[e + 1]
            if a == b:
                continue
            W = st["s"][e].double()[:, of_k] * st["q"][e].double()
            if st["off"] is not None:
                W += st["off"][e].double()[:, of_k]
            rows = st["x"].double()[src[a:b]]
            y[a:b] = torch.mm(rows, W.t().contiguous() if op == "w4" else W)
            if st["bias"] is not None:
                y[a:b] += st["bias"][e].double()
        return [y]
    H = case["H"]
    if op == "dispatch":
        flat, order = _sorted_slots(st["ids"])
        slot_of_row = np.full(S, -1, np.int32)
        slot_of_row[:order.size] = order
        row_of_slot = np.full(S, -1, np.int32)
        row_of_slot[order] = np.arange(order.size)
        offsets = np.array([np.count_nonzero((flat >= 0) & (flat < e)) for e in range(E + 1)],
                           np.int32)
        xs = torch.zeros(S, H, dtype=torch.float64, device="cuda")
        xs[:order.size] = st["x"].double()[torch.from_numpy(order // k).cuda()]
        return [xs, torch.from_numpy(offsets).cuda(),
                torch.from_numpy(row_of_slot.reshape(T, k)).cuda(),
                torch.from_numpy(slot_of_row).cuda()]
    # a token's slots come from the rows' side here: one scatter over the rows
    sor = st["slot_of_row"].long()
    rows = torch.nonzero(sor >= 0).squeeze(1)
    slot = sor[rows]
    token = slot // k
    if op == "dispatch_grad":
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        return [y.index_add_(0, token, st["dxs"].double()[rows])]
    w = st["weights"].double().reshape(-1)
    if op == "combine":
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        return [y.index_add_(0, token, st["z"].double()[rows] * w[slot, None])]
    dy = st["dy"].double()
    dz = torch.zeros(S, H, dtype=torch.float64, device="cuda")
    dz[rows] = dy[token] * w[slot, None]
    dw = torch.zeros(S, dtype=torch.float64, device="cuda")
    dw[slot] = (dy[token] * st["z"].double()[rows]).sum(dim=1)
    return [dz, dw.reshape(T, k)]
