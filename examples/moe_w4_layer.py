"""A layer of experts with packed 4-bit weights, served and trained around.

Every token goes to top_k of the experts; an expert is a gated MLP whose
weights are int4 blobs (packed once), the rows stay in bf16:

    serving   qmoe_sort -> qgemm_w4_experts through the row map (no sorted copy)
              -> silu(gate) * up -> qgemm_w4_experts -> qmoe_combine
    training  qmoe_dispatch, the same products, qmoe_combine, and their gradients
              to the tokens and to the router's weights; the 4-bit weights are
              frozen (adapters or the router learn); first derivatives only

MxExpertLayer is the same layer with MXFP4 weights, as a checkpoint holds them; it
can also serve with MXFP4 rows: the tokens are quantized once, before their copies
to the experts, and the gated rows once more between the products.

Run it on an MI355X:  python examples/moe_w4_layer.py
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import conv_qpack_weights_amd as qp  # noqa: E402


def quantize_int4(w, group=32):
    """Symmetric int4 values (one per int8 byte) and f32 scales of w [E, N, K]."""
    E, N, K = w.shape
    G = -(-K // group)
    padded = torch.nn.functional.pad(w.float(), (0, G * group - K)).view(E, N, G, group)
    scale = padded.abs().amax(dim=3).clamp_min(1e-8) / 7
    q = torch.clamp(torch.round(padded / scale[..., None]), -8, 7).to(torch.int8)
    return q.view(E, N, G * group)[:, :, :K].contiguous(), scale


class _Once(torch.autograd.Function):
    """A first derivative: still tied to what it depends on, so that to
    differentiate it again is an error and not a result without its terms."""

    @staticmethod
    def forward(ctx, compute, *tensors):
        return compute(*tensors)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("cannot differentiate twice through the expert layer")


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, ids, experts):
        xs, offsets, row_of_slot, slot_of_row = qp.qmoe_dispatch(x, ids, experts)
        ctx.save_for_backward(row_of_slot)
        ctx.mark_non_differentiable(offsets, row_of_slot, slot_of_row)
        return xs, offsets, row_of_slot, slot_of_row

    @staticmethod
    def backward(ctx, dxs, *_):
        row_of_slot, = ctx.saved_tensors
        dx = _Once.apply(lambda d: qp.qmoe_dispatch_grad(d.contiguous(), row_of_slot), dxs)
        return dx, None, None


class _Experts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, blobs, info, offsets):
        ctx.save_for_backward(blobs, offsets)
        ctx.info = info
        return qp.qgemm_w4_experts(x, blobs, info, offsets)

    @staticmethod
    def backward(ctx, dy):
        blobs, offsets = ctx.saved_tensors
        dx = _Once.apply(
            lambda d: qp.qgemm_w4_experts_dx(d.contiguous(), blobs, ctx.info, offsets), dy)
        return dx, None, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, weights, row_of_slot, slot_of_row):
        ctx.save_for_backward(z, weights, row_of_slot, slot_of_row)
        return qp.qmoe_combine(z, row_of_slot, weights)

    @staticmethod
    def backward(ctx, dy):
        z, weights, row_of_slot, slot_of_row = ctx.saved_tensors
        dz, dw = _Once.apply(
            lambda d, z, w: qp.qmoe_combine_grad(d.contiguous(), z, row_of_slot, slot_of_row, w),
            dy, z, weights)
        return dz, dw, None, None


class ExpertLayer:
    """gate_up [E, 2F, H] and down [E, H, F] float weights, packed to int4."""

    def __init__(self, gate_up, down, group=32):
        self.experts = gate_up.shape[0]
        self.up = qp.pack_s4_experts(*quantize_int4(gate_up, group), group)
        self.down = qp.pack_s4_experts(*quantize_int4(down, group), group)

    @staticmethod
    def _gate(h):
        gate, up = h.chunk(2, dim=1)
        return torch.nn.functional.silu(gate) * up

    def _experts(self, x, which, offsets):
        return _Experts.apply(x, *which, offsets)

    def _matrices(self, which, dtype):
        blobs, info = which
        return [qp.qunpack_weights(b, info, values=False, scales=False, dequant=True)[3].to(dtype)
                for b in blobs]

    def serve(self, x, ids, weights):
        """x [T, H], ids int [T, top_k] (negative: no expert), weights f32 [T, top_k]."""
        offsets, row_of_slot, slot_of_row = qp.qmoe_sort(ids, self.experts)
        h = qp.qgemm_w4_experts(x, *self.up, offsets, rows=slot_of_row, row_div=ids.shape[1])
        z = qp.qgemm_w4_experts(self._gate(h), *self.down, offsets)
        return qp.qmoe_combine(z, row_of_slot, weights)

    def train(self, x, ids, weights):
        """The same with gradients to x and weights."""
        xs, offsets, row_of_slot, slot_of_row = _Dispatch.apply(x, ids, self.experts)
        h = self._experts(xs, self.up, offsets)
        z = self._experts(self._gate(h), self.down, offsets)
        return _Combine.apply(z, weights, row_of_slot, slot_of_row)

    def dense(self, x, ids, weights):
        """The layer from the formulas in x's type: a loop over tokens' choices."""
        mats = [self._matrices(which, x.dtype) for which in (self.up, self.down)]
        y = torch.zeros_like(x)
        for e in range(self.experts):
            for j in range(ids.shape[1]):
                t = torch.nonzero(ids[:, j] == e).squeeze(1)
                if t.numel():
                    z = self._gate(x[t] @ mats[0][e].t()) @ mats[1][e].t()
                    y = y.index_add(0, t, weights[t, j, None].to(x.dtype) * z)
        return y


class _MxExperts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(offsets)
        ctx.w = w
        return qp.qgemm_w4_mx_experts(x, w, offsets)

    @staticmethod
    def backward(ctx, dy):
        offsets, = ctx.saved_tensors
        dx = _Once.apply(lambda d: qp.qgemm_w4_mx_experts_dx(d.contiguous(), ctx.w, offsets), dy)
        return dx, None, None


class MxExpertLayer(ExpertLayer):
    """gate_up [E, 2F, H] and down [E, H, F]: MX4 matrices, or float weights that are
    quantized to them.  With ``rows4`` serve() quantizes the rows of both products."""

    def __init__(self, gate_up, down, rows4=False):
        self.up, self.down = (w if isinstance(w, qp.MX4) else qp.qquantize_rows_mx4(w, "ceil")
                              for w in (gate_up, down))
        self.experts = self.up.shape[0]
        self.rows4 = rows4

    def serve(self, x, ids, weights):
        offsets, row_of_slot, slot_of_row = qp.qmoe_sort(ids, self.experts)
        k = ids.shape[1]
        if self.rows4:
            h = qp.qgemm_a4w4_mx_experts(qp.qquantize_rows_mx4(x, "ceil"), self.up, offsets,
                                         rows=slot_of_row, row_div=k, out_dtype=x.dtype)
            z = qp.qgemm_a4w4_mx_experts(qp.qquantize_rows_mx4(self._gate(h), "ceil"), self.down,
                                         offsets, out_dtype=x.dtype)
        else:
            h = qp.qgemm_w4_mx_experts(x, self.up, offsets, rows=slot_of_row, row_div=k)
            z = qp.qgemm_w4_mx_experts(self._gate(h), self.down, offsets)
        return qp.qmoe_combine(z, row_of_slot, weights)

    def _experts(self, x, which, offsets):
        return _MxExperts.apply(x, which, offsets)

    def _matrices(self, which, dtype):
        return [qp.qdequantize_rows_mx4(which[e]).to(dtype) for e in range(self.experts)]


def make(experts=8, H=512, F=1408, seed=0, device="cuda", mx=False, rows4=False):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    up = torch.randn(experts, 2 * F, H, generator=g, device=device) / H ** 0.5
    down = torch.randn(experts, H, F, generator=g, device=device) / F ** 0.5
    return (MxExpertLayer(up, down, rows4) if mx else ExpertLayer(up, down)), g


def route(g, T, H, experts, top_k, device="cuda"):
    x = torch.randn(T, H, generator=g, device=device)
    logits = torch.randn(T, experts, generator=g, device=device)
    top, ids = torch.topk(logits, top_k, dim=1)
    return x, ids, torch.softmax(top, dim=1).contiguous()


def compare(T=64, experts=8, H=512, F=1408, top_k=2, dtype=torch.bfloat16, seed=0,
            mx=False):
    """Relative errors (norms) of the served output, the trained output and the
    gradients against the f64 formulas on the same 4-bit weights."""
    layer, g = make(experts, H, F, seed, mx=mx)
    x, ids, weights = route(g, T, H, experts, top_k)
    ids[0] = -1                                     # a padding token
    x = x.to(dtype)
    dy = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    x64 = x.double().requires_grad_()
    w64 = weights.double().requires_grad_()
    y64 = layer.dense(x64, ids, w64)
    y64.backward(dy.double())
    xt = x.clone().requires_grad_()
    wt = weights.clone().requires_grad_()
    yt = layer.train(xt, ids, wt)
    yt.backward(dy)
    rel = lambda a, b: float((a.detach().double() - b.detach()).norm() / b.detach().norm())
    return {"served": rel(layer.serve(x, ids, weights), y64), "trained": rel(yt, y64),
            "dx": rel(xt.grad, x64.grad), "dweights": rel(wt.grad, w64.grad)}


def main():
    for what, mx in (("int4", False), ("MXFP4", True)):
        for name, err in compare(mx=mx).items():
            print("%-5s %-10s relative error against the formulas in 64 bits: %.2e" %
                  (what, name, err))
    for what, kind in (("int4 weights", {}), ("MXFP4 weights", {"mx": True}),
                       ("MXFP4 weights and rows", {"mx": True, "rows4": True})):
        layer, g = make(experts=16, H=4096, F=11008 // 2, **kind)
        for T in (1, 16, 256):
            x, ids, weights = route(g, T, 4096, 16, 2)
            x = x.bfloat16()
            for _ in range(3):
                layer.serve(x, ids, weights)
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            for _ in range(20):
                layer.serve(x, ids, weights)
            end.record()
            end.synchronize()
            print("%-22s %4d tokens, 16 experts of 4096 x 5504, 2 a token: %.1f us a layer" %
                  (what, T, start.elapsed_time(end) / 20 * 1e3))


if __name__ == "__main__":
    main()
