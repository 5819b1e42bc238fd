#!/usr/bin/env python3
"""An MoE layer on 4-bit experts, as training and serving use it.

* ``train_step``: forward and backward through a layer whose experts are frozen (only what
  lies around them learns: the router, and the layers below through dx).  Activations cross
  the experts in FP8; the SwiGLU's input is kept as an 8-bit checkpoint.
* ``train_block``: the layer behind its norm, with the residual stream, and the experts learn
  too: gradients of their weights from the FP8 activations that the forward pass kept, and
  ``Experts.quantize`` writes updated master weights over the 4-bit ones.
* ``decode``: the same layer for the few tokens of a decoding step, in four launches (the
  numbers of the slots, which never change, are made once by the caller).

    python examples/moe_layer.py
"""
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp8_mxfp4_grouped_gb300 import hg  # noqa: E402


def _quantize(w, *out):
    """Both orientations of float weights of any strides and type; BF16 as they are, others through
    float32."""
    w = w.cuda() if w.device.type == "cpu" else w
    w = w if w.dtype == torch.bfloat16 else w.float()
    return hg.hg_quantize_weights(w.contiguous(), True, *out)


@dataclass
class Experts:
    """MXFP4 weights [E, out, in/2] with E8M0 scales [E, out, in/32]: gate rows then up rows,
    the down projection, and both transposed (quantised along their own inputs) for the
    gradient of the activations."""
    gate_up: tuple
    down: tuple
    gate_up_t: tuple
    down_t: tuple

    @staticmethod
    def from_float(gate_up: torch.Tensor, down: torch.Tensor) -> "Experts":
        """gate_up [E, 2F, D], down [E, D, F]."""
        g, d = _quantize(gate_up), _quantize(down)
        return Experts(g[:2], d[:2], g[2:], d[2:])

    def quantize(self, gate_up: torch.Tensor, down: torch.Tensor):
        """The same weights after an update, over the ones that are there."""
        _quantize(gate_up, *self.gate_up, *self.gate_up_t)
        _quantize(down, *self.down, *self.down_t)


def forward(x, logits, top_k, experts, keep=True, acts=None, weight_grads=False):
    """x [M, D] BF16, logits [M, E] float32 -> out [M, D] BF16 and what the backward needs, with
    weight_grads the products' FP8 inputs too (M * top_k * (D + F) bytes).
    acts: x as FP8 codes with scales, where the norm before has made them."""
    E = logits.shape[1]
    ids, weights = hg.hg_router_topk(logits, top_k)
    offsets, _, place = hg.hg_plan_expert_offsets(ids, E)
    if acts is None:
        a, a_scale = hg.hg_quantize_scatter_acts(x, top_k, place)
    else:
        a, a_scale = hg.hg_dispatch_acts(*acts, top_k, place)
    z = hg.hg_grouped_w4a8_gemm(a, a_scale, *experts.gate_up, offsets)
    h, h_scale, z8, z8_scale = hg.hg_swiglu_quantize(z, checkpoint=keep)
    y = hg.hg_grouped_w4a8_gemm(h, h_scale, *experts.down, offsets)
    out = hg.hg_combine_topk(y, place, weights)
    if not keep:
        return out, None
    inputs = ((a, a_scale), (h, h_scale)) if weight_grads else None
    return out, (logits, ids, weights, offsets, place, z8, z8_scale, y, inputs)


def backward(dout, ctx, top_k, experts, weight_grads=False):
    """(dx [M, D] BF16, dlogits [M, E] float32) of dout [M, D] BF16, and with weight_grads the
    gradients of gate_up [E, 2F, D] and down [E, D, F] in float32."""
    logits, ids, weights, offsets, place, z8, z8_scale, y, inputs = ctx
    assert inputs or not weight_grads, "the forward pass has not kept the products' inputs"
    rows = torch.arange(y.shape[0], dtype=torch.int32, device=y.device)
    dy, dweights = hg.hg_combine_topk_bwd(dout, y, place, weights)
    q, s = hg.hg_quantize_scatter_acts(dy, 1, rows)
    dh = hg.hg_grouped_w4a8_gemm(q, s, *experts.down_t, offsets)
    dz = hg.hg_swiglu_bwd(dh, z8, z8_scale)
    q, s = hg.hg_quantize_scatter_acts(dz, 1, rows)
    dxs = hg.hg_grouped_w4a8_gemm(q, s, *experts.gate_up_t, offsets)
    dx, _ = hg.hg_dispatch_tokens_bwd(dxs, top_k, place)
    dlogits = hg.hg_router_topk_bwd(logits, ids, weights, dweights)
    if not weight_grads:
        return dx, dlogits
    acts, hidden = inputs
    return dx, dlogits, (hg.hg_grouped_wgrad_fp8(dz, *acts, offsets),
                         hg.hg_grouped_wgrad_fp8(dy, *hidden, offsets))


def train_step(x, logits, dout, top_k, experts):
    out, ctx = forward(x, logits, top_k, experts)
    return (out, *backward(dout, ctx, top_k, experts))


def train_block(x, residual, gain, router, dout, top_k, experts):
    """One training step of s = x + residual, y = s + layer(norm(s) * gain): x, residual and dout
    [M, D] BF16, gain [D] BF16, router [D, E] float32.  Returns y, the gradient of x (and of
    residual, which is the same), of gain, of router, and of the experts' weights."""
    n, a, a_scale, s, rstd = hg.hg_rmsnorm_quantize(x, gain, residual=residual)
    out, ctx = forward(n, n.float() @ router, top_k, experts, acts=(a, a_scale), weight_grads=True)
    dn, dlogits, dexperts = backward(dout, ctx, top_k, experts, weight_grads=True)
    drouter = n.float().T @ dlogits
    dn = (dn.float() + dlogits @ router.T).bfloat16()
    dx, dgain = hg.hg_rmsnorm_bwd(dn, s, gain, rstd, dsum=dout)
    return s + out, dx, dgain, drouter, dexperts


def slot_numbers(tokens, top_k, device="cuda"):
    """What hg_combine_topk reads where the rows are in slot order."""
    return torch.arange(tokens * top_k, dtype=torch.int32, device=device)


def decode(x, logits, top_k, experts, slots=None):
    """The layer for a few tokens: no plan, no sorting, BF16 activations throughout.  slots:
    slot_numbers(M, top_k), made here (a launch more) where they are not given."""
    if slots is None:
        slots = slot_numbers(x.shape[0], top_k, x.device)
    ids, weights = hg.hg_router_topk(logits, top_k)
    h = hg.hg_expert_matvec_swiglu(x, ids, *experts.gate_up)
    y = hg.hg_expert_matvec(h, ids, *experts.down)
    return hg.hg_combine_topk(y, slots, weights)


def main():
    D, F, E, top_k = 1024, 512, 16, 4
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    masters = [normal(E, 2 * F, D) / D ** 0.5, normal(E, D, F) / F ** 0.5]
    experts = Experts.from_float(*masters)
    router = normal(D, E) / D ** 0.5
    x, dout = normal(512, D).bfloat16(), normal(512, D).bfloat16()
    out, dx, dlogits = train_step(x, x.float() @ router, dout, top_k, experts)
    drouter = x.float().T @ dlogits
    print("train: out", tuple(out.shape), "dx", tuple(dx.shape), "router gradient norm",
          round(float(drouter.norm()), 4))
    few = decode(x[:3].contiguous(), x[:3].float() @ router, top_k, experts,
                 slot_numbers(3, top_k))
    off = float((few.float() - out[:3].float()).norm() / out[:3].float().norm())
    print("decode: out", tuple(few.shape), "relative difference from the FP8 path", round(off, 4))
    gain = (1 + 0.1 * normal(D)).bfloat16()
    y, _, dgain, _, dexperts = train_block(x, (3 * normal(512, D)).bfloat16(), gain, router, dout,
                                           top_k, experts)
    for w, dw in zip(masters, dexperts):
        w.sub_(1e-3 * dw)
    experts.quantize(*masters)
    print("block: y", tuple(y.shape), "gain gradient norm", round(float(dgain.norm()), 4),
          "expert gradient norms", *(round(float(g.norm()), 2) for g in dexperts))
    status, detail = hg.hg_get_device_status()
    if status != hg.HG_OK:
        raise SystemExit(f"device status {status} detail {detail}")


if __name__ == "__main__":
    main()
