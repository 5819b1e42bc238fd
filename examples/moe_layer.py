#!/usr/bin/env python3
"""An MoE layer on 4-bit experts, as training and serving use it.

* ``train_step``: forward and backward through a layer whose experts are frozen (only what
  lies around them learns: the router, and the layers below through dx).  Activations cross
  the experts in FP8; the SwiGLU's input is kept as an 8-bit checkpoint.
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
from synth import quantize_weights  # noqa: E402


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
        """gate_up [E, 2F, D], down [E, D, F], float32."""
        return Experts(quantize_weights(gate_up), quantize_weights(down),
                       quantize_weights(gate_up.transpose(1, 2).contiguous()),
                       quantize_weights(down.transpose(1, 2).contiguous()))


def forward(x, logits, top_k, experts, keep=True):
    """x [M, D] BF16, logits [M, E] float32 -> out [M, D] BF16 and what the backward needs."""
    E = logits.shape[1]
    ids, weights = hg.hg_router_topk(logits, top_k)
    offsets, _, place = hg.hg_plan_expert_offsets(ids, E)
    a, a_scale = hg.hg_quantize_scatter_acts(x, top_k, place)
    z = hg.hg_grouped_w4a8_gemm(a, a_scale, *experts.gate_up, offsets)
    h, h_scale, z8, z8_scale = hg.hg_swiglu_quantize(z, checkpoint=keep)
    y = hg.hg_grouped_w4a8_gemm(h, h_scale, *experts.down, offsets)
    out = hg.hg_combine_topk(y, place, weights)
    return out, (logits, ids, weights, offsets, place, z8, z8_scale, y) if keep else None


def backward(dout, ctx, top_k, experts):
    """(dx [M, D] BF16, dlogits [M, E] float32) of dout [M, D] BF16."""
    logits, ids, weights, offsets, place, z8, z8_scale, y = ctx
    rows = torch.arange(y.shape[0], dtype=torch.int32, device=y.device)
    dy, dweights = hg.hg_combine_topk_bwd(dout, y, place, weights)
    q, s = hg.hg_quantize_scatter_acts(dy, 1, rows)
    dh = hg.hg_grouped_w4a8_gemm(q, s, *experts.down_t, offsets)
    dz = hg.hg_swiglu_bwd(dh, z8, z8_scale)
    q, s = hg.hg_quantize_scatter_acts(dz, 1, rows)
    dxs = hg.hg_grouped_w4a8_gemm(q, s, *experts.gate_up_t, offsets)
    dx, _ = hg.hg_dispatch_tokens_bwd(dxs, top_k, place)
    dlogits = hg.hg_router_topk_bwd(logits, ids, weights, dweights)
    return dx, dlogits


def train_step(x, logits, dout, top_k, experts):
    out, ctx = forward(x, logits, top_k, experts)
    return (out, *backward(dout, ctx, top_k, experts))


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

    experts = Experts.from_float(normal(E, 2 * F, D) / D ** 0.5, normal(E, D, F) / F ** 0.5)
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
    status, detail = hg.hg_get_device_status()
    if status != hg.HG_OK:
        raise SystemExit(f"device status {status} detail {detail}")


if __name__ == "__main__":
    main()
