"""The MoE layer of examples/moe_layer.py, forward, backward and decoding, against the float64
chain on the same weights.

Tolerance: an E4M3 rounding is off by up to 2^-4 of a value, about 2.6 % in the 2-norm, and a
result passes through at most six (x, h, the checkpoint, dy, dz, and the router's own inputs
through y): sqrt(6) * 2.6 % is 6.4 %; 10 % are allowed.  Decoding rounds to BF16 only: 2 %.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import moe_layer as L
from oracle.formats import E8M0_TABLE, bf16_bits_to_f64, decode_e2m1_packed

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "moe_layer_example", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _f64(t):
    return bf16_bits_to_f64(t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))


def _weights(pair):
    w, s = pair[0].cpu().numpy(), pair[1].cpu().numpy()
    return decode_e2m1_packed(w) * np.repeat(E8M0_TABLE[s], 32, axis=-1)


def _off(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def test_moe_layer_trains_and_decodes(cuda_lib):
    ex = _example()
    D, F, E, k, M = 256, 128, 8, 2, 40
    g = torch.Generator().manual_seed(5)
    experts = ex.Experts.from_float((torch.randn(E, 2 * F, D, generator=g) / D ** 0.5).cuda(),
                                    (torch.randn(E, D, F, generator=g) / F ** 0.5).cuda())
    x = torch.randn(M, D, generator=g).bfloat16()
    logits = torch.randn(M, E, generator=g)
    dout = torch.randn(M, D, generator=g).bfloat16()
    out, dx, dlogits = ex.train_step(x.cuda(), logits.cuda(), dout.cuda(), k, experts)
    few = ex.decode(x[:3].cuda(), logits[:3].cuda(), k, experts)

    xf, df, lf = _f64(x), _f64(dout), logits.double().numpy()
    ids, w = L.router_topk(lf, k, True)
    gu, dn = _weights(experts.gate_up), _weights(experts.down)
    gu_t, dn_t = _weights(experts.gate_up_t), _weights(experts.down_t)
    want_out, want_dx = np.zeros((M, D)), np.zeros((M, D))
    dw = np.zeros((M, k))
    for t in range(M):
        for j in range(k):
            e = ids[t, j]
            z = (gu[e] @ xf[t])[None]
            y = dn[e] @ L.swiglu(z)[0]
            want_out[t] += w[t, j] * y
            dw[t, j] = df[t] @ y
            dh = dn_t[e] @ (w[t, j] * df[t])
            want_dx[t] += gu_t[e] @ L.swiglu_bwd(dh[None], z)[0]
    assert _off(_f64(out), want_out) < 0.1
    assert _off(_f64(dx), want_dx) < 0.1
    assert _off(dlogits.double().cpu().numpy(), L.router_topk_bwd(lf, ids, dw, True)) < 0.1
    assert _off(_f64(few), want_out[:3]) < 0.02
    assert cuda_lib.hg_get_device_status()[0] == cuda_lib.HG_OK
