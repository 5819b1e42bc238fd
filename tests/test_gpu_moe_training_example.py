"""examples/moe_layer.py's training of the experts: the block behind its norm, forward and
backward, against the float64 chain on the same 4-bit weights, and the weights quantised anew.

Tolerance, as for the layer alone: an E4M3 rounding is off by up to 2^-4 of a value, about 2.6 %
in the 2-norm, and a result passes through at most six; sqrt(6) * 2.6 % is 6.4 %; 10 % are
allowed.  y is the residual stream's BF16 (one rounding of s, one of the sum, 2^-8 each) plus a
layer's output that is 10 % off at most.
"""
import numpy as np
import pytest
import torch

from oracle import expert_training as T
from oracle import moe_layer as L
from tests.test_gpu_moe_example import _example, _f64, _off, _weights

pytestmark = pytest.mark.gpu


def test_block_trains_its_experts(cuda_lib):
    ex = _example()
    D, F, E, k, M = 256, 128, 8, 2, 70
    g = torch.Generator().manual_seed(11)
    masters = [torch.randn(E, 2 * F, D, generator=g) / D ** 0.5,
               torch.randn(E, D, F, generator=g) / F ** 0.5]
    experts = ex.Experts.from_float(*(w.cuda() for w in masters))
    x, res, dout = (torch.randn(M, D, generator=g).bfloat16() for _ in range(3))
    gain = (1 + 0.1 * torch.randn(D, generator=g)).bfloat16()
    router = torch.randn(D, E, generator=g) / D ** 0.5
    y, dx, dgain, drouter, (dgu, ddn) = ex.train_block(
        x.cuda(), res.cuda(), gain.cuda(), router.cuda(), dout.cuda(), k, experts)

    s, r, n = T.rmsnorm(_f64(x), _f64(res), _f64(gain), 1e-6)
    # the router's choice is made on BF16 values of n: the same here, since ties are far
    nb = torch.from_numpy(n).bfloat16()
    logits = (nb.float().cuda() @ router.cuda()).double().cpu().numpy()
    ids, w = L.router_topk(logits, k, True)
    gu, dn = _weights(experts.gate_up), _weights(experts.down)
    gu_t, dn_t = _weights(experts.gate_up_t), _weights(experts.down_t)
    df, out, dn_in = _f64(dout), np.zeros((M, D)), np.zeros((M, D))
    want_gu, want_dn, dw = np.zeros(gu.shape), np.zeros(dn.shape), np.zeros((M, k))
    for t in range(M):
        for j in range(k):
            e = ids[t, j]
            z = (gu[e] @ n[t])[None]
            h = L.swiglu(z)
            o = dn[e] @ h[0]
            out[t] += w[t, j] * o
            dw[t, j] = df[t] @ o
            do = w[t, j] * df[t]
            dz = L.swiglu_bwd((dn_t[e] @ do)[None], z)[0]
            dn_in[t] += gu_t[e] @ dz
            want_gu[e] += np.outer(dz, n[t])
            want_dn[e] += np.outer(do, h[0])
    dlogits = L.router_topk_bwd(logits, ids, dw, True)
    dn_in += dlogits @ router.double().numpy().T
    want_dx, want_dgain, _, _ = T.rmsnorm_bwd(dn_in, s, _f64(gain), r, df)
    assert (np.abs(_f64(y) - (s + out)) <= 2.0 ** -8 * np.abs(s + out) + 2.0 ** -8 * np.abs(out) +
            0.1 * np.linalg.norm(out) / np.sqrt(out.size) * 6).all()
    assert _off(_f64(dx) - df, want_dx - df) < 0.1
    for got, want in ((dgain, want_dgain), (drouter, nb.double().numpy().T @ dlogits),
                      (dgu, want_gu), (ddn, want_dn)):
        assert _off(got.double().cpu().numpy(), want) < 0.1
    assert cuda_lib.hg_get_device_status()[0] == cuda_lib.HG_OK

    # an update: the 4-bit weights are those of the new masters, in both orientations
    before = experts.gate_up[0].clone()
    new = [(m.cuda() - 0.05 * d / d.norm() * m.cuda().norm()) for m, d in zip(masters, (dgu, ddn))]
    experts.quantize(*new)
    assert not torch.equal(before, experts.gate_up[0])
    for pair, pair_t, m in ((experts.gate_up, experts.gate_up_t, new[0]),
                            (experts.down, experts.down_t, new[1])):
        m = m.double().cpu().numpy()
        for (q, sc), v in ((pair, m), (pair_t, np.ascontiguousarray(m.transpose(0, 2, 1)))):
            wq, ws = T.quantize_weights(v)
            assert (q.cpu().numpy() == wq).all() and (sc.cpu().numpy() == ws).all()


def test_block_captured_and_replayed(cuda_lib):
    """The whole step as a graph: the same bits as without, on new contents of its inputs too."""
    ex = _example()
    D, F, E, k, M = 256, 128, 4, 2, 40
    g = torch.Generator().manual_seed(12)
    experts = ex.Experts.from_float((torch.randn(E, 2 * F, D, generator=g) / 16).cuda(),
                                    (torch.randn(E, D, F, generator=g) / 11).cuda())
    x, res, dout = (torch.randn(M, D, generator=g).bfloat16().cuda() for _ in range(3))
    gain = torch.ones(D).bfloat16().cuda()
    router = (torch.randn(D, E, generator=g) / 16).cuda()

    def step():
        y, dx, dgain, drouter, grads = ex.train_block(x, res, gain, router, dout, k, experts)
        return y, dx, dgain, drouter, *grads

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (1, 2):
        x.copy_(torch.randn(M, D, generator=torch.Generator().manual_seed(seed)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, step()):
            assert torch.equal(got, want)
    assert cuda_lib.hg_get_device_status()[0] == cuda_lib.HG_OK
