"""The MoE layer's steps on the GPU at the ends of their ranges, against their float64
definitions.  Tolerances are those of test_gpu_moe_layer unless stated at the test.
"""
import numpy as np
import pytest
import torch

from oracle import moe_layer as L
from synth import make_routing, make_weights
from tests.test_gpu_moe_layer import BF16, FP32, _check_matvec, _close, _f64, _normal

pytestmark = pytest.mark.gpu


# ------------------------------------------------ few-token experts -------

# one column; rows of all tokens held; several runs of units per block
@pytest.mark.parametrize("M,k,E,N,K,per_slot", [(1, 8, 32, 2048, 6144, False),
                                                (13, 8, 12, 1024, 3584, False),
                                                (64, 8, 16, 512, 6144, True)])
def test_expert_matvec_survives_a_wait_limit_of_a_microsecond(cuda_lib, M, k, E, N, K, per_slot):
    # whether or not the limit runs out on copies that are on their way, the
    # status says so and the next call is right
    ids = torch.from_numpy(make_routing(M, E, k, "biased", 3)).cuda()
    w, ws = [t.cuda() for t in make_weights(E, N, K, seed=9)]
    x = _normal(2, M * k if per_slot else M, K).bfloat16().cuda()
    cuda_lib.hg_get_device_status()
    want = cuda_lib.hg_expert_matvec(x, ids, w, ws)
    assert cuda_lib.hg_get_device_status()[0] == cuda_lib.HG_OK
    cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    try:
        cuda_lib.lib.hg_set_wait_timeout_us(1)
        for _ in range(5):
            cold.fill_(1)                                   # the weights leave L2
            got = cuda_lib.hg_expert_matvec(x, ids, w, ws)
            status, detail = cuda_lib.hg_get_device_status()
            if status == cuda_lib.HG_OK:
                assert torch.equal(got, want)
            else:
                assert status == cuda_lib.HG_ERR_TIMEOUT and detail >> 24 == 8
    finally:
        cuda_lib.lib.hg_set_wait_timeout_us(0)
    assert torch.equal(cuda_lib.hg_expert_matvec(x, ids, w, ws), want)
    assert cuda_lib.hg_get_device_status()[0] == cuda_lib.HG_OK


def _ones(N, K):
    """One expert whose weights are all 1, as (codes, scales)."""
    return (torch.full((1, N, K // 2), 0x22, dtype=torch.uint8),
            torch.full((1, N, K // 32), 127, dtype=torch.uint8))


def _set_code(w, n, k, code):
    byte = w[0, n, k // 2]
    w[0, n, k // 2] = (byte & 0x0F) | (code << 4) if k & 1 else (byte & 0xF0) | code


@pytest.mark.parametrize("M", [1, 3, 13])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("power", [24, 31, 32, 39, 40, 62, 64, 100, 127])
def test_expert_matvec_outlier_that_meets_zero_weights(cuda_lib, M, swiglu, power):
    # one element of 2^power among elements near 1, or near 2^-power / 2: it
    # meets zeros, so that the sum is the small elements'
    N, K, k0 = 40, 640, 77
    w, ws = _ones(N, K)
    for n in range(N):
        _set_code(w, n, k0, 0)
    x = torch.full((M, K), 2.0 ** -6 if swiglu else 1.0078125)
    x[:, 256:512] = 1.5 * 2.0 ** -(power // 2)
    x[:, 300] = 0.0
    if M > 1:
        x[1] = 0.25                                         # a row without outliers
    x[0, k0] = 2.0 ** power
    x[-1, k0] = -(2.0 ** power)
    ids = np.zeros((M, 1), dtype=np.int32)
    _check_matvec(cuda_lib, M, 1, 1, N, K, False, swiglu, ids=ids, x=x.bfloat16(), w=(w, ws))


@pytest.mark.parametrize("M,E,per_slot", [(1, 1, False), (2, 1, False), (11, 1, False),
                                          (4, 3, True)])
@pytest.mark.parametrize("span", [30, 60, 120])
def test_expert_matvec_any_range_within_a_row(cuda_lib, M, E, per_slot, span):
    # element k of every row lies near 2^p_k, p_k over [-span, span]; weight row
    # n is zero wherever p_k is above a limit of its own, so that each output is
    # decided by elements of another size
    N, K = 48, 896
    rng = np.random.default_rng(span + M)
    p = rng.integers(-span, span + 1, K)
    rows = M * 2 if per_slot else M
    x = torch.from_numpy(rng.choice([-1.0, 1.0], (rows, K)) * rng.uniform(1, 2, (rows, K))
                         * 2.0 ** p).bfloat16()
    code = rng.integers(0, 16, (E, N, K))
    limit = np.linspace(-span + 2, span, N).round()[None, :, None]
    code[np.broadcast_to(p > limit, code.shape)] = 0
    w = torch.from_numpy((code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8))
    ws = torch.from_numpy(rng.integers(120, 126, (E, N, K // 32)).astype(np.uint8))
    ids = rng.integers(0, E, (M, 2)).astype(np.int32)
    _check_matvec(cuda_lib, M, 2, E, N, K, per_slot, False, ids=ids, x=x, w=(w, ws))


@pytest.mark.parametrize("M", [1, 5])
def test_expert_matvec_non_finite_rows_beside_wide_ones(cuda_lib, M):
    # a row of many powers of two next to one with an Inf or a NaN: each decides
    # its own outputs (511 rounds to 512)
    N, K = 18, 512
    w, ws = _ones(N, K)
    x = torch.ones(M, K)
    x[:, 3] = 2.0 ** -50
    x[0, 300] = float("inf")
    if M > 1:
        x[1, 7], x[2, 8] = float("nan"), float("-inf")
        x[3, 9] = 2.0 ** 90
    y = cuda_lib.hg_expert_matvec(x.bfloat16().cuda(), torch.zeros(M, 1, dtype=torch.int32).cuda(),
                                  w.cuda(), ws.cuda()).float().cpu()
    assert (y[0] == float("inf")).all()
    if M > 1:
        assert y[1].isnan().all() and (y[2] == float("-inf")).all()
        assert (y[3] == 2.0 ** 90).all() and (y[4] == K).all()


@pytest.mark.parametrize("M", [1, 3, 12])
def test_expert_matvec_scales_against_rows(cuda_lib, M):
    # 256-element pieces of x near 2^e with weight scales near 2^-e, and groups
    # of zero weights whose scales are anything up to 2^127
    N, K = 34, 1536
    rng = np.random.default_rng(M)
    e = np.array([-120, 124, 60, -60, 125, -118])
    e = rng.permutation(e)
    x = torch.from_numpy(rng.standard_normal((M, K)) * 2.0 ** np.repeat(e, 256)).bfloat16()
    code = rng.integers(0, 16, (1, N, K))
    s = np.broadcast_to(np.clip(127 - np.repeat(e, 8), 0, 254), (1, N, K // 32)).copy()
    s += rng.integers(-1, 1, s.shape)
    none = rng.random(s.shape) < 0.3                        # groups without weights
    code[np.repeat(none, 32, axis=2)] = 0
    s[none] = rng.choice([0, 1, 100, 150, 200, 254], int(none.sum()))
    s = np.clip(s, 0, 254)
    w = torch.from_numpy((code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8))
    ids = np.zeros((M, 1), dtype=np.int32)
    _check_matvec(cuda_lib, M, 1, 1, N, K, False, False, ids=ids, x=x,
                  w=(w, torch.from_numpy(s.astype(np.uint8))))


@pytest.mark.parametrize("M", [1, 5])
def test_expert_matvec_zero_weights_under_the_largest_scale(cuda_lib, M):
    # 0 * 2^127 times a row of 2^15 and more adds nothing
    N, K = 18, 512
    w, ws = _ones(N, K)
    w[:, :, 16:32] = 0                                      # the second group of 32
    ws[:, :, 1] = 254
    x = torch.ones(M, K)
    x[:, 5], x[0, 40] = 2.0 ** 15, 2.0 ** 20
    ids = np.zeros((M, 1), dtype=np.int32)
    _check_matvec(cuda_lib, M, 1, 1, N, K, False, False, ids=ids, x=x.bfloat16(), w=(w, ws))


@pytest.mark.parametrize("M,k,E,K", [(6, 2, 4, 512), (48, 4, 5, 8192), (3, 1, 2, 384)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_expert_matvec_wide_rows_among_others(cuda_lib, M, k, E, K, swiglu):
    # some rows hold elements that their largest would swamp, one belongs to no
    # expert and holds NaN; several runs of units per block in the largest case
    N = 72
    rng = np.random.default_rng(M + K)
    ids = make_routing(M, E, k, "biased", 4)
    x = rng.standard_normal((M, K))
    x[::3] *= 2.0 ** rng.integers(-50, 20, (len(x[::3]), K))
    x[M // 2] = np.nan
    ids[M // 2] = -1
    w, ws = make_weights(E, N, K, seed=11)
    x = torch.from_numpy(x).bfloat16()
    got = cuda_lib.hg_expert_matvec_swiglu if swiglu else cuda_lib.hg_expert_matvec
    y = got(x.cuda(), torch.from_numpy(ids).cuda(), w.cuda(), ws.cuda())
    assert float(y[M // 2 * k:(M // 2 + 1) * k].float().abs().max()) == 0
    x[M // 2] = 0.0                                         # what the definition is given
    ref, mag = L.expert_matvec(_f64(x), ids, w.numpy(), ws.numpy())
    err = 2 * K * FP32 * mag
    if swiglu:
        g, u, eg, eu = ref[:, :N // 2], ref[:, N // 2:], err[:, :N // 2], err[:, N // 2:]
        ref = g * L.sigmoid(g) * u
        err = 1.1 * eg * (np.abs(u) + eu) + np.abs(g * L.sigmoid(g)) * eu + 2.0 ** -16 * np.abs(ref)
    _close(_f64(y), ref, BF16 * np.abs(ref) + err + 2.0 ** -134)


# --------------------------------------------------------- SwiGLU ---------

def test_swiglu_quantize_gates_far_below_zero(cuda_lib):
    # silu(g) leaves FP32's normal numbers below g = -87, u brings h back
    z = torch.zeros(6, 512)
    z[:, :256] = -torch.linspace(60.0, 176.0, 256)
    z[:, 256:] = (2.0 ** torch.tensor([0.0, 60.0, 90.0, 110.0, 120.0, 127.0]))[:, None]
    z[5, 256::2] *= -1.0
    z = z.bfloat16()
    a, s, _, _ = cuda_lib.hg_swiglu_quantize(z.cuda(), False)
    # exp's argument is off by |g| 2^-24 at most
    h = L.swiglu(_f64(z))
    e, amax = L.group_exponents(h)
    got_e = s.cpu().numpy().astype(np.int64) - 127
    near = np.abs(amax / np.ldexp(448.0, got_e) - 1) < 2.0 ** -12
    near |= np.abs(amax / np.ldexp(224.0, got_e) - 1) < 2.0 ** -12
    # below FP32's smallest normal number h may be 0, and its scale then 2^0
    assert np.all((got_e == e) | near | (amax < 2.0 ** -126))
    dec = L.dequantize(a.cpu().numpy(), s.cpu().numpy())
    low = np.repeat(np.ldexp(1.0, got_e - 10), 128, axis=1)
    # 2^-126 is FP32's smallest normal number
    _close(dec, h, np.maximum(2.0 ** -4 * np.abs(h), low) + 2.0 ** -12 * np.abs(h) + 2.0 ** -126)


def _swiglu_bwd(cuda_lib, g, u, dh):
    """Codes and scales of checkpoints of one group each; dz and what it should be."""
    zf = np.concatenate([g, u], axis=1)
    q, qs = L.quantize(zf)
    zf = L.dequantize(q, qs)
    d = torch.from_numpy(dh).bfloat16()
    dz = cuda_lib.hg_swiglu_bwd(d.cuda(), torch.from_numpy(q).cuda(), torch.from_numpy(qs).cuda())
    want = L.swiglu_bwd(_f64(d), zf)
    F = dh.shape[1]
    gate, up, s = zf[:, :F], zf[:, F:], L.sigmoid(zf[:, :F])
    mag = np.concatenate([np.abs(_f64(d) * up) * s * (1 + np.abs(gate) * L.sigmoid(-gate)),
                          np.abs(_f64(d) * gate) * s], axis=1)
    return _f64(dz), want, mag


@pytest.mark.parametrize("low,high,u,d", [(-170.0, -80.0, 2.0 ** 100, 2.0 ** 20),
                                          (-170.0, -80.0, 2.0 ** 20, 2.0 ** 100),
                                          (-120.0, -60.0, 2.0 ** 100, 2.0 ** 90),
                                          (-80.0, -70.0, 2.0 ** 127, 2.0 ** 80),
                                          (-300.0, 300.0, 1.0, 1.0),
                                          (-100.0, -88.0, 2.0 ** -20, 2.0 ** 127)])
def test_swiglu_bwd_far_below_zero_and_large(cuda_lib, low, high, u, d):
    # s alone underflows, or dh * u alone overflows, where the gradient does neither
    g = np.linspace(low, high, 256)[None]
    sign = np.where(np.arange(256) % 3 == 0, -1.0, 1.0)[None]
    got, want, mag = _swiglu_bwd(cuda_lib, g, u * sign, d * np.ones((1, 256)))
    assert np.abs(want).max() < 2.0 ** 127
    _close(got, want, BF16 * np.abs(want) + 2.0 ** -16 * mag + 2.0 ** -134)


# ------------------------------------------------------------ router ------

def _saturated(M, E, seed):
    """Logits of which one per row is larger than the others by 0 to 40."""
    l = _normal(seed, M, E)
    top = torch.randint(0, E, (M,), generator=torch.Generator().manual_seed(seed))
    l[torch.arange(M), top] = l.amax(1) + torch.linspace(0.0, 40.0, M)
    return l


@pytest.mark.parametrize("E,k", [(64, 8), (16, 1), (160, 6), (600, 4), (8, 8)])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_of_saturated_rows(cuda_lib, E, k, renorm):
    # relative to the gradient's own size, which is that of the small weights
    # where one is nearly 1: with q_i the other probabilities, dl_j is w_j times
    # sum_i q_i (dw_j - dw_i), and each factor is off by (E + 64) * 2^-24 of itself
    M = 41
    logits = _saturated(M, E, E + k)
    dw = _normal(E, M, k)
    ids, w = cuda_lib.hg_router_topk(logits.cuda(), k, renorm)
    d = cuda_lib.hg_router_topk_bwd(logits.cuda(), ids, w, dw.cuda(), renorm)
    got, lf, df, chosen = d.double().cpu().numpy(), logits.double().numpy(), dw.double().numpy(), \
        ids.cpu().numpy()
    p = np.exp(lf - lf.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    want, mag = np.zeros_like(p), np.zeros_like(p)
    for t in range(M):
        q, full = p[t].copy(), np.zeros(E)
        if renorm:
            outside = np.ones(E, bool)
            outside[chosen[t]] = False
            q[outside] = 0.0
            q /= q.sum()
        full[chosen[t]] = df[t]
        for e in range(E):
            want[t, e] = q[e] * np.sum(q * (full[e] - full))
            mag[t, e] = q[e] * np.sum(q * (np.abs(full[e]) + np.abs(full)) * (np.arange(E) != e))
    _close(got, want, 4 * (E + 64) * FP32 * mag + 2.0 ** -126)
    # the exact row adds up to 0
    assert np.all(np.abs(got.sum(1)) <= 4 * (E + 64) * FP32 * mag.sum(1) + E * 2.0 ** -126)


@pytest.mark.parametrize("E,k", [(48, 6), (700, 3), (9, 9)])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_with_choices_dropped_since(cuda_lib, E, k, renorm):
    # choices taken out after the gate, the first among them: the others keep
    # their weights, and the gradient is that of sum over them of w dw
    M = 24
    logits = _normal(E, M, E) * 2
    logits[3] = logits[3] - 200.0 * (torch.arange(E) != 5)    # the rest's weights vanish
    dw = _normal(E + 1, M, k)
    ids, w = cuda_lib.hg_router_topk(logits.cuda(), k, renorm)
    rng = np.random.default_rng(E)
    keep = rng.random((M, k)) < 0.6
    keep[:8, 0] = False
    keep[8] = False
    kept_ids = np.where(keep, ids.cpu().numpy(), np.where(rng.random((M, k)) < 0.5, -1, E))
    d = cuda_lib.hg_router_topk_bwd(logits.cuda(), torch.from_numpy(kept_ids.astype(np.int32)).cuda(),
                                    w, dw.cuda(), renorm).double().cpu().numpy()
    lf, df, chosen = logits.double().numpy(), dw.double().numpy(), ids.cpu().numpy()
    for t in range(M):
        p = np.exp(lf[t] - lf[t].max())
        p /= p.sum()
        wt = p[chosen[t]] / (p[chosen[t]].sum() if renorm else 1.0)
        c = np.sum((wt * df[t])[keep[t]])
        want = np.zeros(E) if renorm else -p * c
        at = chosen[t][keep[t]]
        want[at] += wt[keep[t]] * (df[t][keep[t]] - (c if renorm else 0.0))
        mag = np.sum(np.abs(wt * df[t])) + np.abs(want)
        _close(d[t], want, 4 * (E + 64) * FP32 * mag + 2.0 ** -126, t)


@pytest.mark.parametrize("M", [1, 5, 12])
@pytest.mark.parametrize("spread", [3, 20])
def test_expert_matvec_on_activations_of_many_powers(cuda_lib, M, spread):
    # a SwiGLU's outputs, whose gates far below zero leave e^g: much of a row is far
    # below its largest, and shows only in outputs that are small themselves
    k, E, N, K = 2, 3, 1000, 2048
    g, u = _normal(40 + M, M * k, K) * spread, _normal(41 + M, M * k, K)
    x = (g * torch.sigmoid(g) * u).bfloat16()
    ids = make_routing(M, E, k, "biased", 8)
    w, ws = make_weights(E, N, K, seed=12)
    w[:, 5:9, :K // 4] = 0                                  # rows that miss a row's largest
    big = x.float().abs().amax(0) > 2.0 ** -20
    code = torch.stack([w & 15, w >> 4], dim=-1).view(E, N, K)
    code[:, 20:24, big] = 0                                 # and some that miss all but the smallest
    w = (code[..., 0::2] | code[..., 1::2] << 4).contiguous()
    _check_matvec(cuda_lib, M, k, E, N, K, True, False, ids=ids, x=x, w=(w, ws))
