"""The MoE layer's steps on the GPU against their float64 definitions: dispatch and the
gradients of dispatch and combine, SwiGLU with its 8-bit checkpoint, the few-token expert
product, the router's gate.

Tolerances, fixed before the first run:

* BF16 has 8 significant bits, so one rounding is off by at most 2^-8 of the value (2^-134 in
  the subnormal range).
* An FP32 sum of n terms in any order is off by at most (n - 1) * 2^-24 of the sum of the
  terms' magnitudes (to first order); tensor-core sums may cut instead of rounding: twice that.
* E4M3 rounding is off by at most 2^-4 of the value, or 2^-10 of the scale below 2^-6 of it.
"""
import numpy as np
import pytest
import torch

from oracle import moe_layer as L
from oracle.formats import E8M0_TABLE, bf16_bits_to_f64
from oracle.moe_io import quantize_rows
from oracle.plan import plan_expert_offsets
from synth import make_routing, make_weights

pytestmark = pytest.mark.gpu

BF16, FP32 = 2.0 ** -8, 2.0 ** -24
BF16_OVERFLOW = (2.0 - 2.0 ** -8) * 2.0 ** 127             # values from here on round to infinity


def _f64(t):
    return bf16_bits_to_f64(t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))


def _normal(seed, *shape):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g)


def _close(got, want, bound, what=""):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           got[bad][:3], want[bad][:3])


def _place(M, E, k, seed, drop=0):
    ids = make_routing(M, E, k, "biased", seed)
    _, _, d2s, _ = plan_expert_offsets(ids, E)
    d2s = d2s.copy()
    d2s[np.random.default_rng(seed).permutation(M * k)[:drop]] = -1
    return d2s


# ------------------------------------------------- tokens by expert -------

# one token; odd sizes; a row of one 16-byte chunk; one chunk more than a
# block's 2048 columns and than two of them; many choices; the layer's widths
TOKENS = [(1, 8, 1, 4, 0), (1, 6144, 8, 32, 0), (7, 40, 3, 8, 4), (33, 2056, 8, 32, 9),
          (5, 4104, 12, 16, 7), (19, 8200, 2, 4, 5), (3, 264, 40, 64, 11), (300, 2048, 8, 32, 100),
          (70, 16392, 1, 8, 6)]


@pytest.mark.parametrize("M,K,k,E,drop", TOKENS)
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_tokens(cuda_lib, M, K, k, E, drop, weighted):
    place = _place(M, E, k, M + K, drop)
    x = _normal(M + K, M, K).to(torch.bfloat16)
    w = torch.softmax(_normal(k, M, k), 1) if weighted else None
    out = torch.full((M * k, K), 7.0, dtype=torch.bfloat16, device="cuda")
    got = cuda_lib.hg_dispatch_tokens(x.cuda(), k, torch.from_numpy(place).cuda(),
                                      None if w is None else w.cuda(), out=out)
    assert got is out
    want = L.dispatch(_f64(x), place.reshape(M, k), None if w is None else w.double().numpy(),
                      np.full((M * k, K), 7.0))
    _close(_f64(out), want, (BF16 + FP32) * np.abs(want) if weighted else 0.0)


@pytest.mark.parametrize("M,K,k,E,drop", TOKENS)
@pytest.mark.parametrize("weighted,dots", [(False, False), (True, True), (False, True),
                                           (True, False)])
def test_dispatch_tokens_bwd(cuda_lib, M, K, k, E, drop, weighted, dots):
    place = _place(M, E, k, M + K + 1, drop)
    x = _normal(1, M, K).to(torch.bfloat16)
    rows = _normal(2, M * k, K).to(torch.bfloat16)
    w = _normal(3, M, k) if weighted else None
    dx, dw = cuda_lib.hg_dispatch_tokens_bwd(rows.cuda(), k, torch.from_numpy(place).cuda(),
                                             None if w is None else w.cuda(),
                                             x.cuda() if dots else None)
    want, mag = L.combine(_f64(rows), place.reshape(M, k),
                          None if w is None else w.double().numpy())
    _close(_f64(dx), want, BF16 * np.abs(want) + k * FP32 * mag + 2.0 ** -134, "dx")
    if not dots:
        assert dw is None
        return
    want, mag = L.row_dots(_f64(rows), _f64(x), place.reshape(M, k))
    _close(dw.double().cpu().numpy(), want, K * FP32 * mag, "dw")


@pytest.mark.parametrize("M,N,k,E,drop", TOKENS)
def test_combine_topk_bwd(cuda_lib, M, N, k, E, drop):
    place = _place(M, E, k, M + N + 2, drop)
    dout = _normal(4, M, N).to(torch.bfloat16)
    y = _normal(5, M * k, N).to(torch.bfloat16)
    w = torch.softmax(_normal(6, M, k), 1)
    dy = torch.full((M * k, N), 7.0, dtype=torch.bfloat16, device="cuda")
    _, dw = cuda_lib.hg_combine_topk_bwd(dout.cuda(), y.cuda(), torch.from_numpy(place).cuda(),
                                         w.cuda(), dy=dy)
    want = L.dispatch(_f64(dout), place.reshape(M, k), w.double().numpy(), np.full((M * k, N), 7.0))
    _close(_f64(dy), want, (BF16 + FP32) * np.abs(want), "dy")
    want, mag = L.row_dots(_f64(y), _f64(dout), place.reshape(M, k))
    _close(dw.double().cpu().numpy(), want, N * FP32 * mag, "dw")


# tokens enough for a warp each: several passes over a row, one choice, more
# choices than are reduced together
@pytest.mark.parametrize("M,N,k,E,drop", [(2500, 2056, 1, 8, 40), (2433, 1032, 9, 16, 300),
                                          (2600, 520, 3, 8, 0)])
def test_token_gradients_of_many_tokens(cuda_lib, M, N, k, E, drop):
    place = _place(M, E, k, M + N + 3, drop)
    p, d2s = place.reshape(M, k), torch.from_numpy(place).cuda()
    x = _normal(15, M, N).to(torch.bfloat16)
    rows = _normal(16, M * k, N).to(torch.bfloat16)
    w = _normal(17, M, k)
    xf, rf, wf = _f64(x), _f64(rows), w.double().numpy()
    dx, dw = cuda_lib.hg_dispatch_tokens_bwd(rows.cuda(), k, d2s, w.cuda(), x.cuda())
    want, mag = L.combine(rf, p, wf)
    _close(_f64(dx), want, BF16 * np.abs(want) + k * FP32 * mag + 2.0 ** -134, "dx")
    dots, mag = L.row_dots(rf, xf, p)
    _close(dw.double().cpu().numpy(), dots, N * FP32 * mag, "dw")
    dy = torch.full((M * k, N), 7.0, dtype=torch.bfloat16, device="cuda")
    _, dw = cuda_lib.hg_combine_topk_bwd(x.cuda(), rows.cuda(), d2s, w.cuda(), dy=dy)
    _close(dw.double().cpu().numpy(), dots, N * FP32 * mag, "dw of the combine")
    want = L.dispatch(xf, p, wf, np.full((M * k, N), 7.0))
    _close(_f64(dy), want, (BF16 + FP32) * np.abs(want), "dy")


def test_tokens_with_every_choice_dropped_and_entries_out_of_range(cuda_lib):
    M, K, k = 6, 136, 2
    place = np.array([-1, -1, 3, 12, -5, 0, 1 << 30, -1, 2, 1, -2 ** 31, 4], dtype=np.int32)
    d2s = torch.from_numpy(place).cuda()
    x = _normal(7, M, K).to(torch.bfloat16)
    rows = _normal(8, M * k, K).to(torch.bfloat16)
    rows[5] = float("nan")                              # a row nobody names is not read
    w = _normal(9, M, k)
    out = torch.full((M * k, K), 7.0, dtype=torch.bfloat16, device="cuda")
    cuda_lib.hg_dispatch_tokens(x.cuda(), k, d2s, out=out)
    p = place.reshape(M, k)
    assert np.array_equal(_f64(out), L.dispatch(_f64(x), p, None, np.full((M * k, K), 7.0)))
    dx, dw = cuda_lib.hg_dispatch_tokens_bwd(rows.cuda(), k, d2s, w.cuda(), x.cuda())
    _, dw2 = cuda_lib.hg_combine_topk_bwd(x.cuda(), rows.cuda(), d2s, w.cuda(), dy=out)
    clean = np.nan_to_num(_f64(rows))
    want, mag = L.combine(clean, p, w.double().numpy())
    _close(_f64(dx), want, BF16 * np.abs(want) + k * FP32 * mag + 2.0 ** -134)
    want, mag = L.row_dots(clean, _f64(x), p)
    _close(dw.double().cpu().numpy(), want, K * FP32 * mag)
    _close(dw2.double().cpu().numpy(), want, K * FP32 * mag)
    assert float(dx[0].abs().max()) == 0 and dw[0].tolist() == [0, 0]


def test_tokens_offsets_beyond_32_bits(cuda_lib):
    # 2^19 + 8 rows of 8200: element offsets beyond 2^32; sampled rows are checked
    M, k, K = 65537, 8, 8200
    R = M * k
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    place = torch.randperm(R, generator=g, device="cuda").to(torch.int32)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    rows = cuda_lib.hg_dispatch_tokens(x, k, place)
    for t in (0, 1, M // 2, M - 1):
        for j in (0, 7):
            assert torch.equal(rows[int(place[t * k + j])], x[t])
    w = torch.ones(M, k, device="cuda")
    dx, dw = cuda_lib.hg_dispatch_tokens_bwd(rows, k, place, w, x)
    for t in (0, 1, M // 2, M - 1):
        assert torch.equal(dx[t], x[t] * 8)
        want = float(x[t].double().square().sum())
        assert abs(float(dw[t, 3]) - want) <= K * FP32 * want
    dy, dw = cuda_lib.hg_combine_topk_bwd(x, rows, place, w * 0.5)
    for t in (0, M - 1):
        assert torch.equal(dy[int(place[t * k + 7])], x[t] * 0.5)
    assert int((rows == 0).all(dim=1).sum()) == 0        # every row was written


# --------------------------------------------------------- SwiGLU ---------

def _check_swiglu(cuda_lib, z, checkpoint):
    rows, F2 = z.shape
    F = F2 // 2
    a, s, q, qs = cuda_lib.hg_swiglu_quantize(z.cuda(), checkpoint)
    zf = _f64(z)
    h = L.swiglu(zf)
    e, amax = L.group_exponents(h)
    got_e = s.cpu().numpy().astype(np.int64) - 127
    # the scale is the definition's, except where FP32 rounding can carry the
    # largest magnitude over a power of two times 448
    near = np.abs(amax / np.ldexp(448.0, got_e) - 1) < 2.0 ** -12
    near |= np.abs(amax / np.ldexp(224.0, got_e) - 1) < 2.0 ** -12
    assert np.all((got_e == e) | near)
    dec = L.dequantize(a.cpu().numpy(), s.cpu().numpy())
    low = np.repeat(np.ldexp(1.0, got_e - 10), 128, axis=1)
    _close(dec, h, np.maximum(2.0 ** -4 * np.abs(h), low) + 2.0 ** -12 * np.abs(h), "h")
    if not checkpoint:
        assert q is None and qs is None
        return
    rc, rs = L.quantize(zf)
    assert np.array_equal(q.cpu().numpy(), rc) and np.array_equal(qs.cpu().numpy(), rs)


@pytest.mark.parametrize("rows,F", [(1, 128), (1, 2048), (3, 384), (17, 2048), (130, 640),
                                    (1000, 256)])
@pytest.mark.parametrize("checkpoint", [False, True])
def test_swiglu_quantize(cuda_lib, rows, F, checkpoint):
    z = (_normal(rows + F, rows, 2 * F) * 3).to(torch.bfloat16)
    _check_swiglu(cuda_lib, z, checkpoint)


def test_swiglu_quantize_special_values(cuda_lib):
    z = _normal(3, 8, 512).to(torch.bfloat16)
    z[0, :128] = 0.0                        # zero gate group: h = 0, scale 2^0
    z[1, 256:384] = 0.0                     # zero up group
    z[2, :128] = 60.0                       # saturated gates
    z[2, 128:256] = -60.0
    z[3] = z[3] * 2.0 ** 60
    z[4] = z[4] * 2.0 ** -70
    z[5, :128] = 448.0
    _check_swiglu(cuda_lib, z, True)
    z[6, 3] = float("nan")                  # columns 0..127 of h and of g
    z[7, 256 + 130] = float("inf")          # columns 128..255 of h, group 3 of z
    a, s, q, qs = [v.cpu().numpy() for v in cuda_lib.hg_swiglu_quantize(z.cuda(), True)]
    assert s[6].tolist()[0] == 255 and s[6, 1] != 255 and (a[6, :128] == 0x7F).all()
    assert s[7, 1] == 255 and s[7, 0] != 255 and (a[7, 128:] == 0x7F).all()
    assert [v == 255 for v in qs[6]] == [True, False, False, False]
    assert [v == 255 for v in qs[7]] == [False, False, False, True]
    bits = z.view(torch.int16).numpy().view(np.uint16)
    rc, rs = quantize_rows(bits)
    assert np.array_equal(q, rc) and np.array_equal(qs, rs)


def _check_swiglu_bwd(dz, dh, zf):
    F = dh.shape[1]
    want = L.swiglu_bwd(dh, zf)
    g, u = zf[:, :F], zf[:, F:]
    s = L.sigmoid(g)
    # FP32: each factor is off by some 2^-24, exp(-g) by |g| of that: 2^-16 of
    # the terms' magnitudes covers |g| up to 100
    mag = np.concatenate([np.abs(dh * u) * s * (1 + np.abs(g) * L.sigmoid(-g)),
                          np.abs(dh * g) * s], axis=1)
    tiny = 2.0 ** -120 * np.concatenate([np.abs(dh * u * g) + np.abs(dh * u), np.abs(dh * g)], 1)
    _close(_f64(dz), want, BF16 * np.abs(want) + 2.0 ** -16 * mag + tiny + 2.0 ** -134, "dz")


@pytest.mark.parametrize("rows,F", [(1, 128), (1, 2048), (3, 384), (17, 2048), (131, 640),
                                    (1000, 256)])
def test_swiglu_bwd(cuda_lib, rows, F):
    z = (_normal(rows, rows, 2 * F) * 4).to(torch.bfloat16)
    if rows == 17:
        z[3] = z[3] * 25                                  # |g| to 100 and beyond
    dh = _normal(F, rows, F).to(torch.bfloat16)
    _, _, q, qs = cuda_lib.hg_swiglu_quantize(z.cuda(), True)
    dz = cuda_lib.hg_swiglu_bwd(dh.cuda(), q, qs)
    zf = L.dequantize(q.cpu().numpy(), qs.cpu().numpy())
    _check_swiglu_bwd(dz, _f64(dh), zf)


def test_swiglu_bwd_every_code_and_extreme_scales(cuda_lib):
    # all 254 finite E4M3 codes as gate and up, scale codes from 0 (2^-127) upwards
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F] + [0, 0x80], dtype=np.uint8)
    q = np.concatenate([codes, np.roll(codes, 77)])[None, :].repeat(4, 0)
    qs = np.array([[120, 121, 127, 110], [0, 1, 0, 2], [117, 118, 3, 0], [127, 90, 200, 160]],
                  dtype=np.uint8)
    dh = _normal(5, 4, 256).to(torch.bfloat16)
    dz = cuda_lib.hg_swiglu_bwd(dh.cuda(), torch.from_numpy(q).cuda(), torch.from_numpy(qs).cuda())
    _check_swiglu_bwd(dz, _f64(dh), L.dequantize(q, qs))


def test_swiglu_gradient_against_differences(cuda_lib):
    # central differences of the float64 forward at the checkpointed z: off by
    # h^2 / 6 times a third derivative of order 10, beside the BF16 rounding
    z = (_normal(6, 2, 256) * 2).to(torch.bfloat16)
    dh = _normal(7, 2, 128).to(torch.bfloat16)
    _, _, q, qs = cuda_lib.hg_swiglu_quantize(z.cuda(), True)
    dz = _f64(cuda_lib.hg_swiglu_bwd(dh.cuda(), q, qs))
    zf, d, h = L.dequantize(q.cpu().numpy(), qs.cpu().numpy()), _f64(dh), 1e-4
    want = np.zeros_like(zf)
    for i in np.ndindex(zf.shape):
        a, b = zf.copy(), zf.copy()
        a[i] += h
        b[i] -= h
        want[i] = float(((L.swiglu(a) - L.swiglu(b)) * d).sum()) / (2 * h)
    _close(dz, want, BF16 * np.abs(want) + 1e-5)


def test_swiglu_offsets_beyond_32_bits(cuda_lib):
    rows, F = 270000, 8192                                # 4.4e9 elements of z
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    z = torch.randn(1000, 2 * F, generator=g, device="cuda", dtype=torch.bfloat16)
    z = z.repeat(rows // 1000, 1)
    a, s, q, qs = cuda_lib.hg_swiglu_quantize(z, True)
    dz = cuda_lib.hg_swiglu_bwd(z[:, :F].contiguous(), q, qs)
    del z
    for t in (a, s, q, qs, dz):
        assert torch.equal(t[:1000], t[-1000:]) and torch.equal(t[:1000], t[131000:132000])


# ------------------------------------------------ few-token experts -------

def _check_matvec(cuda_lib, M, k, E, N, K, per_slot, swiglu, seed=0, ids=None, x=None, w=None,
                  out=None):
    rng = np.random.default_rng(seed + N + K)
    if ids is None:
        ids = make_routing(M, E, k, "biased", seed + M)
    wq, ws = make_weights(E, N, K, seed=seed) if w is None else w
    if x is None:
        x = torch.from_numpy(rng.standard_normal((M * k if per_slot else M, K))).to(torch.bfloat16)
    f = cuda_lib.hg_expert_matvec_swiglu if swiglu else cuda_lib.hg_expert_matvec
    got = f(x.cuda(), torch.from_numpy(ids).cuda(), wq.cuda(), ws.cuda(), out=out)
    y, mag = L.expert_matvec(_f64(x), ids, wq.numpy(), ws.numpy())
    err = 2 * K * FP32 * mag
    over = np.abs(y) > BF16_OVERFLOW                        # rounds to an infinity
    assert not (swiglu and over.any())
    if swiglu:
        # h = silu(g) u: |silu'| <= 1.1, and FP32 steps of its own
        F = N // 2
        g, u = y[:, :F], y[:, F:]
        eg, eu = err[:, :F], err[:, F:]
        want = g * L.sigmoid(g) * u
        bound = 1.1 * eg * (np.abs(u) + eu) + np.abs(g * L.sigmoid(g)) * eu
        bound += 2.0 ** -16 * np.abs(want)
    else:
        want, bound = y, err
    gf = _f64(got)
    if over.any():
        assert np.array_equal(gf[over], np.copysign(np.inf, want[over]))
        # below that, a partial sum may pass FP32's largest on the way, in one
        # order of the terms and not in another: nothing is said of these
        over |= mag > 2.0 ** 127
        gf, want = np.where(over, 0.0, gf), np.where(over, 0.0, want)
    _close(gf, want, BF16 * np.abs(want) + bound + 2.0 ** -134)
    # in the 2-norm BF16 rounding alone is off by less than 2^-8
    assert np.linalg.norm(gf - want) <= 2.0 ** -8 * np.linalg.norm(want)
    return got


# one row, one group of scales; heights that end inside a tile; one expert
# with many tokens; more slots than a column block; experts shared and alone
MATVEC = [(1, 1, 1, 1, 128), (1, 1, 1, 2, 128), (1, 2, 4, 6, 256), (1, 8, 32, 500, 640),
          (3, 2, 4, 34, 384), (1, 8, 32, 256, 6144), (2, 8, 12, 130, 3584), (20, 1, 1, 66, 512),
          (13, 8, 12, 96, 1280), (64, 8, 8, 48, 256), (7, 3, 64, 1000, 2048), (9, 1, 2, 18, 16384),
          (2, 2, 2, 22, 32768)]


@pytest.mark.parametrize("M,k,E,N,K", MATVEC)
@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("swiglu", [False, True])
def test_expert_matvec(cuda_lib, M, k, E, N, K, per_slot, swiglu):
    if swiglu and N % 2:
        N += 1
    _check_matvec(cuda_lib, M, k, E, N, K, per_slot, swiglu)


@pytest.mark.parametrize("seed", range(8))
def test_expert_matvec_random(cuda_lib, seed):
    rng = np.random.default_rng(500 + seed)
    E = int(rng.integers(1, 20))
    k = int(rng.integers(1, min(E, 8) + 1))
    M = int(rng.integers(1, 40))
    N = 2 * int(rng.integers(1, 300))
    K = 128 * int(rng.integers(1, 20))
    _check_matvec(cuda_lib, M, k, E, N, K, bool(seed & 1), bool(seed & 2), seed=seed)


@pytest.mark.parametrize("swiglu", [False, True])
def test_expert_matvec_ids_out_of_range_give_zeros(cuda_lib, swiglu):
    ids = np.array([[-1, 3, 0], [4, 1 << 30, -2 ** 31], [2, -1, 4], [1, 1, 1]], dtype=np.int32)
    out = torch.full((12, 10 if swiglu else 20), float("nan"), dtype=torch.bfloat16, device="cuda")
    _check_matvec(cuda_lib, 4, 3, 4, 20, 256, True, swiglu, ids=ids, out=out)
    assert float(out[[0, 3, 4, 5, 7, 8]].abs().max()) == 0
    # no slot with an expert at all
    out.fill_(float("nan"))
    none = np.full((4, 3), -1, dtype=np.int32)
    f = cuda_lib.hg_expert_matvec_swiglu if swiglu else cuda_lib.hg_expert_matvec
    w, ws = make_weights(4, 20, 256, seed=0)
    f(torch.ones(4, 256, dtype=torch.bfloat16).cuda(), torch.from_numpy(none).cuda(), w.cuda(),
      ws.cuda(), out=out)
    assert float(out.abs().max()) == 0


@pytest.mark.parametrize("M,k,E,N,K,per_slot", [
    (20, 4, 6, 40, 384, False), (40, 2, 300, 16, 128, True), (33, 1, 2, 70, 512, False),
    (64, 8, 5, 24, 256, True), (100, 5, 1 << 20, 2, 128, False)])
def test_expert_matvec_many_slots_with_ids_out_of_range(cuda_lib, M, k, E, N, K, per_slot):
    # more than 32 slots: experts met once and often, a choice met twice by a
    # token, ids out of range anywhere among them
    rng = np.random.default_rng(M + E)
    few = rng.integers(0, E, 5) if E > 100 else np.arange(E)
    ids = rng.choice(few, (M, k)).astype(np.int32)
    ids[rng.random((M, k)) < 0.15] = -1
    ids[rng.random((M, k)) < 0.1] = E
    ids[0, 0], ids[-1, -1] = 2 ** 31 - 1, -2 ** 31
    x = torch.from_numpy(rng.standard_normal((M * k if per_slot else M, K))).to(torch.bfloat16)
    w = torch.from_numpy(rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8))
    ws = torch.from_numpy(rng.integers(120, 130, (E, N, K // 32), dtype=np.uint8))
    out = torch.full((M * k, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    _check_matvec(cuda_lib, M, k, E, N, K, per_slot, False, ids=ids, x=x, w=(w, ws), out=out)
    bad = (ids.reshape(-1) < 0) | (ids.reshape(-1) >= E)
    assert bad.any() and float(out[torch.from_numpy(bad).cuda()].abs().max()) == 0


def test_expert_matvec_wide_range(cuda_lib):
    # rows whose elements span many powers of two, and weight scales from 2^-127
    # to 2^60: what is small beside the row's largest element still counts where
    # the largest meets a zero weight
    M, N, K = 4, 40, 512
    rng = np.random.default_rng(8)
    x = rng.standard_normal((M, K)) * 2.0 ** rng.integers(-12, 13, (M, K))
    x[1] *= 2.0 ** 100
    x[2] *= 2.0 ** -110
    x[3] = 0.0
    w = rng.integers(0, 256, (2, N, K // 2)).astype(np.uint8)
    ws = rng.integers(100, 150, (2, N, K // 32)).astype(np.uint8)
    ws[0, 3] = 0
    ws[0, 4] = 187
    ws[1, 5, ::2] = 0
    k = int(np.abs(x[0]).argmax())
    w[:, 7, k // 2] = 0                                     # the row's largest meets zero
    ids = np.array([[0], [1], [0], [1]], dtype=np.int32)
    ws = np.where((ids[1] == 1) & (np.arange(2)[:, None, None] == 1), np.minimum(ws, 140), ws)
    _check_matvec(cuda_lib, M, 1, 2, N, K, False, False, ids=ids,
                  x=torch.from_numpy(x).to(torch.bfloat16),
                  w=(torch.from_numpy(w), torch.from_numpy(ws.astype(np.uint8))))


def test_expert_matvec_nonfinite_rows(cuda_lib):
    # Inf and NaN reach every output of their slot, and no other slot
    M, N, K = 4, 33, 256
    w = torch.full((1, N, K // 2), 0x22, dtype=torch.uint8)          # all weights 1
    ws = torch.full((1, N, K // 32), 127, dtype=torch.uint8)
    x = torch.ones(M, K, dtype=torch.bfloat16)
    x[1, 200] = float("inf")
    x[2, 3] = float("nan")
    x[3, 5] = float("-inf")
    ids = torch.zeros(M, 1, dtype=torch.int32)
    y = cuda_lib.hg_expert_matvec(x.cuda(), ids.cuda(), w.cuda(), ws.cuda()).float().cpu()
    assert (y[0] == K).all() and (y[1] == float("inf")).all()
    assert y[2].isnan().all() and (y[3] == float("-inf")).all()


def test_expert_matvec_repeats_and_agrees_with_gemm(cuda_lib):
    # the same bits every time; and the grouped GEMM's result on activations
    # that E4M3 holds exactly
    M, k, E, N, K = 6, 4, 8, 256, 1024
    ids = make_routing(M, E, k, "uniform", 3)
    x = torch.randint(-8, 9, (M, K), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    w, ws = make_weights(E, N, K, seed=4)
    w, ws, xc, idc = w.cuda(), ws.cuda(), x.cuda(), torch.from_numpy(ids).cuda()
    y = cuda_lib.hg_expert_matvec(xc, idc, w, ws)
    for _ in range(5):
        assert torch.equal(y, cuda_lib.hg_expert_matvec(xc, idc, w, ws))
    off, _, d2s = cuda_lib.hg_plan_expert_offsets(idc, E)
    a, s = cuda_lib.hg_quantize_scatter_acts(xc, k, d2s)
    g = cuda_lib.hg_grouped_w4a8_gemm(a, s, w, ws, off)[d2s.long()]
    ref, mag = L.expert_matvec(_f64(x), ids, w.cpu().numpy(), ws.cpu().numpy())
    _close(_f64(y), _f64(g), 2 * BF16 * np.abs(ref) + 4 * K * FP32 * mag)


@pytest.mark.parametrize("M,K,offset", [(1, 512, 4), (1, 256, 8), (1, 1024, 12), (9, 512, 4),
                                        (9, 256, 4), (9, 1536, 8)])
def test_expert_matvec_scales_at_any_multiple_of_four(cuda_lib, M, K, offset):
    # a view into a larger tensor: the same bits as from a tensor of its own
    k, E, N = 3, 4, 72
    ids = torch.from_numpy(make_routing(M, E, k, "uniform", 5)).cuda()
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    w, ws = (t.cuda() for t in make_weights(E, N, K, seed=7))
    inside = torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")
    inside[offset:offset + ws.numel()] = ws.reshape(-1)
    view = inside[offset:offset + ws.numel()].view(ws.shape)
    assert view.data_ptr() % 16 == offset
    want = cuda_lib.hg_expert_matvec(x, ids, w, ws)
    assert torch.equal(cuda_lib.hg_expert_matvec(x, ids, w, view), want)
    ref, mag = L.expert_matvec(_f64(x), ids.cpu().numpy(), w.cpu().numpy(), ws.cpu().numpy())
    _close(_f64(want), ref, BF16 * np.abs(ref) + 2 * K * FP32 * mag)


def test_expert_matvec_weights_beyond_32_bits(cuda_lib):
    E, N, K = 512, 2100, 8192                                # 4.4 GB of codes
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(120, 130, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    ids = torch.tensor([[0, 511, 510]], dtype=torch.int32)
    x = torch.randn(1, K, generator=g, device="cuda", dtype=torch.bfloat16)
    y = cuda_lib.hg_expert_matvec(x, ids.cuda(), w, ws)
    sub = [0, 511, 510]
    ref, mag = L.expert_matvec(_f64(x), np.array([[0, 1, 2]]), w[sub].cpu().numpy(),
                               ws[sub].cpu().numpy())
    _close(_f64(y), ref, BF16 * np.abs(ref) + 2 * K * FP32 * mag)


# ------------------------------------------------------------ router ------

def _check_router(cuda_lib, logits, k, renorm, seed=0):
    ids, w = cuda_lib.hg_router_topk(logits.cuda(), k, renorm)
    l = logits.double().numpy()
    want_ids, want_w = L.router_topk(l, k, renorm)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    # exp is off by a few 2^-24 times its argument's magnitude, the sum by E of that
    E = l.shape[1]
    rel = (E + 64) * FP32
    _close(w.double().cpu().numpy(), want_w, rel * want_w + 2.0 ** -126, "weights")
    dw = _normal(seed + 1, *w.shape)
    d = cuda_lib.hg_router_topk_bwd(logits.cuda(), ids, w, dw.cuda(), renorm)
    want = L.router_topk_bwd(l, want_ids, dw.double().numpy(), renorm)
    mag = np.abs(want_w * dw.double().numpy()).sum(1, keepdims=True)
    _close(d.double().cpu().numpy(), want, 4 * rel * np.maximum(mag, 2.0 ** -100), "dlogits")
    return ids, w, d


@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 32, 8), (5, 7, 7), (9, 33, 32), (100, 160, 6),
                                   (3, 512, 8), (2, 2000, 4), (1000, 64, 2)])
@pytest.mark.parametrize("renorm", [False, True])
def test_router(cuda_lib, M, E, k, renorm):
    _check_router(cuda_lib, _normal(M + E, M, E) * 2, k, renorm)


@pytest.mark.parametrize("renorm", [False, True])
def test_router_ties_masks_and_empty_rows(cuda_lib, renorm):
    inf = float("inf")
    l = _normal(11, 40, 48)
    l[0] = 0.0                                             # all equal
    l[1] = -inf                                            # nothing open
    l[2, 3:] = -inf                                        # fewer than k open
    l[3] = -3.4028234663852886e38                          # the type's lowest value, open
    l[4, :40] = -3.4028234663852886e38
    l[5] = torch.randint(0, 3, (48,), generator=torch.Generator().manual_seed(2)).float()
    l[6] = l[6] * 40                                       # weights that underflow
    l[7, ::2] = -inf
    l[8, 47] = 100.0
    l[9, 31:33] = 9.0                                      # a tie across the warp's strides
    ids, w, d = _check_router(cuda_lib, l, 8, renorm)
    assert ids[0].tolist() == list(range(8)) and ids[1].tolist() == [-1] * 8
    assert ids[2].tolist()[3:] == [-1] * 5 and w[1].tolist() == [0] * 8
    assert float(d[1].abs().max()) == 0


@pytest.mark.parametrize("renorm", [False, True])
def test_router_nan_and_inf(cuda_lib, renorm):
    l = _normal(12, 3, 40)
    l[0, 5] = float("nan")
    l[1, 6] = float("inf")
    ids, w = cuda_lib.hg_router_topk(l.cuda(), 4, renorm)
    assert 5 not in ids[0].tolist() and ids[1, 0] == 6
    assert w[0].isnan().all() and w[1].isnan().any() and not w[2].isnan().any()
    order = torch.argsort(l[0].nan_to_num(nan=-1e30), descending=True)[:4]
    assert ids[0].tolist() == order.tolist()


@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_against_differences(cuda_lib, renorm):
    l = _normal(13, 4, 20)
    dw = _normal(14, 4, 5)
    ids, w = cuda_lib.hg_router_topk(l.cuda(), 5, renorm)
    d = cuda_lib.hg_router_topk_bwd(l.cuda(), ids, w, dw.cuda(), renorm).double().cpu().numpy()
    lf, i, h = l.double().numpy(), ids.cpu().numpy(), 1e-4
    for e in range(20):
        a, b = lf.copy(), lf.copy()
        a[:, e] += h
        b[:, e] -= h
        diff = (L.router_value(a, i, dw.double().numpy(), renorm)
                - L.router_value(b, i, dw.double().numpy(), renorm)) / (2 * h)
        # h^2 / 6 of a third derivative below 10, and FP32
        _close(d[:, e], diff, 1e-5)


# ------------------------------------------- streams, graphs, empty -------

def _every_call(hg, M, k, E, N, K, seed, stream=None):
    """One call of every operator on `stream`; the outputs."""
    F = N // 2
    logits = _normal(seed, M, E).cuda()
    x = _normal(seed + 1, M, K).to(torch.bfloat16).cuda()
    place = torch.from_numpy(_place(M, E, k, seed)).cuda()
    rows = _normal(seed + 2, M * k, K).to(torch.bfloat16).cuda()
    z = _normal(seed + 3, M * k, 2 * F).to(torch.bfloat16).cuda()
    dh = _normal(seed + 4, M * k, F).to(torch.bfloat16).cuda()
    dw = _normal(seed + 5, M, k).cuda()
    w, ws = [t.cuda() for t in make_weights(E, N, K, seed=seed)]
    torch.cuda.synchronize()

    def calls():
        ids, wt = hg.hg_router_topk(logits, k, True, stream=stream)
        out = [ids, wt, hg.hg_router_topk_bwd(logits, ids, wt, dw, False, stream=stream)]
        out.append(hg.hg_dispatch_tokens(x, k, place, wt, stream=stream))
        out += hg.hg_dispatch_tokens_bwd(rows, k, place, wt, x, stream=stream)
        out += hg.hg_combine_topk_bwd(x, rows, place, wt, stream=stream)
        q = hg.hg_swiglu_quantize(z, True, stream=stream)
        out += [*q, hg.hg_swiglu_bwd(dh, q[2], q[3], stream=stream)]
        out.append(hg.hg_expert_matvec(x, ids, w, ws, stream=stream))
        out.append(hg.hg_expert_matvec_swiglu(x, ids, w, ws, stream=stream))
        return out
    return calls


def test_other_stream_and_graph(cuda_lib):
    # on a stream of its own behind a long fill, and captured and replayed on a
    # graph, the results are those of the default stream
    calls = _every_call(cuda_lib, 6, 4, 16, 256, 512, 21)
    want = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    late = torch.empty(1 << 28, device="cuda")
    torch.cuda.synchronize()
    on_s = _every_call(cuda_lib, 6, 4, 16, 256, 512, 21, stream=s)
    with torch.cuda.stream(s):
        late.fill_(1.0)
    got = on_s()
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = calls()
    for t in captured:
        t.view(torch.uint8).fill_(0x55)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert cuda_lib.hg_get_device_status()[0] == cuda_lib.HG_OK


def test_empty_problems(cuda_lib):
    dev = dict(device="cuda")
    none = torch.empty(0, dtype=torch.int32, **dev)
    x0 = torch.empty(0, 64, dtype=torch.bfloat16, **dev)
    f0 = torch.empty(0, 2, **dev)
    assert cuda_lib.hg_dispatch_tokens(x0, 2, none).shape == (0, 64)
    assert cuda_lib.hg_dispatch_tokens_bwd(x0, 2, none, f0, x0)[0].shape == (0, 64)
    assert cuda_lib.hg_combine_topk_bwd(x0, x0, none, f0)[1].shape == (0, 2)
    z0 = torch.empty(0, 256, dtype=torch.bfloat16, **dev)
    a, s, q, qs = cuda_lib.hg_swiglu_quantize(z0, True)
    assert a.shape == (0, 128) and qs.shape == (0, 2)
    assert cuda_lib.hg_swiglu_bwd(z0[:, :128].contiguous(), q, qs).shape == (0, 256)
    w, ws = [t.cuda() for t in make_weights(2, 16, 128, seed=1)]
    ids0 = torch.empty(0, 2, dtype=torch.int32, **dev)
    x0 = torch.empty(0, 128, dtype=torch.bfloat16, **dev)
    assert cuda_lib.hg_expert_matvec(x0, ids0, w, ws).shape == (0, 16)
    l0 = torch.empty(0, 4, **dev)
    ids, wt = cuda_lib.hg_router_topk(l0, 2)
    assert cuda_lib.hg_router_topk_bwd(l0, ids, wt, wt).shape == (0, 4)


def test_calls_back_to_back_see_each_others_results(cuda_lib):
    # each call may be launched while the one before drains: a chain of calls on
    # shared buffers, with inputs that change from pass to pass and nothing
    # waited for, gives what the same calls give with a wait after each
    hg = cuda_lib
    M, k, E, D, F = 8, 2, 8, 512, 256
    gu = [t.cuda() for t in make_weights(E, 2 * F, D, seed=5)]
    dn = [t.cuda() for t in make_weights(E, D, F, seed=6)]
    xs = [_normal(30 + i, M, D).to(torch.bfloat16).cuda() for i in range(3)]
    ls = [_normal(40 + i, M, E).cuda() for i in range(3)]
    slots = torch.arange(M * k, dtype=torch.int32, device="cuda")
    buf = dict(x=torch.empty_like(xs[0]), l=torch.empty_like(ls[0]),
               ids=torch.empty(M, k, dtype=torch.int32, device="cuda"),
               w=torch.empty(M, k, device="cuda"),
               h=torch.empty(M * k, F, dtype=torch.bfloat16, device="cuda"),
               y=torch.empty(M * k, D, dtype=torch.bfloat16, device="cuda"),
               o=torch.empty(M, D, dtype=torch.bfloat16, device="cuda"),
               dy=torch.empty(M * k, D, dtype=torch.bfloat16, device="cuda"),
               dw=torch.empty(M, k, device="cuda"),
               dl=torch.empty(M, E, device="cuda"),
               z=torch.empty(M * k, 2 * F, dtype=torch.bfloat16, device="cuda"),
               q=torch.empty(M * k, F, dtype=torch.uint8, device="cuda"),
               qs=torch.empty(M * k, F // 128, dtype=torch.uint8, device="cuda"),
               z8=torch.empty(M * k, 2 * F, dtype=torch.uint8, device="cuda"),
               zs=torch.empty(M * k, 2 * F // 128, dtype=torch.uint8, device="cuda"),
               dz=torch.empty(M * k, 2 * F, dtype=torch.bfloat16, device="cuda"))
    b = buf

    def chain(i, wait):
        steps = [lambda: (b["x"].copy_(xs[i]), b["l"].copy_(ls[i])),
                 lambda: hg.hg_router_topk(b["l"], k, True, b["ids"], b["w"]),
                 lambda: hg.hg_expert_matvec_swiglu(b["x"], b["ids"], *gu, out=b["h"]),
                 lambda: hg.hg_expert_matvec(b["h"], b["ids"], *dn, out=b["y"]),
                 lambda: hg.hg_combine_topk(b["y"], slots, b["w"], b["o"]),
                 lambda: hg.hg_combine_topk_bwd(b["o"], b["y"], slots, b["w"], b["dy"], b["dw"]),
                 lambda: hg.hg_router_topk_bwd(b["l"], b["ids"], b["w"], b["dw"], True, b["dl"]),
                 lambda: hg.hg_expert_matvec(b["x"], b["ids"], *gu, out=b["z"]),
                 lambda: hg.hg_swiglu_quantize(b["z"], True, b["q"], b["qs"], b["z8"], b["zs"]),
                 lambda: hg.hg_swiglu_bwd(b["h"], b["z8"], b["zs"], b["dz"]),
                 lambda: hg.hg_dispatch_tokens(b["o"], k, slots, b["w"], out=b["dy"]),
                 lambda: hg.hg_dispatch_tokens_bwd(b["dy"], k, slots, b["w"], b["o"], b["x"],
                                                   b["dw"])]
        for f in steps:
            f()
            if wait:
                torch.cuda.synchronize()
        return [b[n].clone() for n in ("h", "o", "dl", "dz", "x", "dw")]

    want = [chain(i, True) for i in range(3)]
    got = [(i % 3, chain(i % 3, False)) for i in range(30)]
    torch.cuda.synchronize()
    for i, outs in got:
        for a, w in zip(outs, want[i]):
            assert torch.equal(a, w)
