"""The operators that training the experts adds, on the GPU against their float64 definitions:
the gradient of the weights, weights to MXFP4 and back, the RMS norm with its gradient, 8-bit
rows into expert order.

Tolerances, fixed before the first run:

* BF16 has 8 significant bits, so one rounding is off by at most 2^-8 of the value (2^-134 in
  the subnormal range).
* An FP32 sum of n terms in any order is off by at most (n - 1) * 2^-24 of the sum of the
  terms' magnitudes (to first order); tensor-core sums may cut instead of rounding: twice that.
  Products of two BF16 are exact in FP32.
* The norm's sums are trees: a lane adds up at most 32 terms, 5 steps join a warp and 15 the
  warps of a team, so that 52 roundings meet a term, and half as many 1 / sqrt(sum).
* E4M3 rounding is off by at most 2^-4 of the value, or 2^-10 of the scale below 2^-6 of it.
"""
import numpy as np
import pytest
import torch

from oracle import expert_training as T
from oracle.formats import E4M3_TABLE, E8M0_TABLE, bf16_bits_to_f64

pytestmark = pytest.mark.gpu

BF16, FP32 = 2.0 ** -8, 2.0 ** -24
TREE = 52 * FP32


def _f64(t):
    if t.dtype == torch.float32:
        return t.cpu().numpy().astype(np.float64)
    return bf16_bits_to_f64(t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))


def _normal(seed, *shape):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g)


def _close(got, want, bound, what=""):
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - want) <= bound) | (np.isnan(got) & np.isnan(want)) | (got == want))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           got[bad][:3], want[bad][:3])


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


def _codes(seed, rows, K, lo=0, hi=255):
    """Random E4M3 codes without NaN and E8M0 codes in [lo, hi)."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256, (rows, K)).astype(np.uint8)
    c[(c & 0x7F) == 0x7F] -= 1
    return torch.from_numpy(c), torch.from_numpy(rng.integers(lo, hi, (rows, K // 128))
                                                 .astype(np.uint8))


def _decode(codes, scale):
    return E4M3_TABLE[codes.numpy()] * np.repeat(E8M0_TABLE[scale.numpy()], 128, axis=1)


# ------------------------------------------------- gradient of the weights --

# (rows of the experts, N, K): one row; stages of 128 rows and MMAs of 16 just missed and just
# passed; experts without rows at either end and in the middle; one column block; tiles of 256
# missed and passed; an expert of more than one chunk of 512 rows; rows that are cut into parts
WGRAD = [([1], 8, 128), ([0], 264, 128), ([0, 5, 0, 0, 17, 0], 72, 256), ([64], 256, 256),
         ([63, 65, 16, 15], 264, 384), ([1, 127, 128, 129], 520, 128), ([512, 513], 248, 640),
         ([1300, 3, 700], 136, 256), ([4200], 200, 384), ([8200, 90], 64, 128)]


@pytest.mark.parametrize("x", ["bf16", "fp8"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,N,K", WGRAD)
def test_wgrad(cuda_lib, counts, N, K, out, x):
    hg = cuda_lib
    if x == "bf16":
        K -= 56                                           # no multiple of 16 is needed
    rows, spare = sum(counts), 70                         # rows behind the last expert's
    off = _offsets(counts)
    dy = _normal(N + K, rows + spare, N).bfloat16()
    dy[rows:] = float("nan")
    if x == "fp8":
        a, s = _codes(N, rows + spare, K, 110, 140)
        s[rows:] = 255
        xv = _decode(a, s)
        got = hg.hg_grouped_wgrad_fp8(dy.cuda(), a.cuda(), s.cuda(), off.cuda(), dtype=out)
    else:
        xb = _normal(N, rows + spare, K).bfloat16()
        xb[rows:] = float("inf")
        xv = _f64(xb)
        got = hg.hg_grouped_wgrad(dy.cuda(), xb.cuda(), off.cuda(), dtype=out)
    want, mag = T.wgrad(_f64(dy[:rows]), xv[:rows], off.tolist())
    assert got.dtype == out
    n = np.array(counts)[:, None, None]
    _close(_f64(got), want, 2 * (n + 1) * FP32 * mag +
           (BF16 * np.abs(want) + 2.0 ** -134 if out == torch.bfloat16 else 0.0))
    assert hg.hg_get_device_status()[0] == hg.HG_OK


@pytest.mark.parametrize("counts,N,K", [([3, 0, 70], 40, 128), ([4130], 256, 128)])
@pytest.mark.parametrize("x", ["bf16", "fp8"])
def test_wgrad_accumulates(cuda_lib, counts, N, K, x):
    hg = cuda_lib
    rows, off = sum(counts), _offsets(counts)
    dy, start = _normal(1, rows, N).bfloat16(), _normal(2, len(counts), N, K)
    dw = start.cuda()
    if x == "fp8":
        a, s = _codes(3, rows, K, 120, 130)
        xv, args, f = _decode(a, s), (a.cuda(), s.cuda()), hg.hg_grouped_wgrad_fp8
    else:
        xb = _normal(3, rows, K).bfloat16()
        xv, args, f = _f64(xb), (xb.cuda(),), hg.hg_grouped_wgrad
    back = f(dy.cuda(), *args, off.cuda(), dw=dw, accumulate=True)
    assert back is dw
    f(dy.cuda(), *args, off.cuda(), dw=dw, accumulate=True)
    once, mag = T.wgrad(_f64(dy), xv, off.tolist())
    n = np.array(counts)[:, None, None]
    want = 2 * once + _f64(start)
    _close(_f64(dw), want, 2 * (2 * n + 3) * FP32 * (2 * mag + np.abs(_f64(start))))
    empty = [e for e, c in enumerate(counts) if c == 0]
    assert torch.equal(dw[empty].cpu(), start[empty])


def test_wgrad_neighbours_do_not_mix(cuda_lib):
    """An expert whose rows are Inf and NaN, between others, in the same stages and MMAs."""
    hg = cuda_lib
    counts, N, K = [5, 3, 6, 50], 16, 128
    rows, off = sum(counts), _offsets(counts)
    for what in ("dy", "x"):
        dy, x = _normal(4, rows, N).bfloat16(), _normal(5, rows, K).bfloat16()
        (dy if what == "dy" else x)[5:8] = torch.tensor([float("inf"), float("nan"), -3e38]
                                                         ).bfloat16()[:, None]
        got = _f64(hg.hg_grouped_wgrad(dy.cuda(), x.cuda(), off.cuda()))
        assert not np.isfinite(got[1]).any()
        with np.errstate(invalid="ignore"):
            want, mag = T.wgrad(_f64(dy), _f64(x), off.tolist())
        for e in (0, 2, 3):
            _close(got[e], want[e], 2 * (counts[e] + 1) * FP32 * mag[e])


def test_wgrad_fp8_every_code_and_scale(cuda_lib):
    """One row: dw is the row itself, every code under every scale that BF16 holds."""
    hg = cuda_lib
    K = 256
    row = torch.arange(K, dtype=torch.uint8)              # NaN among them
    off, dy = _offsets([1]).cuda(), torch.zeros(1, 8).bfloat16()
    dy[0, 0] = 1.0
    for scale in (0, 1, 9, 10, 60, 126, 127, 128, 133, 134, 135, 136, 200, 245, 246, 255):
        s = torch.full((1, K // 128), scale, dtype=torch.uint8)
        got = _f64(hg.hg_grouped_wgrad_fp8(dy.cuda(), row[None].cuda(), s.cuda(), off))[0, 0]
        want = _decode(row[None], s)[0]
        # FP32's subnormal numbers may count as zero in the tensor core
        _close(got, want, np.where(np.abs(want) < 2.0 ** -126, 2.0 ** -126, 0.0), scale)


def test_wgrad_repeats_bit_for_bit(cuda_lib):
    hg = cuda_lib
    for counts, N, K in (([700, 20, 1100], 264, 520), ([4150], 128, 256)):
        dy, x = _normal(1, sum(counts), N).bfloat16().cuda(), _normal(2, sum(counts), K).bfloat16()
        off, x = _offsets(counts).cuda(), x.cuda()
        first = hg.hg_grouped_wgrad(dy, x, off)
        for _ in range(3):
            assert torch.equal(hg.hg_grouped_wgrad(dy, x, off), first)


def test_wgrad_bad_offsets(cuda_lib):
    hg = cuda_lib
    rows, N, K = 100, 64, 128
    dy, x = _normal(1, rows, N).bfloat16(), _normal(2, rows, K).bfloat16()
    a, s = _codes(3, rows, K, 120, 130)
    assert hg.hg_get_device_status()[0] == hg.HG_OK
    for off in ([0, 40, 20, 100], [0, 40, 101, 100], [-1, 40, 60, 100], [0, 90, 20, 19],
                [0, 2 ** 31 - 1, -2 ** 31, 100]):
        at = torch.tensor(off, dtype=torch.int32).cuda()
        for call, xv in ((lambda: hg.hg_grouped_wgrad(dy.cuda(), x.cuda(), at), _f64(x)),
                         (lambda: hg.hg_grouped_wgrad_fp8(dy.cuda(), a.cuda(), s.cuda(), at),
                          _decode(a, s))):
            dw = call()
            want, mag = T.wgrad(_f64(dy), xv, off)
            _close(_f64(dw), want, 2 * (rows + 1) * FP32 * mag, off)
            assert hg.hg_get_device_status()[0] == hg.HG_ERR_BAD_OFFSETS


def test_wgrad_no_rows(cuda_lib):
    hg = cuda_lib
    off = torch.zeros(4, dtype=torch.int32).cuda()
    dy, x = torch.empty(0, 72).bfloat16().cuda(), torch.empty(0, 264).bfloat16().cuda()
    assert (hg.hg_grouped_wgrad(dy, x, off) == 0).all()
    dw = torch.full((3, 72, 264), 2.0).cuda()
    assert (hg.hg_grouped_wgrad(dy, x, off, dw=dw, accumulate=True) == 2).all()


def test_wgrad_leaves_its_surroundings(cuda_lib):
    """dw inside a larger buffer: nothing around it changes, whatever the tiles' edges."""
    hg = cuda_lib
    for dtype in (torch.float32, torch.bfloat16):
        E, N, K, pad = 2, 40, 72, 64
        buf = torch.full((E * N * K + 2 * pad,), 7.0, dtype=dtype).cuda()
        dw = buf[pad:-pad].view(E, N, K)
        dy, x = _normal(1, 30, N).bfloat16().cuda(), _normal(2, 30, K).bfloat16().cuda()
        hg.hg_grouped_wgrad(dy, x, _offsets([10, 20]).cuda(), dw=dw)
        assert (buf[:pad] == 7).all() and (buf[-pad:] == 7).all() and (dw != 7).any()


# ---------------------------------------------------------- 4-bit weights --

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,N,K", [(1, 1, 32), (1, 32, 32), (3, 33, 96), (2, 160, 96), (1, 128, 128),
                                   (2, 128, 256), (1, 288, 544), (5, 64, 64), (1, 480, 640)])
def test_quantize_weights(cuda_lib, E, N, K, dtype):
    hg = cuda_lib
    w = (_normal(N + K, E, N, K) * torch.exp(3 * _normal(3, E, 1, K))).to(dtype)
    w[0, 0, :32] = 0                                       # a group of zeros
    both = N % 32 == 0
    got = hg.hg_quantize_weights(w.cuda(), transposed=both)
    q, s = T.quantize_weights(_f64(w))
    assert (got[0].cpu().numpy() == q).all() and (got[1].cpu().numpy() == s).all()
    if both:
        q, s = T.quantize_weights(np.ascontiguousarray(_f64(w).transpose(0, 2, 1)))
        assert (got[2].cpu().numpy() == q).all() and (got[3].cpu().numpy() == s).all()
        alone = hg.hg_quantize_weights(w.cuda())
        assert torch.equal(alone[0], got[0]) and torch.equal(alone[1], got[1])
        assert alone[2] is None and alone[3] is None
    for out in (torch.float32, torch.bfloat16):
        back = hg.hg_dequantize_weights(got[0], got[1], dtype=out)
        want = T.dequantize_weights(got[0].cpu().numpy(), got[1].cpu().numpy())
        assert back.dtype == out and (_f64(back) == want).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_weights_ends_of_the_range(cuda_lib, dtype):
    """Ties, the scale's borders, subnormal and largest numbers, Inf and NaN, each a group."""
    hg = cuda_lib
    big = torch.finfo(dtype).max
    rows = []
    for e in (-149, -133, -130, -127, -126, -120, -1, 0, 1, 100, 125):
        for m in (1.0, 1.5, 1.5078125, 1.9921875):
            rows.append([m * 2.0 ** e, -0.75 / 6 * m * 2.0 ** e, 0.0, -0.0] + [2.0 ** e / 64] * 28)
    ties = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0]
    rows += [ties + [0.0] * 17, [big] * 32, [-big] + [1.0] * 31]
    bad = len(rows)
    rows += [[v] + [1.0] * 31 for v in (float("inf"), -float("inf"), float("nan"))]
    rows += [[0.0] * 32] * (-len(rows) % 32)
    w = torch.tensor(rows, dtype=torch.float64).to(dtype)
    q, s = T.quantize_weights(_f64(w)[None])
    qt, st = T.quantize_weights(np.ascontiguousarray(_f64(w).T)[None])
    got = hg.hg_quantize_weights(w[None].contiguous().cuda(), transposed=True)
    assert (got[1].cpu().numpy() == s).all() and (got[3].cpu().numpy() == st).all()
    assert (got[0].cpu().numpy() == q).all() and (got[2].cpu().numpy() == qt).all()
    assert (s[0, bad:bad + 3] == 255).all()
    back = _f64(hg.hg_dequantize_weights(got[0], got[1], dtype=dtype))
    want = T.dequantize_weights(q, s)
    want[np.abs(want) > big] = np.sign(want[np.abs(want) > big]) * np.inf
    _close(back, want, 0.0)


def test_dequantize_every_scale(cuda_lib):
    hg = cuda_lib
    codes = torch.arange(256, dtype=torch.uint8).view(256, 1, 1).expand(256, 1, 16).contiguous()
    scale = torch.arange(256, dtype=torch.uint8).view(256, 1, 1).contiguous()
    for dtype in (torch.float32, torch.bfloat16):
        got = _f64(hg.hg_dequantize_weights(codes.cuda(), scale.cuda(), dtype=dtype))
        want = T.dequantize_weights(codes.numpy(), scale.numpy())
        want[np.abs(want) > torch.finfo(dtype).max] *= np.inf
        _close(got, want, 0.0)


def test_quantized_weights_feed_the_gemm(cuda_lib):
    """The GEMM on quantised weights is the product with what dequantisation gives."""
    from oracle.formats import decode_e4m3, decode_e8m0
    hg = cuda_lib
    E, N, K, counts = 2, 128, 256, [30, 9]
    w = _normal(1, E, N, K) / 16
    q, s, qt, st = hg.hg_quantize_weights(w.cuda(), transposed=True)
    x = _normal(2, sum(counts), K).bfloat16().cuda()
    a, sc = hg.hg_quantize_scatter_acts(x, 1, torch.arange(sum(counts), dtype=torch.int32).cuda())
    out = _f64(hg.hg_grouped_w4a8_gemm(a, sc, q, s, _offsets(counts).cuda()))
    xv = decode_e4m3(a.cpu().numpy()) * np.repeat(decode_e8m0(sc.cpu().numpy()), 128, axis=1)
    wv = _f64(hg.hg_dequantize_weights(q, s, dtype=torch.float32))
    off = _offsets(counts).tolist()
    for e in range(E):
        at = slice(off[e], off[e + 1])
        want, mag = xv[at] @ wv[e].T, np.abs(xv[at]) @ np.abs(wv[e]).T
        _close(out[at], want, BF16 * np.abs(want) + 2 * K * FP32 * mag)
    back = _f64(hg.hg_dequantize_weights(qt, st, dtype=torch.float32)).transpose(0, 2, 1)
    assert np.abs(back - _f64(w)).max() <= np.abs(_f64(w)).max() / 6      # both stand for w


# ------------------------------------------------------------------- norm --

def _check_norm(hg, x, residual, gain, eps, D, codes=True):
    want_s, want_r, want_v = T.rmsnorm(_f64(x), None if residual is None else _f64(residual),
                                       _f64(gain), eps)
    y, a, sc, s, r = hg.hg_rmsnorm_quantize(
        x.cuda(), gain.cuda(), residual=None if residual is None else residual.cuda(), eps=eps,
        codes=codes)
    if residual is None:
        assert s is None
    else:
        _close(_f64(s), want_s, 0.0, "sum")
    rel = (52 / 2 + 5) * FP32
    _close(_f64(r), want_r, rel * want_r + 2.0 ** -149, "rstd")
    mag = np.abs(want_v)
    _close(_f64(y), want_v, (BF16 + 2 * rel) * mag + 2.0 ** -133, "y")
    if not codes:
        assert a is None and sc is None
        return
    sc = sc.cpu().numpy()
    assert sc.shape == (len(mag), D // 128)
    if len(mag) == 0:
        return
    # v is FP32: its two products round to multiples of 2^-149 below 2^-126, so that each is off
    # by up to 2^-150 there (the first times a gain below 2 in these tests)
    tiny = 2.0 ** -148
    low = np.maximum(mag * (1 - 2 * rel) - tiny, 0.0)
    lo, hi = T.quantize_rows_f64(low)[1], T.quantize_rows_f64(mag * (1 + 2 * rel) + tiny)[1]
    gone = low.reshape(*sc.shape, 128).max(-1) == 0       # may be zeros, whose scale is 1
    assert ((sc == lo) | (sc == hi) | (gone & ((sc <= hi) | (sc == 127)))).all()
    value = np.repeat(E8M0_TABLE[sc], 128, axis=1)
    got = E4M3_TABLE[a.cpu().numpy()] * value
    fine = np.isfinite(value)
    _close(got[fine], want_v[fine],
           ((2.0 ** -4 + 4 * rel) * mag + 2.0 ** -10 * value + tiny)[fine], "codes")
    assert (a.cpu().numpy()[~fine] == 0x7F).all()


# one token; teams of 1, 2, 4, 8 and 16 warps; pieces that do not fill the team; the widest row
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,D", [(1, 128), (1, 6144), (3, 1024), (9, 1152), (5, 2048), (33, 2176),
                                 (7, 4096), (2, 5120), (3, 8192), (2, 8320), (2, 16384), (0, 256)])
def test_rmsnorm(cuda_lib, M, D, residual):
    x = _normal(M + D, M, D).bfloat16()
    res = (3 * _normal(1, M, D)).bfloat16() if residual else None
    _check_norm(cuda_lib, x, res, (1 + 0.2 * _normal(2, D)).bfloat16(), 1e-6, D)


@pytest.mark.parametrize("M,D", [(3, 8), (2, 24), (5, 264), (2, 1000), (3, 4104), (1, 16376)])
def test_rmsnorm_without_codes_takes_any_eight(cuda_lib, M, D):
    x, gain = _normal(M, M, D).bfloat16(), _normal(2, D).bfloat16()
    _check_norm(cuda_lib, x, None, gain, 1e-5, D, codes=False)
    _check_norm(cuda_lib, x, (2 * x.float()).bfloat16(), gain, 1e-5, D, codes=False)


def test_rmsnorm_ends_of_the_range(cuda_lib):
    """Rows whose squares pass FP32's range, vanish in it, or are not finite."""
    for D in (128, 1152, 6144, 16384):
        x = _normal(5, 9, D)
        for m, scale in enumerate((1e37, 3e17, 1e19, 1e-20, 1e-38, 1e-40, 0.0)):
            x[m] *= scale
        x = x.bfloat16()
        x[7, D // 2] = float("inf")
        x[8, 3] = float("nan")
        for eps in (1e-30, 1e-6, 1e30):
            _check_norm(cuda_lib, x, None, (1 + 0.2 * _normal(2, D)).bfloat16(), eps, D)
            _check_norm(cuda_lib, x, (x.float() / 2).bfloat16(), torch.ones(D).bfloat16(), eps, D)
        big = torch.full((2, D), 3.3e38).bfloat16()
        _check_norm(cuda_lib, big, None, torch.ones(D).bfloat16(), 1e-6, D)


def test_rmsnorm_in_place(cuda_lib):
    hg = cuda_lib
    for M, D in ((4, 256), (2, 6144)):
        x, res = _normal(1, M, D).bfloat16().cuda(), _normal(2, M, D).bfloat16().cuda()
        gain = _normal(3, D).bfloat16().cuda()
        want = hg.hg_rmsnorm_quantize(x, gain, residual=res)
        for name in ("x", "residual"):
            a, b = x.clone(), res.clone()
            into = a if name == "x" else b
            other = {} if name == "x" else {"y": a}
            got = hg.hg_rmsnorm_quantize(a, gain, residual=b, summed=into, **other)
            assert got[3] is into
            for g, w in zip(got, want):
                assert torch.equal(g, w)
        huge = torch.full((M, D), 2e38).bfloat16().cuda()    # the wide way reads s again
        want = hg.hg_rmsnorm_quantize(huge, gain, residual=-huge / 2)
        a = huge.clone()
        got = hg.hg_rmsnorm_quantize(a, gain, residual=-huge / 2, summed=a)
        for g, w in zip(got, want):
            assert torch.equal(g, w)


@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("M,D", [(1, 8), (1, 6144), (7, 264), (40, 128), (2500, 128), (700, 1152),
                                 (333, 6144), (2, 8200), (3, 16384), (0, 128)])
def test_rmsnorm_bwd(cuda_lib, M, D, dsum):
    hg = cuda_lib
    dy, s = _normal(1, M, D).bfloat16(), (3 * _normal(2, M, D)).bfloat16()
    gain = (1 + 0.2 * _normal(3, D)).bfloat16()
    r = (1 / torch.sqrt(s.double().square().mean(1) + 1e-6)).float()
    ds = _normal(4, M, D).bfloat16() if dsum else None
    dx, dg = hg.hg_rmsnorm_bwd(dy.cuda(), s.cuda(), gain.cuda(), r.cuda(),
                               dsum=None if ds is None else ds.cuda())
    wx, wg, mx, mg = T.rmsnorm_bwd(_f64(dy), _f64(s), _f64(gain), _f64(r),
                                   None if ds is None else _f64(ds))
    _close(_f64(dx), wx, BF16 * np.abs(wx) + (TREE + 8 * FP32) * mx, "dx")
    _close(_f64(dg), wg, (M + 4) * FP32 * mg, "dgain")
    only, none = hg.hg_rmsnorm_bwd(dy.cuda(), s.cuda(), gain.cuda(), r.cuda(),
                                   dsum=None if ds is None else ds.cuda(), want_dgain=False)
    assert none is None and torch.equal(only, dx)
    again, dg2 = hg.hg_rmsnorm_bwd(dy.cuda(), s.cuda(), gain.cuda(), r.cuda(),
                                   dsum=None if ds is None else ds.cuda())
    assert torch.equal(again, dx) and torch.equal(dg2, dg)


def test_rmsnorm_bwd_in_place(cuda_lib):
    hg = cuda_lib
    M, D = 30, 2176
    dy, s, ds = (_normal(i, M, D).bfloat16().cuda() for i in range(3))
    gain, r = _normal(3, D).bfloat16().cuda(), _normal(4, M).abs().cuda()
    want = hg.hg_rmsnorm_bwd(dy, s, gain, r, dsum=ds)
    for name in ("dy", "summed", "dsum"):
        t = {"dy": dy.clone(), "summed": s.clone(), "dsum": ds.clone()}
        got = hg.hg_rmsnorm_bwd(t["dy"], t["summed"], gain, r, dsum=t["dsum"], dx=t[name])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rmsnorm_gradient_by_differences(cuda_lib):
    """Along random directions: the norm's own outputs, FP32-exact inputs of wide steps."""
    hg = cuda_lib
    M, D, eps, step = 4, 256, 1e-6, 2.0 ** -6
    s, dy = _normal(1, M, D).bfloat16(), _normal(2, M, D).bfloat16()
    gain = (1 + 0.2 * _normal(3, D)).bfloat16()
    _, _, _, _, r = hg.hg_rmsnorm_quantize(s.cuda(), gain.cuda(), eps=eps)
    dx, dg = hg.hg_rmsnorm_bwd(dy.cuda(), s.cuda(), gain.cuda(), r)
    d = _f64((_normal(4, M, D)).bfloat16())
    loss = lambda x, g: (T.rmsnorm(x, None, g, eps)[2] * _f64(dy)).sum()      # noqa: E731
    g = _f64(gain)
    diff = (loss(_f64(s) + step * d, g) - loss(_f64(s) - step * d, g)) / (2 * step)
    # third derivatives times step^2, and BF16's rounding of dx
    assert abs((_f64(dx) * d).sum() - diff) <= step ** 2 * np.abs(_f64(dy)).sum() + \
        BF16 * (np.abs(_f64(dx)) * np.abs(d)).sum()
    e = _f64(_normal(5, D).bfloat16())
    diff = (loss(_f64(s), g + e) - loss(_f64(s), g - e)) / 2                  # linear in gain
    assert abs((_f64(dg) * e).sum() - diff) <= 1e-5 * np.abs(_f64(dg) * e).sum() + 1e-4


# ------------------------------------------------------------ 8-bit rows --

@pytest.mark.parametrize("M,K,k,drop", [(1, 128, 1, 0), (13, 2048, 8, 5), (7, 16384, 3, 4),
                                        (5, 16512, 2, 0), (3, 40960, 40, 30), (300, 384, 8, 100),
                                        (0, 128, 2, 0)])
def test_dispatch_acts(cuda_lib, M, K, k, drop):
    hg = cuda_lib
    rng = np.random.default_rng(M + K)
    place = rng.permutation(M * k).astype(np.int32)
    place[rng.permutation(M * k)[:drop]] = np.array([-1, M * k, 2 ** 31 - 1, -2 ** 31]
                                                    )[rng.integers(0, 4, drop)].astype(np.int32)
    a = torch.from_numpy(rng.integers(0, 256, (M, K)).astype(np.uint8))
    s = torch.from_numpy(rng.integers(0, 256, (M, K // 128)).astype(np.uint8))
    ra, rs = torch.full((M * k, K), 77, dtype=torch.uint8), torch.full((M * k, K // 128), 78,
                                                                        dtype=torch.uint8)
    ga, gs = hg.hg_dispatch_acts(a.cuda(), s.cuda(), k, torch.from_numpy(place).cuda(),
                                 out_fp8=ra.cuda(), out_scale=rs.cuda())
    wa, ws = T.dispatch_acts(a.numpy(), s.numpy(), place.reshape(M, k), ra.numpy(), rs.numpy())
    assert (ga.cpu().numpy() == wa).all() and (gs.cpu().numpy() == ws).all()


def test_dispatch_acts_is_the_other_half_of_the_scatter(cuda_lib):
    hg = cuda_lib
    M, K, k = 50, 1152, 4
    x = _normal(1, M, K).bfloat16().cuda()
    place = torch.randperm(M * k, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    a, s = hg.hg_quantize_scatter_acts(x, 1, torch.arange(M, dtype=torch.int32).cuda())
    got = hg.hg_dispatch_acts(a, s, k, place)
    want = hg.hg_quantize_scatter_acts(x, k, place)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------- streams and graphs ------

def _calls(hg):
    """Each call on fixed inputs, as a function of a stream, with fixed outputs."""
    M, D, k, E = 40, 256, 2, 4
    x, res = _normal(1, M, D).bfloat16().cuda(), _normal(2, M, D).bfloat16().cuda()
    gain, w = _normal(3, D).bfloat16().cuda(), _normal(4, E, 128, D).cuda()
    off = _offsets([10, 0, 25, 5]).cuda()
    long = torch.tensor([0, 4096], dtype=torch.int32).cuda()
    dy, xl = _normal(5, 4096, 64).bfloat16().cuda(), _normal(6, 4096, 128).bfloat16().cuda()
    place = torch.randperm(M * k, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    q = hg.hg_quantize_weights(w, transposed=True)
    a = hg.hg_rmsnorm_quantize(x, gain)
    return {
        "norm": lambda s=None: hg.hg_rmsnorm_quantize(x, gain, residual=res, stream=s),
        "norm bwd": lambda s=None: hg.hg_rmsnorm_bwd(x, res, gain, a[4], dsum=x, stream=s),
        "weights": lambda s=None: hg.hg_quantize_weights(w, transposed=True, stream=s),
        "back": lambda s=None: (hg.hg_dequantize_weights(q[0], q[1], stream=s),),
        "acts": lambda s=None: hg.hg_dispatch_acts(a[1], a[2], k, place, stream=s),
        "wgrad": lambda s=None: (hg.hg_grouped_wgrad(x, res, off, stream=s),),
        "wgrad fp8": lambda s=None: (hg.hg_grouped_wgrad_fp8(x, a[1], a[2], off, stream=s),),
        "wgrad split": lambda s=None: (hg.hg_grouped_wgrad(dy, xl, long, stream=s),),
    }


NAMES = ["norm", "norm bwd", "weights", "back", "acts", "wgrad", "wgrad fp8", "wgrad split"]


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream_and_in_a_graph(cuda_lib, name):
    call = _calls(cuda_lib)[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = call()
        second = call()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    for outs in (first, second):
        for g, w in zip(outs, want):
            assert torch.equal(g, w)


def test_two_streams_at_once(cuda_lib):
    """Calls that overlap, each with outputs and workspaces of its own."""
    calls = _calls(cuda_lib)
    want = {n: calls[n]() for n in NAMES}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):
        for j, s in enumerate(streams):
            for n in NAMES[j:] + NAMES[:j]:
                got.append((n, calls[n](s)))
    torch.cuda.synchronize()
    for n, outs in got:
        for g, w in zip(outs, want[n]):
            assert torch.equal(g, w), n
    assert cuda_lib.hg_get_device_status()[0] == cuda_lib.HG_OK
