"""The gradients of the weights and of the norm where a block has more to do than it does at once:
several tiles per pair of CTAs, several groups of rows per block.  Against their float64 definitions.

Tolerances are those of test_gpu_expert_training but for dgain: a block adds up its teams' rows
one after the other, and there are at least as many teams as SMs, 152, so that a team has at most
M / 152 rows and one group more (48 rows at most, eight teams' six); the teams (8) and the parts of
up to 456 blocks by 32 warps (15 each, 5 steps more) follow, and a term has two roundings of its own.
"""
import numpy as np
import pytest
import torch

from oracle import expert_training as T
from tests.test_gpu_expert_training import (BF16, FP32, TREE, _close, _codes, _decode, _f64, _normal,
                                            _offsets)
from tests.test_gpu_expert_training_large import _bf16

pytestmark = pytest.mark.gpu


# ------------------------------------------------- gradient of the weights --

# 45 experts of 3 x 3 tiles: 405 units on some 76 pairs.  Nothing, one row, MMAs of 16 and stages
# of 128 rows just missed, met and passed, accumulators of 512 rows passed once and twice
COUNTS = [0, 1, 15, 16, 17, 127, 129, 513, 1100] * 5
N, K = 520, 768


def _operands(x):
    rows = sum(COUNTS)
    dy = _normal(1, rows, N).bfloat16()
    if x == "fp8":
        a, s = _codes(2, rows, K, 120, 130)
        return dy, (a.cuda(), s.cuda()), _decode(a, s)
    xb = _normal(2, rows, K).bfloat16()
    return dy, (xb.cuda(),), _f64(xb)


def _call(hg, x):
    return hg.hg_grouped_wgrad_fp8 if x == "fp8" else hg.hg_grouped_wgrad


@pytest.mark.parametrize("x", ["bf16", "fp8"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_wgrad_many_tiles_a_pair(cuda_lib, x, out):
    hg = cuda_lib
    dy, args, xv = _operands(x)
    got = _call(hg, x)(dy.cuda(), *args, _offsets(COUNTS).cuda(), dtype=out)
    want, mag = T.wgrad(_f64(dy), xv, _offsets(COUNTS).tolist())
    n = np.array(COUNTS)[:, None, None]
    _close(_f64(got), want, 2 * (n + 1) * FP32 * mag +
           (BF16 * np.abs(want) + 2.0 ** -134 if out == torch.bfloat16 else 0.0))
    assert hg.hg_get_device_status()[0] == hg.HG_OK


@pytest.mark.parametrize("x", ["bf16", "fp8"])
def test_wgrad_accumulates_over_many_tiles_a_pair(cuda_lib, x):
    hg = cuda_lib
    dy, args, xv = _operands(x)
    start = _normal(3, len(COUNTS), N, K)
    dw = start.cuda()
    _call(hg, x)(dy.cuda(), *args, _offsets(COUNTS).cuda(), dw=dw, accumulate=True)
    want, mag = T.wgrad(_f64(dy), xv, _offsets(COUNTS).tolist(), _f64(start))
    n = np.array(COUNTS)[:, None, None]
    _close(_f64(dw), want, 2 * (n + 2) * FP32 * mag)      # mag counts what was there
    assert torch.equal(dw[::9].cpu(), start[::9])         # the experts without rows
    assert hg.hg_get_device_status()[0] == hg.HG_OK


# -------------------------------------------------- gradient of the norm ----

def _dgain_bound(M, mag):
    return (M / 152 + 48 + 8 + 15 + 5 + 2) * FP32 * mag


# rows of a group of their own, three and twenty groups a block; several rows a team, the last
# group of some of them; teams of one, two, eight and sixteen warps
@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("M,D", [(1500, 6144), (30000, 128), (9001, 264), (2001, 4096),
                                 (5003, 1024), (3000, 8200)])
def test_rmsnorm_bwd_many_groups_a_block(cuda_lib, M, D, dsum):
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
    _close(_f64(dg), wg, _dgain_bound(M, mg), "dgain")
    assert hg.hg_get_device_status()[0] == hg.HG_OK


@pytest.mark.parametrize("M,D", [(1501, 2176), (1500, 6144), (9001, 264)])
def test_rmsnorm_bwd_many_groups_in_place(cuda_lib, M, D):
    hg = cuda_lib
    dy, s, ds = (_normal(i, M, D).bfloat16().cuda() for i in range(3))
    gain, r = _normal(3, D).bfloat16().cuda(), _normal(4, M).abs().cuda()
    want = hg.hg_rmsnorm_bwd(dy, s, gain, r, dsum=ds)
    for name in ("dy", "summed", "dsum"):
        t = {"dy": dy.clone(), "summed": s.clone(), "dsum": ds.clone()}
        got = hg.hg_rmsnorm_bwd(t["dy"], t["summed"], gain, r, dsum=t["dsum"], dx=t[name])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_norm_gradient_beyond_32_bits(cuda_lib):
    """Every row counts in dgain: all terms are positive, and a group is a thousandth of a sum."""
    hg = cuda_lib
    M, D = 280_000, 8192                                  # 2.3e9 elements
    dy, s, gain = _bf16(1, M, D).abs_(), _bf16(2, M, D).abs_(), _bf16(3, D)
    r = torch.empty(M, device="cuda")
    want = torch.zeros(D, dtype=torch.float64, device="cuda")
    for at in range(0, M, 20_000):
        rows = slice(at, at + 20_000)
        sd = s[rows].double()
        r[rows] = (1 / torch.sqrt(sd.square().mean(1) + 1e-6)).float()
        want += (dy[rows].double() * sd * r[rows].double()[:, None]).sum(0)
    dx, dgain = hg.hg_rmsnorm_bwd(dy, s, gain, r)
    want = want.cpu().numpy()
    _close(_f64(dgain), want, _dgain_bound(M, want))
    for rows in (slice(0, 50), slice(M // 2, M // 2 + 50), slice(M - 50, M)):
        wx, _, mx, _ = T.rmsnorm_bwd(_f64(dy[rows]), _f64(s[rows]), _f64(gain), _f64(r[rows]))
        _close(_f64(dx[rows]), wx, BF16 * np.abs(wx) + (TREE + 8 * FP32) * mx)


# -------------------------------------------------- waits that give up -------

def _survives(hg, call, roles):
    """Whether or not a limit of a microsecond runs out on copies that are on their way, the status
    says so, and the next call is right."""
    hg.hg_get_device_status()
    want = call()
    assert hg.hg_get_device_status()[0] == hg.HG_OK
    cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        try:
            hg.lib.hg_set_wait_timeout_us(1)
            cold.fill_(1)                                 # the inputs leave L2
            got = call()
            status, detail = hg.hg_get_device_status()
        finally:
            hg.lib.hg_set_wait_timeout_us(0)
        if status == hg.HG_OK:
            assert all(torch.equal(g, w) for g, w in zip(got, want))
        else:
            assert status == hg.HG_ERR_TIMEOUT and detail >> 24 in roles
        assert all(torch.equal(g, w) for g, w in zip(call(), want))
        assert hg.hg_get_device_status()[0] == hg.HG_OK


@pytest.mark.parametrize("x", ["bf16", "fp8"])
@pytest.mark.parametrize("counts,N,K", [([3], 64, 128), ([700, 0, 129, 2000], 520, 768),
                                        (COUNTS, 520, 768), ([9000], 256, 512)])
def test_wgrad_survives_a_wait_limit_of_a_microsecond(cuda_lib, counts, N, K, x):
    hg = cuda_lib
    dy, off = _normal(1, sum(counts), N).bfloat16().cuda(), _offsets(counts).cuda()
    if x == "fp8":
        args = [t.cuda() for t in _codes(2, sum(counts), K, 120, 130)]
    else:
        args = [_normal(2, sum(counts), K).bfloat16().cuda()]
    # the producer's, the issuer's, the epilogue's and the clearing warp's waits
    _survives(hg, lambda: (_call(hg, x)(dy, *args, off),), (1, 3, 4, 9))


@pytest.mark.parametrize("M,D", [(3, 6144), (9001, 264), (1500, 6144), (400, 16384)])
def test_rmsnorm_bwd_survives_a_wait_limit_of_a_microsecond(cuda_lib, M, D):
    hg = cuda_lib
    dy, s, ds = (_normal(i, M, D).bfloat16().cuda() for i in range(3))
    gain, r = _normal(3, D).bfloat16().cuda(), _normal(4, M).abs().cuda()
    _survives(hg, lambda: hg.hg_rmsnorm_bwd(dy, s, gain, r, dsum=ds), (10,))
