"""The operators that training the experts adds where offsets pass 32 bits: the end of a large call
gives the bits of a small call on that part alone.  And the calls after hg_shutdown."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(seed, *shape):
    return torch.randn(*shape, generator=_gen(seed), device="cuda", dtype=torch.bfloat16)


def test_wgrad_dw_beyond_32_bits(cuda_lib):
    hg = cuda_lib
    E, N, K = 10, 16384, 16384                            # 2.7e9 elements of dw
    counts = [7, 0, 130, 64, 1, 20, 33, 200, 15, 50]
    off = torch.tensor([sum(counts[:e]) for e in range(E + 1)], dtype=torch.int32).cuda()
    dy, x = _bf16(1, sum(counts), N), _bf16(2, sum(counts), K)
    dw = hg.hg_grouped_wgrad(dy, x, off, dtype=torch.bfloat16)
    for e in (0, 1, 2, E - 1):
        lo, hi = int(off[e]), int(off[e + 1])
        one = torch.tensor([0, hi - lo], dtype=torch.int32).cuda()
        want = hg.hg_grouped_wgrad(dy[lo:hi].contiguous(), x[lo:hi].contiguous(), one,
                                   dtype=torch.bfloat16)[0]
        assert torch.equal(dw[e], want), e
    assert hg.hg_get_device_status()[0] == hg.HG_OK


def test_wgrad_rows_beyond_32_bits(cuda_lib):
    """Operands of more than 2^32 bytes; the last expert's rows at their end."""
    hg = cuda_lib
    rows, N, K = 300_000, 8192, 256
    dy, x = _bf16(1, rows, N), _bf16(2, rows, K)
    off = torch.tensor([rows - 700, rows - 690, rows - 690, rows], dtype=torch.int32).cuda()
    dw = hg.hg_grouped_wgrad(dy, x, off)
    tail = torch.tensor([0, 10, 10, 700], dtype=torch.int32).cuda()
    assert torch.equal(dw, hg.hg_grouped_wgrad(dy[-700:].contiguous(), x[-700:].contiguous(), tail))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weights_beyond_32_bits(cuda_lib, dtype):
    hg = cuda_lib
    E, N, K = 9, 16384, 16384
    w = torch.empty(E, N, K, dtype=dtype, device="cuda")
    for e in range(E):
        w[e] = _bf16(e, N, K)
    both = hg.hg_quantize_weights(w, transposed=True)
    alone = hg.hg_quantize_weights(w)
    last = hg.hg_quantize_weights(w[-1:].contiguous(), transposed=True)
    for i in range(4):
        assert torch.equal(both[i][-1:], last[i])
        assert i > 1 or torch.equal(alone[i], both[i])
    back = hg.hg_dequantize_weights(both[0], both[1], dtype=dtype)
    assert torch.equal(back[-1:], hg.hg_dequantize_weights(last[0], last[1], dtype=dtype))


def test_norm_beyond_32_bits(cuda_lib):
    hg = cuda_lib
    M, D = 280_000, 8192                                  # 2.3e9 elements
    x, res = _bf16(1, M, D), _bf16(2, M, D)
    gain = _bf16(3, D)
    big = hg.hg_rmsnorm_quantize(x, gain, residual=res)
    small = hg.hg_rmsnorm_quantize(x[-5:].contiguous(), gain, residual=res[-5:].contiguous())
    for b, s in zip(big, small):
        assert torch.equal(b[-5:], s)
    dx, dgain = hg.hg_rmsnorm_bwd(x, big[3], gain, big[4], dsum=res)
    sx, _ = hg.hg_rmsnorm_bwd(x[-5:].contiguous(), small[3], gain, small[4],
                              dsum=res[-5:].contiguous())
    assert torch.equal(dx[-5:], sx) and torch.isfinite(dgain).all()


def test_acts_beyond_32_bits(cuda_lib):
    hg = cuda_lib
    M, K, k = 70_000, 8192, 8                             # 4.6e9 bytes of rows
    a = torch.randint(0, 256, (M, K), generator=_gen(1), device="cuda", dtype=torch.uint8)
    s = torch.randint(0, 256, (M, K // 128), generator=_gen(2), device="cuda", dtype=torch.uint8)
    place = torch.randperm(M * k, generator=_gen(3), device="cuda").to(torch.int32)
    rows, scales = hg.hg_dispatch_acts(a, s, k, place)
    for t in (0, M // 2, M - 1):
        at = place[t * k:(t + 1) * k].long()
        assert (rows[at] == a[t]).all() and (scales[at] == s[t]).all()
    for r in (0, M * k - 1):
        src = int((place == r).nonzero()) // k
        assert torch.equal(rows[r], a[src]) and torch.equal(scales[r], s[src])


def test_calls_after_shutdown(cuda_lib):
    hg = cuda_lib
    x, res, gain = _bf16(1, 40, 256), _bf16(2, 40, 256), _bf16(3, 256)
    w, off = torch.randn(2, 128, 256, device="cuda"), torch.tensor([0, 15, 40]).int().cuda()

    def calls():
        n = hg.hg_rmsnorm_quantize(x, gain, residual=res)
        return (*n, *hg.hg_rmsnorm_bwd(x, n[3], gain, n[4]), *hg.hg_quantize_weights(w, True),
                hg.hg_grouped_wgrad(x, res, off), hg.hg_grouped_wgrad_fp8(x, n[1], n[2], off))

    before = calls()
    torch.cuda.synchronize()
    hg.hg_shutdown()
    for a, b in zip(calls(), before):
        assert torch.equal(a, b)
    assert hg.hg_get_device_status()[0] == hg.HG_OK
