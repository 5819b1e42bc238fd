"""The float64 definitions of the MoE layer's steps, checked on the CPU: gradients against
central differences, quantisation against the pinned row quantiser, the product against a
direct sum."""
import numpy as np
import pytest

from oracle import moe_io, moe_layer as L
from oracle.formats import E2M1_TABLE, bf16_bits_to_f64, round_f64_to_bf16_bits

# A central difference of step h of a function with third derivative D is off by D h^2 / 6,
# and by the rounding 2^-52 |f| / h: with h = 1e-5 and values and derivatives of order 10
# both are below 1e-8.
H, TOL = 1e-5, 1e-8


def _differences(f, x):
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += H
        b[i] -= H
        d[i] = (f(a) - f(b)) / (2 * H)
    return d


def _place(rng, M, k, drop=0):
    p = rng.permutation(M * k).astype(np.int64).reshape(M, k)
    for i in range(drop):
        p.reshape(-1)[2 * i] = -1
    return p


def test_dispatch_and_combine_gradients():
    rng = np.random.default_rng(0)
    M, k, n = 5, 3, 4
    place = _place(rng, M, k, drop=2)
    x, w = rng.standard_normal((M, n)), rng.random((M, k))
    drows = rng.standard_normal((M * k, n))
    f = lambda x, w: float((L.dispatch(x, place, w, np.zeros((M * k, n))) * drows).sum())  # noqa: E731
    assert np.abs(_differences(lambda v: f(v, w), x) - L.combine(drows, place, w)[0]).max() < TOL
    assert np.abs(_differences(lambda v: f(x, v), w) - L.row_dots(drows, x, place)[0]).max() < TOL
    y, dout = rng.standard_normal((M * k, n)), rng.standard_normal((M, n))
    f = lambda y, w: float((L.combine(y, place, w)[0] * dout).sum())  # noqa: E731
    dy = L.dispatch(dout, place, w, np.zeros((M * k, n)))
    assert np.abs(_differences(lambda v: f(v, w), y) - dy).max() < TOL
    assert np.abs(_differences(lambda v: f(y, v), w) - L.row_dots(y, dout, place)[0]).max() < TOL


def test_swiglu_gradient():
    rng = np.random.default_rng(1)
    z, dh = 3.0 * rng.standard_normal((3, 8)), rng.standard_normal((3, 4))
    d = _differences(lambda v: float((L.swiglu(v) * dh).sum()), z)
    assert np.abs(d - L.swiglu_bwd(dh, z)).max() < TOL


def test_quantize_is_the_row_quantiser():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((4, 384)) * 2.0 ** rng.integers(-30, 30, (4, 1))
    x[0, :128] = 0.0
    x[1, :128] = 448.0
    x[2, 0:128] = 2.0 ** -130
    bits = round_f64_to_bf16_bits(x)
    codes, scales = L.quantize(bf16_bits_to_f64(bits))
    rc, rs = moe_io.quantize_rows(bits)
    assert np.array_equal(codes, rc) and np.array_equal(scales, rs)


def test_expert_matvec_is_the_sum():
    rng = np.random.default_rng(3)
    E, N, K = 3, 5, 64
    w = rng.integers(0, 256, (E, N, K // 2)).astype(np.uint8)
    s = rng.integers(120, 130, (E, N, K // 32)).astype(np.uint8)
    x = rng.standard_normal((2, K))
    ids = np.array([[2, 0], [3, 1]])                     # 3 is no expert
    y, mag = L.expert_matvec(x, ids, w, s)
    for slot, e in enumerate(ids.reshape(-1)):
        for n in range(N):
            want = 0.0
            for k in range(K):
                if e < E:
                    code = (w[e, n, k // 2] >> (4 * (k % 2))) & 15
                    want += x[slot // 2, k] * E2M1_TABLE[code] * 2.0 ** (int(s[e, n, k // 32]) - 127)
            assert abs(y[slot, n] - want) <= 1e-12 * (1 + mag[slot, n])


@pytest.mark.parametrize("renorm", [False, True])
def test_router(renorm):
    logits = np.array([[1.0, 3.0, 3.0, -2.0, 3.0],
                       [-np.inf, 0.5, -np.inf, -np.inf, 0.25],
                       [-np.inf] * 5,
                       [-3.4e38] * 5])
    ids, w = L.router_topk(logits, 3, renorm)
    assert ids.tolist() == [[1, 2, 4], [1, 4, -1], [-1, -1, -1], [0, 1, 2]]
    assert w[2].tolist() == [0, 0, 0] and w[1, 2] == 0
    assert np.allclose(w[3], 1 / 3 if renorm else 1 / 5)
    rng = np.random.default_rng(4)
    logits, dw = rng.standard_normal((3, 6)), rng.standard_normal((3, 2))
    ids, _ = L.router_topk(logits, 2, renorm)
    d = _differences(lambda v: float(L.router_value(v, ids, dw, renorm).sum()), logits)
    assert np.abs(d - L.router_topk_bwd(logits, ids, dw, renorm)).max() < TOL
