"""The MoE layer's steps on the GPU at the ends of their ranges, against their float64
definitions.  Tolerances are those of test_gpu_moe_layer unless stated at the test.
"""
import pytest
import torch

from synth import make_routing, make_weights
from tests.test_gpu_moe_layer import _normal

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
