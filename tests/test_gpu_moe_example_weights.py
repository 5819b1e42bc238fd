"""The float weights that examples/moe_layer.py takes: any strides and floating-point type, on a GPU
or not, to the same 4-bit weights as the contiguous float32 ones on the GPU."""
import pytest
import torch

from tests.test_gpu_moe_example import _example

pytestmark = pytest.mark.gpu


def _all(experts):
    return [t for pair in (experts.gate_up, experts.down, experts.gate_up_t, experts.down_t)
            for t in pair]


@pytest.mark.parametrize("form", ["transposed", "sliced", "float16", "float64", "cpu"])
def test_experts_from_any_floats(cuda_lib, form):
    ex = _example()
    D, F, E = 256, 128, 3
    g = torch.Generator().manual_seed(3)
    plain = [torch.randn(E, 2 * F, D, generator=g).half().float().cuda(),
             torch.randn(E, D, F, generator=g).half().float().cuda()]
    want = ex.Experts.from_float(*plain)
    given = [{"transposed": lambda w: w.transpose(1, 2).contiguous().transpose(1, 2),
              "sliced": lambda w: torch.stack([w, w], dim=-1)[..., 0],
              "float16": torch.Tensor.half, "float64": torch.Tensor.double,
              "cpu": torch.Tensor.cpu}[form](w) for w in plain]
    for made in (ex.Experts.from_float(*given), ex.Experts.from_float(*(-w for w in plain))):
        made.quantize(*given)
        for got, w in zip(_all(made), _all(want)):
            assert torch.equal(got, w)
    for got, w in zip(_all(ex.Experts.from_float(*given)), _all(want)):
        assert torch.equal(got, w)
