"""A program that takes its workspace once, for its largest batch, has enough of it for every smaller
one: what the queries answer never falls as the rows grow.  No GPU needed."""
import pytest

from tests.test_abi_moe_layer import lib  # noqa: F401  (the fixture)

ROWS = sorted({1, 2, 7, 8, 9, 4095, 4096, 16384, 16385, 1 << 20, (1 << 31) - 1,
               *range(100, 2000, 3), *range(2048, 40000, 509)})


@pytest.mark.parametrize("D", [8, 128, 264, 1024, 2048, 4104, 6144, 8200, 16384])
def test_norm_gradient(lib, D):  # noqa: F811
    f = lib.hg_rmsnorm_bwd_workspace_bytes
    need = [f(M, D) for M in ROWS]
    assert need == sorted(need) and need[0] >= 4 * D
    assert need[-1] <= 4 * D * 152 * 3                    # a row a block, whatever M


@pytest.mark.parametrize("E,N,K", [(1, 256, 256), (1, 1024, 1024), (3, 520, 128), (16, 520, 384),
                                   (32, 4096, 6144)])
def test_weight_gradient(lib, E, N, K):  # noqa: F811
    rows = [r for r in ROWS if r <= 1 << 20]              # (of sizes that the call takes)
    for f in (lib.hg_grouped_wgrad_workspace_bytes, lib.hg_grouped_wgrad_fp8_workspace_bytes):
        need = [f(E, N, K, r) for r in rows]
        assert need == sorted(need)
