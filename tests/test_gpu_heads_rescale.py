"""mtp_heads_attn where the running maximum rises late and often, so that outputs and sums that are
already there are scaled again: both kernels, every width of a head's tile, and warps of which some
rows rise and others do not."""
import pytest
import torch

import verify_spec_greedy_gb300 as lib
from heads_reference import Batch

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("rows", [[(1, 2000)], [(3, 5000), (1, 700)], [(200, 2000)]])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (8, 1, 64), (32, 1, 48), (4, 4, 16), (8, 2, 128), (8, 1, 144),
                                      (4, 1, 256)])
def test_scores_far_apart(Hq, Hkv, D, rows, dtype):
    """Scores of some +-16 D^(1/2)."""
    x = Batch(rows, Hq, Hkv, D, 16, dtype, seed=D + len(rows), std=4.0)
    x.run(lib)
    x.check(heads=sorted({0, Hq - 1}))


def rising(x, step, some):
    """Keys whose first element grows by `step` every 64 positions, and queries whose first element is
    1 / scale (in every other head, where only `some` rise): the scores grow by `step` too."""
    x.q[:, :, 0] = 0
    x.q[:, ::2 if some else 1, 0] = x.scale ** -1
    P = x.P
    for b, (_, n) in enumerate(x.rows):
        at = torch.arange(n, device="cuda")
        up = (at // 64 * step).to(x.dtype)
        x.keys[b][:, :, 0] = up[:, None]
        x.k[x.table[b].long()[at // P], at % P, :, 0] = up[:, None]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("some", [False, True])
@pytest.mark.parametrize("step", [4.0, 8.0, 16.0])
@pytest.mark.parametrize("rows", [[(1, 1500)], [(2, 900), (1, 65), (1, 1400)], [(150, 1100), (40, 40)]])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (16, 1, 16), (8, 2, 128), (4, 1, 256)])
def test_the_maximum_rises_tile_after_tile(Hq, Hkv, D, rows, step, some, dtype):
    x = Batch(rows, Hq, Hkv, D, 32, dtype, seed=D, std=0.5)
    rising(x, step, some)
    x.run(lib)
    x.check(heads=[0, 1, Hq - 1])
    # with a window the maximum falls again from query to query, and rises within each
    x.run(lib, 200, 3)
    x.check(200, 3, heads=[0, 1])
