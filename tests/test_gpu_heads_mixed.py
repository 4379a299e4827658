"""mtp_heads_attn for batches whose rows differ most: a prompt among drafts or among rows of no tokens, on
both sides of the choice between the kernels."""
import pytest
import torch

import verify_spec_greedy_gb300 as lib
from heads_reference import Batch

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("rows", [
    [(0, 0)] * 20 + [(33, 40)] + [(0, 5)] * 43,                          # a prompt among rows of none
    [(1, 90 + i) for i in range(255)] + [(425, 425)],                    # 680 tokens, and one more
    [(1, 90 + i) for i in range(255)] + [(426, 426)],
    [(0, 3)] * 700 + [(701, 900)],                                       # as many tokens as rows, and more
    [(0, 3)] * 700 + [(1402, 1402)], [(0, 3)] * 700 + [(1403, 1500)],
    [(1 + i % 4, 60 + 3 * i) for i in range(256)], [(3, 60 + 3 * i) for i in range(256)]])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 64, BF), (4, 4, 48, F16), (32, 2, 64, BF)])
def test_prompts_among_rows_of_few_tokens_or_none(rows, Hq, Hkv, D, dtype):
    x = Batch(rows, Hq, Hkv, D, 16, dtype, seed=len(rows), pad=2)
    x.run(lib)
    x.check(heads=sorted({0, Hq - 1}))
