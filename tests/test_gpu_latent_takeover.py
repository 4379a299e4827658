"""mtp_latent_prefill's work: a multiprocessor takes over pairs of query tiles whose CTAs have not
started.  The grid has a CTA for every pair that the lengths might give, so ragged calls leave
thousands of CTAs without work among those that have some.  Every pair is done, and calls repeat
bit for bit."""
import pytest
import torch

import verify_spec_greedy_gb300 as lib
from test_gpu_latent_prefill import make, run, verify

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("B,heads,long", [(600, 48, 0), (300, 128, 700), (32, 128, 900), (2, 128, 300)])
def test_thousands_of_ctas_without_work(B, heads, long):
    # two sequences in three have no queries; the last one may be long
    nq = [(7 * i) % 13 + 1 if i % 3 == 1 else 0 for i in range(B)]
    nq[-1] = max(long, 1)
    x = make(nq, nq, heads, 64, 16, 64, BF, seed=B)
    spare = heads * (-(-sum(nq) // 256) + B - 1 - sum(-(-n // 256) for n in nq))
    assert spare > 300 or B == 2                     # more than run at a time: asked for one by one
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want, want_lse = run(x, status)
    for _ in range(20):
        out, lse = run(x, status)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert int(status.item()) == 0
    verify(x, want, want_lse, heads=[0, heads // 2, heads - 1])


@pytest.mark.parametrize("B,heads", [(4, 64), (90, 12)])
def test_long_sequences_behind_empty_ones(B, heads):
    # more pairs than multiprocessors, and more CTAs without work than pairs
    nq = [0] * B
    nq[B // 3], nq[-1] = 700, 1100
    x = make(nq, nq, heads, 128, 64, 128, F16, seed=B)
    want, want_lse = run(x)
    verify(x, want, want_lse, heads=[0, heads - 1])
    for _ in range(10):
        out, lse = run(x)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
