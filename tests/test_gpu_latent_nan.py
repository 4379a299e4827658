"""Queries that hold NaN or infinities: out and lse are NaN, not the zero and -inf of a query that
sees nothing (which such a query still has when it sees nothing), and every other query keeps its
results bit for bit."""
import pytest
import torch

import test_gpu_latent_attn as absorbed
import test_gpu_latent_prefill as expanded

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


def all_nan(t):
    return bool(torch.isnan(t).all())


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("junk", [NAN, INF])
@pytest.mark.parametrize("kv_len,T,H", [
    ([200], 1, 5),                          # one unit cut among CTAs, joined by units
    ([300, 90, 1], 2, 40),                  # two row tiles
    ([700] * 200, 1, 3),                    # whole units, and units joined by CTAs
])
def test_absorbed(kv_len, T, H, junk, dtype):
    x = absorbed.make(kv_len, T, H, 128, 32, 16, dtype, seed=T)
    want, want_lse = absorbed.run(x)
    bad = torch.zeros(len(kv_len), T, H, dtype=torch.bool, device=DEV)
    bad[:, T - 1, H // 2] = True
    bad[0, 0, 0] = True
    # +inf against keys of both signs: scores of both infinities, and +inf less itself
    x["q"][..., 3] = torch.where(bad, torch.tensor(junk, dtype=dtype, device=DEV), x["q"][..., 3])
    out, lse = absorbed.run(x)
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])
    # (an infinity against a single key may leave a score of -inf and nothing else: 0 and -inf)
    seen = torch.tensor(kv_len, device=DEV)[:, None] - (T - 1 - torch.arange(T, device=DEV))
    sure = bad & (seen > (1 if junk == INF else 0))[..., None]
    assert sure.any()
    assert all_nan(out[sure]) and all_nan(lse[sure])


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("junk", [NAN, INF])
def test_expanded(junk, dtype):
    nq, nk = [300, 5, 140], [300, 45, 100]
    x = expanded.make(nq, nk, 3, 64, 32, 64, dtype, seed=2)
    want, want_lse = expanded.run(x)
    bad = torch.zeros(sum(nq), 3, dtype=torch.bool, device=DEV)
    bad[[70, 299, 301, 444], [0, 1, 2, 1]] = True
    x["q"][bad] = junk
    out, lse = expanded.run(x)
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])
    assert all_nan(out[bad]) and all_nan(lse[bad])


def test_queries_that_see_nothing_keep_zero():
    x = absorbed.make([2, 0], 4, 3, 128, 32, 16, BF, seed=3)
    x["q"].fill_(NAN)
    out, lse = absorbed.run(x)
    assert not out[1].any() and (lse[1] == -INF).all()
    assert not out[0, :2].any() and (lse[0, :2] == -INF).all()
    assert all_nan(out[0, 2:]) and all_nan(lse[0, 2:])
    x = expanded.make([200], [60], 2, 64, 32, 64, BF, seed=4)
    x["q"].fill_(NAN)
    out, lse = expanded.run(x)
    assert not out[:140].any() and (lse[:140] == -INF).all()
    assert all_nan(out[140:]) and all_nan(lse[140:])
