"""mtp_latent_prefill with bounds out of range or out of order: reported, and taken as the nearest
good ones, which are in range and not below the bounds before them.  Sequences then never overlap:
the call gives, bit for bit, what it gives for the good bounds."""
import random

import pytest
import torch

import verify_spec_greedy_gb300 as lib
from test_gpu_latent_prefill import make, run, verify

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def taken(cu, n):
    out, top = [], 0
    for c in cu:
        top = max(top, min(c, n))
        out.append(top)
    return out


def compare(cu_q, cu_k, Tq, Tk, heads=3):
    x = make([Tq], [Tk], heads, 64, 32, 64, BF, seed=Tq)
    good = dict(x)
    for name, cu, n in (("cu_q", cu_q, Tq), ("cu_k", cu_k, Tk)):
        x[name] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        good[name] = torch.tensor(taken(cu, n), dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want, want_lse = run(good, status)
    assert int(status.item()) == 0
    verify(good, want, want_lse, heads=[0])
    for _ in range(3):
        status.zero_()
        out, lse = run(x, status)
        assert int(status.item()) == lib.STATUS_BAD_PARAM
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    last = good["cu_q"][-1].item()
    assert (out[last:] == 7.0).all()                # queries of no sequence are not written


@pytest.mark.parametrize("cu_q,cu_k", [
    ([0, 400, 150, 530], [0, 300, 500, 530]),       # a bound below the one before it
    ([0, 530, 0, 530, 0, 530], [0, 100, 200, 300, 400, 530]),   # the whole text three times over
    ([-9, 100, 1 << 30, 530], [0, 530, 530, 530]),
    ([0, 200, 400, 530], [0, 500, 20, 540]),
    ([300, 200, 100, 0], [0, 100, 200, 300]),
    ([0, 531], [0, 530]),
])
def test_bounds_out_of_order(cu_q, cu_k):
    compare(cu_q, cu_k, 530, 530)


@pytest.mark.parametrize("B", [5, 32, 33, 70, 300])
def test_many_bounds_out_of_order(B):
    # up to 32 sequences a lane holds one, beyond a run of them
    r = random.Random(B)
    cu = [[r.randint(-20, 1520) for _ in range(B + 1)] for _ in range(2)]
    cu[0][:3], cu[1][:3] = [0, 300, 40], [5, 2, 900]
    compare(cu[0], cu[1], 1500, 1500)


def test_slips_in_long_texts():
    # ascending but for a slip back every few sequences
    r = random.Random(3)
    cu = sorted(r.randint(0, 3000) for _ in range(101))
    slip = [max(0, c - (900 if i % 7 == 3 else 0)) for i, c in enumerate(cu)]
    compare(slip, cu, 3000, 3000, heads=2)
