"""One high score before many equal low ones, in both forms.  The high key's value is zero, so the
output is made of weights 2^-16 to 2^-21 of the largest.  They are equal, so their roundings do
not cancel: each weight has to be right to half a step of the type.

Scores are exact here (one product each, of small whole numbers).  With n keys of equal weight and
values of one sign, out is off by
  - the rounding of the weights and that of the output:   u each
  - n / 16 additions of 16 products, 2^-22 each at most, and as in the sums below
and ln of the sum by n / 64 additions of a tile's sum and those within a tile, 2^-24 each, and a
few roundings of its own size."""
import math

import pytest
import torch

import test_gpu_latent_attn as absorbed
import test_gpu_latent_prefill as expanded
from latent_reference import attend, check, check_lse, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16
CASES = [(n, gap) for n in (2000, 20000, 100000) for gap in (16.9, 18.4, 19.55, 20.7)]


def bounds(want, lse, n, dtype):
    steps = n / 64 + 20
    return (want * (2 * half_step(dtype) + (n / 16 + 32) * 2.0 ** -22 + steps * 2.0 ** -24),
            steps * 2.0 ** -24 + 2.0 ** -22 * (lse.abs() + 8))


def values(*shape, dtype):
    g = torch.Generator(device=DEV).manual_seed(1)
    return (0.5 + torch.rand(*shape, generator=g, device=DEV)).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("n,gap", CASES)
def test_absorbed(n, gap, dtype):
    # as many rows of one length as multiprocessors: none is cut, so that no part of a row takes
    # its own low scores for high ones
    L, R, page, B = 64, 16, 64, 152
    pages = -(-n // page)
    cache = torch.zeros(pages, page, L + R, dtype=dtype, device=DEV)
    cache[..., :L] = values(pages, page, L, dtype=dtype)
    cache[0, 0] = 0
    cache[0, 0, L] = 8
    q = torch.zeros(B, 1, 2, L + R, dtype=dtype, device=DEV)
    q[..., L] = 8
    x = dict(q=q, cache=cache, table=torch.arange(pages, device=DEV).int().repeat(B, 1),
             kv_len=torch.full((B,), n, dtype=torch.int32, device=DEV), scale=gap * math.log(2) / 64,
             T=1, H=2, L=L, R=R)
    out, lse = absorbed.run(x)
    keys = cache.flatten(0, 1)[:n]
    want, want_lse, _, _ = attend(q[0, 0], keys, keys[:, :L], torch.tensor([n, n], device=DEV),
                                  x["scale"], dtype)
    tol, lse_tol = bounds(want, want_lse, n, dtype)
    for b in range(B):
        check(out[b, 0], want, tol, f"row {b}")
        check_lse(lse[b, 0], want_lse, lse_tol, f"row {b} lse")


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("n,gap", CASES)
def test_expanded(n, gap, dtype):
    N, R, V, nq = 64, 16, 64, 256
    x = expanded.make([nq], [n], 1, N, R, V, dtype)
    for name in ("q", "kv", "rot"):
        x[name].zero_()
    x["kv"][..., N:] = values(n, 1, V, dtype=dtype)
    x["kv"][0] = 0
    x["q"][..., N], x["rot"][0, 0] = 8, 8
    x["scale"] = gap * math.log(2) / 64
    out, lse = expanded.run(x)
    seen = torch.arange(nq, device=DEV) + (n - nq + 1)
    want, want_lse, _, _ = attend(x["q"][:, 0], torch.cat([x["kv"][:, 0, :N], x["rot"]], 1),
                                  x["kv"][:, 0, N:], seen, x["scale"], dtype)
    tol, lse_tol = bounds(want, want_lse, n, dtype)
    check(out[:, 0], want, tol, "out")
    check_lse(lse[:, 0], want_lse, lse_tol, "lse")
