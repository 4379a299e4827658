"""Every key is counted once: queries of zeros weigh all that they see alike, and values are marks
(a one in a column that the key's place decides), so that an output is the share of visible keys
with that mark, and lse the logarithm of their number.  A tile that is dropped, counted twice or
given to another row at a cut of the work shows at once.

Weights are equal powers of two, so sums of weights and of marks are whole numbers times one, exact
in fp32 below 2^24.  What is left is a division, at the joins an exponential of a difference of
logarithms (numbers up to 32, one rounding of which is 2^-20), at most 152 additions there, and the
output's rounding."""
import pytest
import torch

import test_gpu_latent_attn as absorbed
import test_gpu_latent_prefill as expanded
from latent_reference import half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16
JOIN = 8 * 2.0 ** -20 + 152 * 2.0 ** -24


def compare(out, lse, counts, seen):
    """counts [..., columns] of the seen [...] keys."""
    want = counts / seen.clamp(min=1)[..., None]
    off = (out.double() - want).abs() - want * (half_step(out.dtype) + JOIN)
    assert (off <= 0).all(), f"{int((off > 0).sum())} outputs off"
    some = seen > 0
    assert torch.equal(lse == -torch.inf, ~some)
    assert ((lse.double() - seen.clamp(min=1).log())[some].abs() <= JOIN).all()


def running(marks, columns):
    """[n + 1, columns]: the marks among the first keys."""
    c = torch.zeros(len(marks) + 1, columns, dtype=torch.float64, device=DEV)
    c[1:] = torch.nn.functional.one_hot(marks, columns).double().cumsum(0)
    return c


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("kv_len,T,H,L,page", [
    ([20000], 7, 24, 512, 128),                          # one row over all SMs, three row tiles
    ([100001], 1, 16, 512, 64),                          # 11 tiles a CTA, joined by units
    ([29201], 3, 5, 64, 48),                             # three tiles a CTA, one key in the last
    ([130, 1, 17], 3, 5, 192, 16),
    ([(977 * i) % 3001 for i in range(200)], 4, 16, 512, 64),     # joined by CTAs
    ([(61 * i) % 130 for i in range(900)], 1, 3, 128, 24),        # many whole units a CTA
    ([900, 2000, 30, 0, 1111], 4, 128, 512, 16),         # eight row tiles side by side
    ([5000, 900], 9, 64, 128, 8),                        # nine: two groups of five, one idle
])
@pytest.mark.parametrize("every", [64, 1])               # a mark a tile of keys, a mark a key
def test_absorbed(kv_len, T, H, L, page, every, dtype):
    R = 16
    x = absorbed.make(kv_len, T, H, L, R, page, dtype, seed=len(kv_len))
    x["q"].zero_()
    x["cache"].zero_()
    longest = max(kv_len)
    at = torch.arange(longest, device=DEV)
    marks = []
    for b, n in enumerate(kv_len):
        m = (at[:n] // every + 5 * b) % L                # another row's keys bear other marks
        x["cache"][x["table"][b, at[:n] // page].long(), at[:n] % page, m] = 1
        marks.append(m)
    out, lse = absorbed.run(x)
    for b, n in enumerate(kv_len):
        seen = (n - (T - 1 - torch.arange(T, device=DEV))).clamp(min=0)
        counts = running(marks[b], L)[seen]
        compare(out[b], lse[b], counts[:, None], seen[:, None].double().expand(T, H))


@pytest.mark.parametrize("dtype", [BF, F16])
def test_absorbed_at_every_cut(dtype):
    # lengths that move the cut of the work through a unit, tile by tile
    L, page = 64, 64
    for n in range(64 * 150, 64 * 156, 64):
        for extra in (1, 63, 64):
            x = absorbed.make([n + extra, 64 * 7, n - extra], 1, 2, L, 16, page, dtype)
            x["q"].zero_()
            x["cache"].zero_()
            at = torch.arange(n + 64, device=DEV)
            for b, k in enumerate(x["kv_len"].tolist()):
                x["cache"][x["table"][b, at[:k] // page].long(), at[:k] % page, (at[:k] // 64 + b) % L] = 1
            out, lse = absorbed.run(x)
            for b, k in enumerate(x["kv_len"].tolist()):
                seen = torch.full((1, 2), k, device=DEV)
                compare(out[b], lse[b], running((at[:k] // 64 + b) % L, L)[seen], seen.double())


@pytest.mark.parametrize("dtype", [BF, F16])
def test_the_longest_text(dtype):
    # one page, repeated over 2^31 - 256 positions: 220,000 tiles a CTA
    P, L, R, n = 4096, 64, 16, 2 ** 31 - 256
    x = absorbed.make([P], 1, 2, L, R, P, dtype)
    page = int(x["table"][0, 0])
    x["q"].zero_()
    x["cache"].zero_()
    at = torch.arange(P, device=DEV)
    x["cache"][page, at, at // 64] = 1
    x["table"] = torch.full((1, 2 ** 31 // P), page, dtype=torch.int32, device=DEV)
    x["kv_len"] = torch.tensor([n], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = absorbed.run(x, status)
    assert int(status) == 0
    counts = torch.full((L,), n // P * 64, device=DEV).double()
    counts[:n % P // 64] += 64
    assert counts.sum() == n
    compare(out[0, 0], lse[0, 0], counts.expand(2, L), torch.full((2,), n, device=DEV).double())


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("nq,nk,H,N,V", [
    ([8192], [8192], 3, 128, 128),
    ([700, 1, 300, 0, 2049], [7700, 500, 200, 77, 2050], 5, 64, 64),
    ([(97 * i) % 400 for i in range(50)], [(97 * i) % 400 + 3 * i for i in range(50)], 40, 128, 128),
    ([257] * 9 + [900], [257] * 9 + [1300], 64, 64, 128),
])
def test_expanded(nq, nk, H, N, V, dtype):
    R = 32
    x = expanded.make(nq, nk, H, N, R, V, dtype)
    x["q"].zero_()
    x["kv"].zero_()
    at = torch.cat([torch.arange(n, device=DEV) for n in nk])
    seq = torch.repeat_interleave(torch.arange(len(nk), device=DEV), torch.tensor(nk, device=DEV))
    for h in range(H):                                   # heads and sequences bear other marks
        mark = (at // (128 if h % 2 else 1) + 3 * h + 7 * seq) % V
        x["kv"][torch.arange(len(at), device=DEV), h, N + mark] = 1
    out, lse = expanded.run(x)
    cq = x["cu_q"].tolist()
    for b in range(len(nq)):
        seen = (torch.arange(nq[b], device=DEV) + (nk[b] - nq[b] + 1)).clamp(min=0)
        for h in {0, 1, H // 2, H - 1}:
            counts = running((torch.arange(nk[b], device=DEV) // (128 if h % 2 else 1) + 3 * h + 7 * b) % V, V)
            compare(out[cq[b]:cq[b + 1], h], lse[cq[b]:cq[b + 1], h], counts[seen], seen.double())
