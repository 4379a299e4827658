"""mtp_heads_append against its formulas in 64 bits."""
import pytest
import torch

import verify_spec_greedy_gb300 as lib
from latent_reference import E32, half_step, rms_norm, rotate

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


def rnd(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def turned(x, w, eps, cos_sin, pos, R, interleaved):
    """(value, bound): a norm and a rotation in fp32, rounded once.  The norm's sum, division, root
    and products are off by at most (D + 16) 2^-22 of the value, a rotation's three operations by
    4 * 2^-24 of |a| + |b|."""
    y = x.double() if w is None else rms_norm(x, w, eps)
    size = y.abs().clone()
    c = cos_sin[pos.long()][:, None]
    out = y.clone()
    out[..., :R] = rotate(y[..., :R], c.expand(-1, x.shape[1], -1), interleaved)
    # a turned pair is at most as large as both its elements together
    big = size[..., :R].amax(-1, keepdim=True) * 2
    size[..., :R] = torch.maximum(size[..., :R], big.expand(-1, -1, R))
    u = half_step(x.dtype)
    tol = u * out.abs() + ((x.shape[-1] + 16) * E32 + 4 * 2.0 ** -24) * size
    tiny = torch.finfo(x.dtype).tiny * u * 2
    return out, tol + tiny


def case(T, Hq, Hkv, D, R, P, dtype, interleaved=False, norm=True, layout="slots", seed=0, place=False):
    g = torch.Generator(device="cuda").manual_seed(seed + T + D)
    qkv = rnd(g, T, Hq + 2 * Hkv, D + 8, dtype=dtype)[..., :D]
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    B, longest = 3, 2 * T + 9
    wide = -(-longest // P)
    pages = B * wide + 2
    table = torch.randperm(pages, generator=g, device="cuda")[:B * wide].view(B, wide).int()
    row = torch.randint(0, B, (T,), generator=g, device="cuda").int()
    pos = torch.randperm(longest, generator=g, device="cuda")[:T].int()
    shape = (pages, Hkv, P, D) if layout == "heads" else (pages, P, Hkv, D)
    kc, vc = (rnd(g, *shape, dtype=dtype) for _ in range(2))
    if layout == "heads":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    angle = rnd(g, longest, R // 2)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1)
    w = [(1 + 0.3 * rnd(g, D)).to(dtype) if norm else None for _ in range(2)]
    k0, v0, q0 = kc.clone(), vc.clone(), q.clone()
    q_out = q if place else torch.empty(T, Hq, D, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eps = 1e-5
    lib.mtp_heads_append(k, v, cos_sin, row, pos, table, kc, vc, k_norm_w=w[0], q=q, q_out=q_out,
                         q_norm_w=w[1], eps=eps, interleaved=interleaved, status=status)
    assert int(status) == 0
    page, off = table[row.long(), pos.long() // P].long(), pos.long() % P
    for got, x, wt in ((kc[page, off], k, w[0]), (q_out, q0, w[1])):
        want, tol = turned(x, wt, eps, cos_sin, pos, R, interleaved)
        over = (got.double() - want).abs() - tol
        assert (over <= 0).all(), f"off by {over.max().item():.3e} more than allowed"
    assert torch.equal(vc[page, off], v)
    k0[page, off], v0[page, off] = kc[page, off], vc[page, off]
    assert torch.equal(k0, kc) and torch.equal(v0, vc)       # nothing else was written


@pytest.mark.parametrize("Hq,Hkv,D,R", [(32, 8, 128, 128), (4, 1, 256, 64), (3, 3, 64, 32), (5, 1, 96, 96),
                                        (1, 1, 16, 16), (14, 2, 80, 48), (2, 2, 144, 144), (7, 7, 192, 16),
                                        (40, 8, 48, 32), (16, 2, 256, 256)])
@pytest.mark.parametrize("dtype,interleaved", [(BF, False), (F16, True), (BF, True), (F16, False)])
def test_heads(Hq, Hkv, D, R, dtype, interleaved):
    case(37, Hq, Hkv, D, R, 16, dtype, interleaved)


@pytest.mark.parametrize("T", [1, 2, 7, 64, 1000])
@pytest.mark.parametrize("P,layout", [(8, "slots"), (48, "heads"), (256, "slots")])
def test_tokens(T, P, layout):
    case(T, 12, 4, 128, 64, P, BF, layout=layout)


@pytest.mark.parametrize("interleaved", [False, True])
def test_without_norms_and_in_place(interleaved):
    case(50, 8, 2, 128, 128, 32, BF, interleaved, norm=False, place=True)
    case(50, 9, 3, 64, 64, 32, F16, interleaved, norm=True, place=True)


def test_keys_alone_and_one_norm_alone():
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v, q = (rnd(g, 5, 2, 64, dtype=BF) for _ in range(3))
    kc, vc = (torch.zeros(3, 8, 2, 64, dtype=BF, device="cuda") for _ in range(2))
    angle = rnd(g, 20, 16)
    cs = torch.cat([angle.cos(), angle.sin()], 1)
    row, pos = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.arange(5, device="cuda").int()
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    lib.mtp_heads_append(k, v, cs, row, pos, table, kc, vc)
    want, tol = turned(k, None, 0, cs, pos, 32, False)
    assert ((kc[2, :5].double() - want).abs() <= tol).all() and torch.equal(vc[2, :5], v)
    w = (1 + rnd(g, 64)).to(BF)
    out = torch.empty_like(q)
    lib.mtp_heads_append(k, v, cs, row, pos, table, kc, vc, q=q, q_out=out, q_norm_w=w, eps=0.1)
    assert ((kc[2, :5].double() - want).abs() <= tol).all()
    want, tol = turned(q, w, 0.1, cs, pos, 32, False)
    assert ((out.double() - want).abs() <= tol).all()


def test_padding_and_bad_tokens():
    g = torch.Generator(device="cuda").manual_seed(2)
    T = 7
    k, v, q = (rnd(g, T, 2, 128, dtype=BF) for _ in range(3))
    kc, vc = (torch.zeros(4, 8, 2, 128, dtype=BF, device="cuda") for _ in range(2))
    cs = torch.cat([torch.zeros(30, 8), torch.ones(30, 8)], 1).cuda()  # a quarter turn
    #                  good  pad  row     position  position  page  page
    row = torch.tensor([0, -1, 2, 1, 1, 1, 0], dtype=torch.int32, device="cuda")
    pos = torch.tensor([3, 4, 5, -1, 16, 9, 12], dtype=torch.int32, device="cuda")
    table = torch.tensor([[3, 4], [1, -1]], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 9)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.mtp_heads_append(k, v, cs, row, pos, table, kc, vc, q=q, q_out=out, status=status)
    assert int(status) == lib.STATUS_BAD_PARAM
    assert kc.count_nonzero() and kc[3, 3].count_nonzero() == kc.count_nonzero()
    assert torch.equal(vc[3, 3], v[0]) and vc[3, 3].count_nonzero() == vc.count_nonzero()
    assert (out[1:5] == 9).all()
    for t in (0, 5, 6):
        assert torch.equal(out[t, :, :8], -q[t, :, 8:16]) and torch.equal(out[t, :, 16:], q[t, :, 16:])
    for t in (0, 1, 2):                                        # a padding token alone is no fault
        status.zero_()
        lib.mtp_heads_append(k[1:2], v[1:2], cs, row[1:2], pos[1:2], table, kc, vc, status=status)
        assert int(status) == 0


def test_far_slots_and_long_positions():
    """Pages whose offsets need 64 bits, and positions up to a million."""
    pages, P, Hkv, D = 2 ** 31 // (64 * 4 * 128) + 5, 64, 4, 128
    kc = torch.zeros(pages, P, Hkv, D, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (rnd(g, 2, Hkv, D, dtype=BF) for _ in range(2))
    n = 1_000_000
    angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, 32, 2, device="cuda", dtype=torch.float64) / 32)
    cs = torch.cat([angle.cos(), angle.sin()], 1).float()
    table = torch.full((1, n // P), pages - 1, dtype=torch.int32, device="cuda")
    pos = torch.tensor([n - 2, n - 1], dtype=torch.int32, device="cuda")
    lib.mtp_heads_append(k, v, cs, torch.zeros(2, dtype=torch.int32, device="cuda"), pos, table, kc, vc)
    want, tol = turned(k, None, 0, cs, pos, 32, False)
    at = pos.long() % P
    assert ((kc[-1, at].double() - want).abs() <= tol).all() and torch.equal(vc[-1, at], v)
