"""mtp_latent_append against the formulas in 64 bits: every row, position type, stride and
page size; tokens that are padding or out of range; what must stay untouched."""
import pytest
import torch

import verify_spec_greedy_gb300 as lib
from latent_reference import E32, check, half_step, rms_norm, rotate

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16


def make(T, B, H, L, R, page, max_pages, dtype, seed=0, extra_pages=2):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)  # noqa: E731
    pages = B * max_pages + extra_pages
    slots = max_pages * page
    order = torch.randperm(B * slots, generator=g, device=DEV)[:T]
    a = torch.randn(slots, R // 2, generator=g, device=DEV) * 40
    return dict(latent=rn(T, L), rot=rn(T, R), cos_sin=torch.cat([a.cos(), a.sin()], 1).contiguous(),
                tok_row=(order // slots).int(), positions=(order % slots).int(),
                block_table=torch.randperm(pages, generator=g, device=DEV)[:B * max_pages]
                .reshape(B, max_pages).int(),
                cache=rn(pages, page, L + R), norm_w=rn(L), q_rot=rn(T, H, R),
                q_out=torch.zeros(T, H, R, dtype=dtype, device=DEV))


def expected(x, interleaved, norm, eps):
    """(values, tolerance) of each token's cache row and of its queries."""
    dt = x["latent"].dtype
    u = half_step(dt)
    c = rms_norm(x["latent"], x["norm_w"], eps) if norm else x["latent"].double()
    c_tol = c.abs() * (u + 16 * E32) if norm else torch.zeros_like(c)
    cs = x["cos_sin"][x["positions"].long().clamp(0, x["cos_sin"].shape[0] - 1)]
    k = rotate(x["rot"].double(), cs, interleaved)
    # two products and a sum in fp32 of values up to |a| + |b|, then one rounding
    mag = rotate(x["rot"].double().abs(), cs.abs() * torch.cat(
        [torch.ones_like(cs[:, :1]).expand(-1, cs.shape[1] // 2),
         torch.ones_like(cs[:, :1]).expand(-1, cs.shape[1] // 2)], 1), interleaved).abs()
    big = x["rot"].double().abs().amax(1, keepdim=True) * 2
    k_tol = k.abs() * u + 2 * E32 * torch.maximum(mag, big)
    q = rotate(x["q_rot"].double(), cs[:, None].expand(-1, x["q_rot"].shape[1], -1), interleaved)
    q_tol = q.abs() * u + 4 * E32 * x["q_rot"].double().abs().amax(-1, keepdim=True)
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    return (torch.cat([c, k], 1), torch.cat([c_tol, k_tol], 1) + tiny, q, q_tol + tiny)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("T,B,H,L,R,page,max_pages,norm,interleaved", [
    (1, 1, 1, 512, 64, 64, 3, True, True),
    (1, 1, 16, 64, 16, 8, 1, False, False),
    (7, 3, 5, 256, 32, 16, 2, True, False),
    (33, 2, 24, 512, 64, 48, 1, False, True),
    (257, 5, 3, 448, 48, 24, 4, True, True),
    (1000, 9, 128, 512, 64, 128, 2, True, False),
])
def test_rows_and_queries(dtype, T, B, H, L, R, page, max_pages, norm, interleaved):
    x = make(T, B, H, L, R, page, max_pages, dtype, seed=T)
    before = x["cache"].clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.mtp_latent_append(x["latent"], x["rot"], x["cos_sin"], x["tok_row"], x["positions"],
                          x["block_table"], x["cache"], norm_w=x["norm_w"] if norm else None,
                          eps=1e-5, interleaved=interleaved, q_rot=x["q_rot"], q_out=x["q_out"],
                          status=status)
    rows, tol, q, q_tol = expected(x, interleaved, norm, 1e-5)
    pos = x["positions"].long()
    slot = x["block_table"][x["tok_row"].long(), pos // page].long() * page + pos % page
    flat = x["cache"].view(-1, L + R)
    check(flat[slot], rows, tol, "cache rows")
    check(x["q_out"], q, q_tol, "queries")
    rest = torch.ones(flat.shape[0], dtype=torch.bool, device=DEV)
    rest[slot] = False
    assert torch.equal(flat[rest], before.view(-1, L + R)[rest])   # every other row untouched
    assert int(status.item()) == 0


def test_strided_views_and_queries_in_place():
    T, H, L, R = 19, 6, 128, 32
    x = make(T, 2, H, L, R, 16, 4, BF, seed=3)
    down = torch.cat([x["latent"], x["rot"], x["rot"]], 1)            # rows of L + 2R
    wide = torch.zeros(T, H, L + R + 8, dtype=BF, device=DEV)
    wide[..., L:L + R] = x["q_rot"]
    big = torch.zeros(x["cache"].shape[0], 16 + 3, L + R, dtype=BF, device=DEV)
    cache = big[:, :16]                                               # a page stride of its own
    lib.mtp_latent_append(down[:, :L], down[:, L:L + R], x["cos_sin"], x["tok_row"], x["positions"],
                          x["block_table"], cache, q_rot=wide[..., L:L + R], q_out=wide[..., L:L + R])
    rows, tol, q, q_tol = expected(x, True, False, 0.0)
    pos = x["positions"].long()
    page = x["block_table"][x["tok_row"].long(), pos // 16].long()
    check(cache[page, pos % 16], rows, tol, "cache rows")
    check(wide[..., L:L + R], q, q_tol, "queries")
    assert not wide[..., :L].any() and not wide[..., L + R:].any() and not big[:, 16:].any()


def test_the_first_position_is_not_turned():
    x = make(4, 1, 2, 64, 16, 8, 2, F16, seed=9)
    x["cos_sin"][0] = torch.tensor([1.0] * 8 + [0.0] * 8, device=DEV)
    x["positions"].zero_()
    x["tok_row"][1:] = -1                                             # one token, three paddings
    lib.mtp_latent_append(x["latent"], x["rot"], x["cos_sin"], x["tok_row"], x["positions"],
                          x["block_table"], x["cache"], q_rot=x["q_rot"], q_out=x["q_out"])
    row = x["cache"][x["block_table"][0, 0].item(), 0]
    assert torch.equal(row, torch.cat([x["latent"][0], x["rot"][0]]))
    assert torch.equal(x["q_out"][0], x["q_rot"][0]) and not x["q_out"][1:].any()


def test_tokens_out_of_range_write_nothing():
    x = make(8, 2, 3, 64, 16, 8, 2, BF, seed=5)
    x["tok_row"][:] = torch.tensor([0, 1, -1, 2, 0, 1, 0, 1], device=DEV)
    x["positions"][:] = torch.tensor([3, 15, 2, 1, -1, 16, 9, 0], device=DEV)
    x["block_table"][0, 1] = x["cache"].shape[0]                      # token 6's page
    x["block_table"][1, 0] = -5                                       # token 7's page
    before = x["cache"].clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.mtp_latent_append(x["latent"], x["rot"], x["cos_sin"], x["tok_row"], x["positions"],
                          x["block_table"], x["cache"], q_rot=x["q_rot"], q_out=x["q_out"],
                          status=status)
    assert int(status.item()) == lib.STATUS_BAD_PARAM
    rows, tol, q, q_tol = expected(x, True, False, 0.0)
    want = before.clone()
    for t, (pg, off) in {0: (x["block_table"][0, 0].item(), 3),
                         1: (x["block_table"][1, 1].item(), 7)}.items():
        check(x["cache"][pg, off][None], rows[t][None], tol[t][None], f"token {t}")
        want[pg, off] = x["cache"][pg, off]
    assert torch.equal(x["cache"], want)
    good = [0, 1, 6, 7]                                               # good row and position
    check(x["q_out"][good], q[good], q_tol[good], "queries")
    assert not x["q_out"][[2, 3, 4, 5]].any()


def test_positions_past_the_angles_are_refused_on_the_device():
    x = make(2, 1, 1, 64, 16, 8, 2, BF, seed=6)
    x["tok_row"].zero_()
    x["positions"][:] = torch.tensor([5, 6], device=DEV)
    before = x["cache"].clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lib.mtp_latent_append(x["latent"], x["rot"], x["cos_sin"][:6].contiguous(), x["tok_row"],
                          x["positions"], x["block_table"], x["cache"], status=status)
    assert int(status.item()) == lib.STATUS_BAD_PARAM
    pg = x["block_table"][0, 0].item()
    assert torch.equal(x["cache"][pg, 6], before[pg, 6])
    assert not torch.equal(x["cache"][pg, 5], before[pg, 5])


def test_no_tokens_no_launch():
    x = make(1, 1, 1, 64, 16, 8, 1, BF)
    n = lib.mtpspec_launch_count()
    lib.mtp_latent_append(x["latent"][:0], x["rot"][:0], x["cos_sin"], x["tok_row"][:0],
                          x["positions"][:0], x["block_table"], x["cache"])
    assert lib.mtpspec_launch_count() == n


def test_a_cache_of_more_than_32_bits():
    # 4.3e9 values: the last page starts beyond 2^32 elements
    L, R, page = 512, 64, 128
    pages = (1 << 32) // ((L + R) * page) + 2
    cache = torch.empty(pages, page, L + R, dtype=BF, device=DEV)
    x = make(3, 1, 2, L, R, page, 1, BF, seed=8)
    x["block_table"][0, 0] = pages - 1
    cache[pages - 1].zero_()
    lib.mtp_latent_append(x["latent"], x["rot"], x["cos_sin"], x["tok_row"], x["positions"],
                          x["block_table"], cache)
    rows, tol, _, _ = expected(x, True, False, 0.0)
    check(cache[pages - 1][x["positions"].long()], rows, tol, "cache rows")
