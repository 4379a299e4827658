"""mtp_latent_attn against the formulas in 64 bits: rows and keys from one to many, pages that
end inside a tile, rows that see nothing, what lies beyond a length, strides, streams and
graphs."""
import pytest
import torch

import verify_spec_greedy_gb300 as lib
from latent_reference import attend, check, check_lse

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16


def make(kv_len, T, H, L, R, page, dtype, seed=0, spare=0, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B = len(kv_len)
    per = max(1, -(-max(kv_len) // page)) + spare
    pages = B * per + 2
    x = dict(q=(torch.randn(B, T, H, L + R, generator=g, device=DEV) * std).to(dtype),
             cache=torch.randn(pages, page, L + R, generator=g, device=DEV).to(dtype),
             table=torch.randperm(pages, generator=g, device=DEV)[:B * per].reshape(B, per).int(),
             kv_len=torch.tensor(kv_len, dtype=torch.int32, device=DEV), scale=(L // 4 + R) ** -0.5,
             T=T, H=H, L=L, R=R)
    return x


def buffers(x):
    q, L = x["q"], x["L"]
    B, T, H, _ = q.shape
    n = lib.mtp_latent_attn_workspace_bytes(B, T, H, L, x["R"])
    return (torch.full((B, T, H, L), 7.0, dtype=q.dtype, device=DEV),
            torch.full((B, T, H), 7.0, device=DEV), torch.empty(n, dtype=torch.uint8, device=DEV))


def run(x, status=None, stream=None):
    out, lse, ws = buffers(x)
    lib.mtp_latent_attn(x["q"], x["cache"], x["table"], x["kv_len"], out, x["scale"], lse=lse,
                        workspace=ws, status=status, stream=stream)
    return out, lse


def verify(x, out, lse, rows=None):
    T, H, L = x["T"], x["H"], x["L"]
    for b in rows if rows is not None else range(x["q"].shape[0]):
        n = max(0, int(x["kv_len"][b]))
        keys = x["cache"][x["table"][b].long()].flatten(0, 1)[:n]
        seen = n - (T - 1 - torch.arange(T, device=DEV)).repeat_interleave(H)
        want, wl, tol, ltol = attend(x["q"][b].flatten(0, 1), keys, keys[:, :L], seen, x["scale"],
                                     x["q"].dtype)
        check(out[b].reshape(T * H, L), want, tol, f"row {b}")
        check_lse(lse[b].reshape(-1), wl, ltol, f"row {b} lse")


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("kv_len,T,H,L,R,page", [
    ([1], 1, 1, 512, 64, 64),                       # one key
    ([64], 1, 16, 512, 64, 64),                     # exactly one tile
    ([65, 63], 1, 64, 512, 64, 8),                  # a tile and one key; a tile less one
    ([130, 1, 17], 3, 5, 512, 64, 16),              # short rows: queries that see nothing
    ([700, 333, 1500], 4, 16, 512, 64, 48),         # pages that end inside a tile
    ([911, 40, 2049], 2, 37, 256, 32, 24),
    ([513], 5, 13, 64, 16, 128),                    # two row tiles, the narrowest latent
    ([1000, 77], 1, 100, 448, 48, 64),              # pieces of 256, 128 and 64 columns
    ([260, 129], 1, 65, 320, 16, 32),               # one row into the second tile
    ([3000, 5], 2, 3, 384, 64, 1024),               # pages larger than a tile
    ([900, 2000, 30], 4, 128, 512, 64, 64),         # eight row tiles side by side
    ([500, 90], 9, 64, 128, 64, 64),                # nine: two groups of five, one idle
    ([20000], 7, 24, 512, 64, 128),                 # one row over all SMs
])
def test_against_64_bits(kv_len, T, H, L, R, page, dtype):
    x = make(kv_len, T, H, L, R, page, dtype, seed=len(kv_len) * 100 + H)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = run(x, status)
    assert int(status.item()) == 0
    verify(x, out, lse)


def test_many_short_rows():
    lens = [(i * 37) % 91 for i in range(301)]      # zeros among them
    x = make(lens, 1, 4, 512, 64, 16, BF, seed=1)
    out, lse = run(x)
    verify(x, out, lse)


def test_rows_that_see_nothing():
    x = make([0, 5, 0, 2, 300], 4, 8, 512, 64, 16, BF, seed=2)
    out, lse = run(x)
    verify(x, out, lse)
    assert not out[0].any() and not out[2].any() and (lse[[0, 2]] == -torch.inf).all()
    assert not out[3, :2].any() and (lse[3, :2] == -torch.inf).all()   # 2 keys, 4 queries
    assert (lse[3, 2:] > -torch.inf).all()
    x = make([0, 0], 1, 8, 512, 64, 16, BF)                            # nothing at all to do
    out, lse = run(x)
    assert not out.any() and (lse == -torch.inf).all()


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_what_lies_beyond_a_length_has_no_effect(junk):
    x = make([100, 64, 193, 1], 2, 16, 512, 64, 48, BF, seed=3, spare=2)
    want, want_lse = run(x)
    held = torch.zeros(x["cache"].shape[:2], dtype=torch.bool, device=DEV)
    for b, n in enumerate(x["kv_len"].tolist()):
        at = torch.arange(n, device=DEV)
        held[x["table"][b, at // 48].long(), at % 48] = True
    x["cache"][~held] = junk                                           # every row of no position
    for b, n in enumerate(x["kv_len"].tolist()):
        x["table"][b, -(-n // 48):] = torch.tensor([-7, 1 << 30], device=DEV)[b % 2].int()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = run(x, status)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert int(status.item()) == 0                                     # unneeded pages: not read


@pytest.mark.parametrize("dtype", [BF, F16])
def test_scores_that_climb_fall_and_stay(dtype):
    # the running maximum is raised at every tile, never, and for one row at one tile
    L, R, n = 512, 64, 1000
    x = make([n, n, n], 1, 3, L, R, 64, dtype, seed=4, std=0.02)
    ramp = torch.linspace(-1, 1, n, device=DEV)
    step = (torch.arange(n, device=DEV) > 517).float()
    for b, shape in enumerate([ramp, -ramp, step]):
        keys = x["cache"][x["table"][b].long()].flatten(0, 1)
        keys[:n, L + R - 1] = (shape * 60).to(dtype)
        x["cache"][x["table"][b].long()] = keys.view(-1, 64, L + R)
    x["q"][..., L + R - 1] = torch.tensor([30.0, 2.0, 0.0], device=DEV).to(dtype)
    out, lse = run(x)
    verify(x, out, lse)


def test_equal_scores_give_the_mean():
    x = make([777], 1, 2, 512, 64, 64, F16, seed=5)
    x["q"].zero_()
    out, lse = run(x)
    verify(x, out, lse)
    assert torch.allclose(lse, torch.tensor(777.0).log().to(DEV), rtol=1e-6)


def test_strides():
    B, T, H, L, R, page = 3, 2, 6, 256, 32, 16
    x = make([100, 31, 222], T, H, L, R, page, BF, seed=6)
    want, want_lse = run(x)
    wide = torch.zeros(H, B, T, L + R + 24, dtype=BF, device=DEV)
    q = wide.permute(1, 2, 0, 3)[..., 8:8 + L + R]
    q.copy_(x["q"])
    big = torch.zeros(x["cache"].shape[0], page + 5, L + R, dtype=BF, device=DEV)
    big[:, :page] = x["cache"]
    obuf = torch.full((T, B, H, L + 8), 5.0, dtype=BF, device=DEV)
    out = obuf.permute(1, 0, 2, 3)[..., :L]
    _, _, ws = buffers(x)
    lib.mtp_latent_attn(q, big[:, :page], x["table"], x["kv_len"], out, x["scale"], workspace=ws)
    assert torch.equal(out, want) and (obuf[..., L:] == 5.0).all()


def test_bad_lengths_and_pages_are_reported():
    x = make([64, 100, 64, 64], 1, 4, 128, 32, 16, BF, seed=7)
    x["kv_len"][0] = -3
    x["kv_len"][1] = 1 << 30                        # taken as all the row's pages
    x["table"][2, 1] = x["cache"].shape[0]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = run(x, status)
    assert int(status.item()) == lib.STATUS_BAD_PARAM
    assert not out[0].any() and (lse[0] == -torch.inf).all()
    x["kv_len"][1] = x["table"].shape[1] * 16
    verify(x, out, lse, rows=[1, 3])
    keys = x["cache"][x["table"][2].long().clamp(max=x["cache"].shape[0] - 1)].flatten(0, 1)[:64].clone()
    keys[16:32] = 0                                 # the bad page's positions are zeros
    want, wl, tol, ltol = attend(x["q"][2].flatten(0, 1), keys, keys[:, :128],
                                 torch.full((4,), 64, device=DEV), x["scale"], BF)
    check(out[2].reshape(4, 128), want, tol, "row 2")
    check_lse(lse[2].reshape(-1), wl, ltol, "row 2 lse")
    for only in (0, 1, 2):                          # each of them alone is reported
        y = make([64, 100, 64, 64], 1, 4, 128, 32, 16, BF, seed=7)
        y["kv_len"][only] = [-3, 1 << 30, 64][only]
        if only == 2:
            y["table"][2, 1] = -1
        status.zero_()
        run(y, status)
        assert int(status.item()) == lib.STATUS_BAD_PARAM


def test_repeats_bit_for_bit_without_lse_and_on_another_stream():
    x = make([2500, 900, 31], 3, 40, 512, 64, 64, BF, seed=8)
    want, want_lse = run(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out, lse = run(x, stream=s)
        s.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    out, _, ws = buffers(x)
    lib.mtp_latent_attn(x["q"], x["cache"], x["table"], x["kv_len"], out, x["scale"], workspace=ws)
    assert torch.equal(out, want)


def test_a_captured_call_follows_new_lengths():
    x = make([500, 100], 2, 16, 512, 64, 64, F16, seed=9, spare=20)
    out, lse, ws = buffers(x)
    call = lambda: lib.mtp_latent_attn(x["q"], x["cache"], x["table"], x["kv_len"], out,  # noqa: E731
                                       x["scale"], lse=lse, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([500, 100], [3, 1600], [0, 1], [1781, 1777]):
        x["kv_len"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        verify(x, out, lse)


def test_a_cache_of_more_than_32_bits():
    L, R, page = 512, 64, 128
    pages = (1 << 32) // ((L + R) * page) + 8
    x = make([1000], 1, 8, L, R, page, BF, seed=10)
    cache = torch.empty(pages, page, L + R, dtype=BF, device=DEV)
    cache[pages - 8:] = x["cache"][x["table"][0].long()]
    x["cache"] = cache
    x["table"] = torch.arange(pages - 8, pages, device=DEV).int()[None]
    out, lse = run(x)
    verify(x, out, lse)


def test_short_workspace_is_refused():
    x = make([64], 1, 4, 128, 32, 16, BF)
    out, lse, ws = buffers(x)
    with pytest.raises(lib.MtpSpecError):
        lib.mtp_latent_attn(x["q"], x["cache"], x["table"], x["kv_len"], out, 0.1, workspace=ws[:-1])
    with pytest.raises(lib.MtpSpecError):
        lib.mtp_latent_attn(x["q"], x["cache"], x["table"], x["kv_len"], out, 0.1)


@pytest.mark.parametrize("length", [2 ** 31 - 256, 2 ** 31 - 1])
def test_the_longest_text(length):
    # one page, repeated: position n has the scores of n % 4096; a longer length is reported
    # and taken as the longest
    P, L, R = 4096, 64, 16
    longest = 2 ** 31 - 256
    x = make([P], 1, 2, L, R, P, BF, seed=12)
    page = int(x["table"][0, 0])
    x["table"] = torch.full((1, 2 ** 31 // P), page, dtype=torch.int32, device=DEV)
    x["kv_len"] = torch.tensor([length], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = run(x, status=status)
    assert int(status) == (0 if length == longest else lib.STATUS_BAD_PARAM)
    keys = x["cache"][page].double()
    times = torch.full((P,), longest // P, device=DEV).double()
    times[:longest % P] += 1
    s = x["q"][0, 0].double() @ keys.T * x["scale"] + times.log()
    want, A = s.softmax(1) @ keys[:, :L], s.softmax(1) @ keys[:, :L].abs()
    # four additions a tile of a CTA's share, none off by more than 2^-22 of the sum so far
    steps = 4 * (longest // 64 // 152 + 1) + 16 + 152
    tol = (steps + 2 * 80) * 2.0 ** -22 + 2.0 ** -8
    assert ((out[0, 0].double() - want).abs() <= tol * A + 2.0 ** -8 * want.abs()).all()
    assert ((lse[0, 0].double() - s.logsumexp(1)).abs() <= tol).all()


@pytest.mark.parametrize("page", [8, 16, 24, 32, 40, 64, 192])
@pytest.mark.parametrize("L,R", [(512, 64), (448, 16), (320, 32), (256, 48), (192, 64)])
def test_pages_of_every_height(L, R, page):
    x = make([page, 333, 129, 1], 2, 5, L, R, page, BF, seed=page, spare=1)
    out, lse = run(x)
    verify(x, out, lse)
