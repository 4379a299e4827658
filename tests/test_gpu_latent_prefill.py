"""mtp_latent_prefill against the formulas in 64 bits: ragged prompts from one token to many
tiles, chunks behind a prefix, queries that see nothing, neighbours that must not leak,
strides, streams and graphs."""
import pytest
import torch

import verify_spec_greedy_gb300 as lib
from latent_reference import attend, check, check_lse

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16


def make(nq, nk, H, N, R, V, dtype, seed=0, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: (torch.randn(*s, generator=g, device=DEV) * std).to(dtype)  # noqa: E731
    cu = lambda n: torch.tensor([0] + n, device=DEV).cumsum(0).int()  # noqa: E731
    return dict(q=rn(sum(nq), H, N + R), kv=rn(sum(nk), H, N + V), rot=rn(sum(nk), R), cu_q=cu(nq),
                cu_k=cu(nk), scale=(N + R) ** -0.5, N=N, V=V)


def run(x, status=None, stream=None):
    Tq, H, _ = x["q"].shape
    out = torch.full((Tq, H, x["V"]), 7.0, dtype=x["q"].dtype, device=DEV)
    lse = torch.full((Tq, H), 7.0, device=DEV)
    lib.mtp_latent_prefill(x["q"], x["kv"], x["rot"], x["cu_q"], x["cu_k"], out, x["scale"], lse=lse,
                           status=status, stream=stream)
    return out, lse


def verify(x, out, lse, heads=None):
    cq, ck = x["cu_q"].tolist(), x["cu_k"].tolist()
    for b in range(len(cq) - 1):
        q, kv, rot = x["q"][cq[b]:cq[b + 1]], x["kv"][ck[b]:ck[b + 1]], x["rot"][ck[b]:ck[b + 1]]
        seen = torch.arange(len(q), device=DEV) + (len(kv) - len(q) + 1)
        for h in heads or range(q.shape[1]):
            want, wl, tol, ltol = attend(q[:, h], torch.cat([kv[:, h, :x["N"]], rot], 1),
                                         kv[:, h, x["N"]:], seen, x["scale"], q.dtype)
            check(out[cq[b]:cq[b + 1], h], want, tol, f"sequence {b} head {h}")
            check_lse(lse[cq[b]:cq[b + 1], h], wl, ltol, f"sequence {b} head {h} lse")


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("nq,nk,H,N,R,V", [
    ([1], [1], 1, 128, 64, 128),
    ([128], [128], 2, 128, 64, 128),
    ([129, 127], [129, 127], 3, 128, 64, 128),
    ([256, 257, 1], [256, 257, 1], 2, 128, 64, 128),
    ([300, 5, 640], [300, 5, 640], 2, 64, 32, 64),
    ([900], [900], 2, 128, 48, 64),
    ([70, 1, 513], [1070, 900, 514], 2, 64, 16, 128),   # behind a prefix; a single query
    ([200, 40, 9], [60, 0, 9], 2, 128, 64, 128),        # queries that see nothing, no keys at all
    ([400], [130], 1, 128, 64, 128),                    # a whole tile of such queries
    ([1500], [1500], 1, 128, 64, 128),                  # the ring goes round many times
    ([0, 17, 0, 33], [0, 17, 5, 40], 5, 128, 64, 128),  # sequences of no queries
])
def test_against_64_bits(nq, nk, H, N, R, V, dtype):
    x = make(nq, nk, H, N, R, V, dtype, seed=sum(nq))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = run(x, status)
    assert int(status.item()) == 0
    verify(x, out, lse)


def test_many_sequences():
    n = [(i * 53) % 71 for i in range(500)]
    x = make(n, n, 1, 64, 16, 64, BF, seed=1)
    out, lse = run(x)
    verify(x, out, lse)


def test_queries_that_see_nothing():
    x = make([200, 40], [60, 0], 2, 128, 64, 128, BF, seed=2)
    out, lse = run(x)
    assert not out[:140].any() and (lse[:140] == -torch.inf).all()
    assert not out[200:].any() and (lse[200:] == -torch.inf).all()
    assert (lse[140:200] > -torch.inf).all()


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("n", [1, 100, 128, 300])
def test_a_neighbour_has_no_effect(junk, n):
    x = make([n, 50], [n, 50], 2, 128, 64, 128, BF, seed=3)
    want, want_lse = run(x)
    x["kv"][n:] = junk
    x["rot"][n:] = junk
    x["q"][n:] = junk
    out, lse = run(x)
    assert torch.equal(out[:n], want[:n]) and torch.equal(lse[:n], want_lse[:n])


@pytest.mark.parametrize("dtype", [BF, F16])
def test_scores_that_climb_and_fall(dtype):
    n, N, R = 700, 128, 64
    x = make([n], [n], 2, N, R, 128, dtype, seed=4, std=0.05)
    x["rot"][:, 0] = torch.linspace(-60, 60, n, device=DEV).to(dtype)
    x["q"][:, 0, N], x["q"][:, 1, N] = 20.0, -20.0
    out, lse = run(x)
    verify(x, out, lse)


def test_strides_and_tokens_of_no_sequence():
    H, N, R, V = 3, 64, 32, 128
    x = make([40, 129], [50, 129], H, N, R, V, F16, seed=5)
    want, want_lse = run(x)
    q = torch.zeros(H, 169 + 6, N + R + 8, dtype=F16, device=DEV).permute(1, 0, 2)[..., :N + R]
    q[:169] = x["q"]
    kv = torch.zeros(179, H + 1, N + V + 16, dtype=F16, device=DEV)[:, 1:, 8:8 + N + V]
    kv.copy_(x["kv"])
    rot = torch.zeros(179, R + 40, dtype=F16, device=DEV)[:, 32:32 + R]
    rot.copy_(x["rot"])
    obuf = torch.full((H, 175, V + 8), 5.0, dtype=F16, device=DEV)
    out = obuf.permute(1, 0, 2)[..., :V]
    lib.mtp_latent_prefill(q, kv, rot, x["cu_q"], x["cu_k"], out, x["scale"])
    assert torch.equal(out[:169], want)
    assert (out[169:] == 5.0).all() and (obuf[..., V:] == 5.0).all()


def test_bad_bounds_are_reported():
    x = make([100, 30], [100, 30], 1, 64, 16, 64, BF, seed=6)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for name, bad in (("cu_q", [0, 100, 131]), ("cu_k", [0, 100, 1 << 30]), ("cu_q", [-4, 100, 130]),
                      ("cu_k", [0, 100, 90])):
        y = dict(x)
        y[name] = torch.tensor(bad, dtype=torch.int32, device=DEV)
        status.zero_()
        out, lse = run(y, status)
        assert int(status.item()) == lib.STATUS_BAD_PARAM
        assert torch.isfinite(out).all()


def test_repeats_bit_for_bit_on_another_stream_and_captured():
    x = make([600, 31, 700], [900, 31, 700], 4, 128, 64, 128, BF, seed=7)
    want, want_lse = run(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = run(x, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    out.fill_(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.mtp_latent_prefill(x["q"], x["kv"], x["rot"], x["cu_q"], x["cu_k"], out, x["scale"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_no_queries_no_launch():
    x = make([5], [5], 1, 64, 16, 64, BF)
    n = lib.mtpspec_launch_count()
    lib.mtp_latent_prefill(x["q"][:0], x["kv"], x["rot"], x["cu_q"], x["cu_k"],
                           x["q"][:0, :, :64].contiguous(), 1.0)
    assert lib.mtpspec_launch_count() == n


def test_both_forms_agree():
    """The absorbed form over the cache gives what the expanded form gives over the same
    latents: with up-projections W_k and W_v, q . (W_k c) = (W_k^T q) . c."""
    g = torch.Generator(device=DEV).manual_seed(11)
    n, H, L, R, N, V, page = 333, 4, 512, 64, 128, 128, 64
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.float64)  # noqa: E731
    c, kr, q = rn(n, L).to(BF), rn(n, R).to(BF), rn(1, H, N + R).to(BF)
    wk, wv = rn(H, N, L) * L ** -0.5, rn(H, V, L) * L ** -0.5
    kv = torch.cat([torch.einsum("hnl,tl->thn", wk, c.double()),
                    torch.einsum("hvl,tl->thv", wv, c.double())], 2).to(BF)
    scale = (N + R) ** -0.5
    one = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    out = torch.empty(1, H, V, dtype=BF, device=DEV)
    lib.mtp_latent_prefill(q, kv, kr, one, one * n, out, scale)
    pages = -(-n // page)
    cache = torch.zeros(pages * page, L + R, dtype=BF, device=DEV)
    cache[:n] = torch.cat([c, kr], 1)
    qa = torch.cat([torch.einsum("hn,hnl->hl", q[0, :, :N].double(), wk).to(BF), q[0, :, N:]], 1)
    lat = torch.empty(1, 1, H, L, dtype=BF, device=DEV)
    ws = torch.empty(lib.mtp_latent_attn_workspace_bytes(1, 1, H, L, R), dtype=torch.uint8, device=DEV)
    lib.mtp_latent_attn(qa.view(1, 1, H, L + R), cache.view(pages, page, L + R),
                        torch.arange(pages, device=DEV).int()[None], one[1:] * n, lat, scale,
                        workspace=ws)
    got = torch.einsum("hl,hvl->hv", lat[0, 0].double(), wv)
    # both round weights, keys, values or latents to bf16 a few times: some 2^-8 of values of
    # size one each, averaged over the keys
    assert (got - out[0].double()).abs().max() < 8 * 2.0 ** -8


@pytest.mark.parametrize("heads,B,longest,V", [(16, 40, 300, 128), (48, 9, 520, 64), (152, 3, 257, 128), (7, 33, 600, 128)])
def test_more_pairs_than_multiprocessors(heads, B, longest, V):
    # queries that see nothing, sequences without keys or queries among them
    nq = [(37 * i + 11) % longest + 1 for i in range(B)]
    nk = [n + (53 * i) % 150 for i, n in enumerate(nq)]
    nq[1], nk[2], nk[B - 1] = 0, 0, max(1, nq[B - 1] - 140)
    x = make(nq, nk, heads, 128, 64, V, BF, seed=B)
    out, lse = run(x)
    verify(x, out, lse)
    again, _ = run(x)
    assert torch.equal(out, again)
