"""Timed cases of the draft head's attention with grouped heads over a paged cache of keys and
values: the cache's append with the heads' norms and rotation, the attention itself, and the
bookkeeping of the cache's pages.

A draft head's block may be one attention layer with Hq query heads and Hkv key heads, a key head
shared by Hq / Hkv query heads.  Its cache keeps D key and D value elements a token and key head,
in pages that rows hold through a block table.  The cases run from one drafted token of one row
to serving batches with D + 1 verified positions a row, chunks behind long texts and whole
prompts; the pages' cases are what happens to the table between two rounds of drafts.

`run` computes a case with elementary torch operations in 32 bits, or, where `own` is set, with
the library's entry points on the same inputs; `exact` has the same results in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one drafted token of one row: the append's latency
        dict(name="append_b1_t1_h32", op="append", B=1, T=1, H=32, Hkv=8, D=128, R=128, page=64,
             ctx=200, dtype="bf16", norm=True, pairs=False),
        # prompts written whole, wide heads of which a quarter is rotated; lengths that fill no page
        dict(name="append_b6_t1999_h16_f16", op="append", B=6, T=1999, H=16, Hkv=4, D=256, R=64,
             page=32, ctx=0, dtype="f16", norm=True, pairs=True),
        # one drafted token of one row over a short text: the attention's latency
        dict(name="attn_b1_t1_h32_n600", op="attn", B=1, lo=1, hi=1, plo=600, ctx=600, H=32, Hkv=8,
             D=128, page=64, window=0, sinks=0, dtype="bf16"),
        # the verify step of a 256-row serving batch, 3 drafts: bound by the cache's bytes
        dict(name="attn_b256_t4_h32_n4k", op="attn", B=256, lo=4, hi=4, plo=500, ctx=4000, H=32,
             Hkv=8, D=128, page=64, window=0, sinks=0, dtype="bf16"),
        # 64 rows of drafts with a sliding window and four first tokens that stay visible
        dict(name="attn_b64_t1_h64_w1k_s4", op="attn", B=64, lo=1, hi=1, plo=1000, ctx=16000, H=64,
             Hkv=8, D=64, page=16, window=1024, sinks=4, dtype="f16"),
        # the first pass over ragged prompts of a serving batch, admitted together
        dict(name="attn_b8_h32_n1500", op="attn", B=8, lo=77, hi=1500, plo=0, ctx=0, H=32, Hkv=4,
             D=128, page=16, window=0, sinks=0, dtype="bf16"),
        # a mixed batch: chunks of prompts behind what is cached beside rows of a few tokens,
        # five query heads a key head, pages that are no power of two
        dict(name="attn_b6_h40_n1000_p7k", op="attn", B=6, lo=1, hi=1000, plo=5, ctx=7001, H=40,
             Hkv=8, D=128, page=48, window=0, sinks=0, dtype="f16"),
        # one long prompt, wide heads
        dict(name="attn_b1_h16_d256_n8k", op="attn", B=1, lo=8192, hi=8192, plo=0, ctx=0, H=16,
             Hkv=2, D=256, page=128, window=0, sinks=0, dtype="bf16"),
        # between two rounds of a 256-row batch: rejected drafts' pages go back, new ones are taken
        dict(name="resize_b256_p16", op="resize", B=256, N=40000, page=16, ctx=2000, T=40),
        # one row branches into three drafts
        dict(name="fork_b1_f3", op="fork", B=1, F=3, N=600, page=64, ctx=1000, T=4, H=8, D=128),
        # every row of a 64-row batch branches into four drafts
        dict(name="fork_b64_f4", op="fork", B=64, F=4, N=4000, page=64, ctx=2000, T=8, H=4, D=128),
        # a cache that half emptied is moved together before it shrinks
        dict(name="compact_n8k", op="compact", B=128, N=8192, page=32, ctx=1200, H=4, D=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "attn", "attn", "attn", "pages"])
        if op == "pages":
            op = rng.choice(["resize", "fork", "compact"])
            page = rng.choice([8, 16, 32, 64, 48])
            ctx = _log(rng, 1, 4000)
            c = dict(op=op, B=_log(rng, 1, 256), page=page, ctx=ctx, T=rng.randrange(1, 64))
            if op == "resize":
                need = c["B"] * (-(-(ctx + c["T"]) // page) + 1)
                c["N"] = int(need * rng.uniform(1.0, 3.0)) + 1
                return c
            c |= dict(H=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 80]))
            rows = c["B"]
            if op == "fork":
                c["F"] = rng.randrange(1, 6)
                rows = c["B"] * (1 + c["F"])
            c["N"] = int(rows * (-(-(ctx + c["T"]) // page) + 1) * rng.uniform(1.0, 2.5)) + 2
            if c["N"] * page * c["H"] * c["D"] <= 160_000_000 and rows <= 1024:
                return c
            continue
        Hkv = rng.choice([1, 2, 4, 8, 8, 3])
        G = rng.choice([1, 2, 4, 4, 5, 7, 8, 8, 16])
        c = dict(op=op, H=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128, 128, 128, 256, 96]),
                 page=rng.choice([8, 16, 32, 64, 128, 48]), dtype=rng.choice(["bf16", "f16"]))
        if op == "append":
            c |= dict(B=_log(rng, 1, 256), T=_log(rng, 1, 1999), ctx=rng.randrange(0, 700),
                      R=rng.choice([c["D"], c["D"], 32, 64]), norm=rng.random() < 0.7,
                      pairs=rng.random() < 0.5)
            if c["B"] * c["T"] * (c["H"] + Hkv) * c["D"] <= 6 * 1999 * 20 * 256 and \
                    c["B"] * (c["T"] + c["ctx"]) * Hkv * c["D"] <= 40_000_000:
                return c
        else:
            ctx = _log(rng, 1, 100_000) if rng.random() < 0.8 else 0
            lo = _log(rng, 1, 4096)
            c |= dict(B=_log(rng, 1, 256), plo=int(ctx * rng.random()), ctx=ctx, lo=1 if rng.random() < 0.4 else lo,
                      hi=lo, window=rng.choice([0, 0, _log(rng, 1, 4096)]))
            c["sinks"] = rng.choice([0, 4, 64, _log(rng, 1, 300)]) if c["window"] else 0
            if c["hi"] == 1 and not ctx:
                continue
            if c["B"] * c["hi"] * c["H"] * (ctx + c["hi"]) * max(c["D"], 128) <= 8192 * 8192 * 16 * 256 and \
                    c["B"] * (ctx + c["hi"]) * Hkv * c["D"] <= 256 * 4000 * 8 * 128:
                return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 23)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _rows(case):
    """The rows' new tokens and the texts before them: the same for every seed, which shuffles
    them."""
    r = random.Random(case["B"] * 65537 + case["hi"] * 257 + case["ctx"])
    n = [(case["hi"], case["ctx"])]
    while len(n) < case["B"]:
        n.append((r.randint(case["lo"], case["hi"]), r.randint(case["plo"], case["ctx"])))
    return n


def _table(g, B, per_row):
    """A block table of B rows over shuffled pages, with a few pages that no row holds."""
    pages = B * per_row + 3
    order = torch.randperm(pages, generator=g, device="cuda")[:B * per_row]
    return pages, order.reshape(B, per_row).to(torch.int32)


def _angles(n, R):
    """[n, R]: the cosines, then the sines, of every position's R / 2 angles, stretched for long
    texts as position interpolation does."""
    f = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R) / 4
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _lens(case, g, n):
    """n lengths up to ctx, the first of them ctx."""
    x = torch.randint(1, case["ctx"] + 1, (n,), generator=g, device="cuda")
    x[0] = case["ctx"]
    return x.int()


def _held_table(g, B, N, held, wide):
    """Rows that hold pages of their own out of N, shuffled; -1 behind them."""
    order = torch.randperm(N, generator=g, device="cuda").int()
    at = torch.arange(wide, device="cuda")
    mine = at < held[:, None]
    place = (held.cumsum(0) - held)[:, None] + at
    table = torch.where(mine, order[place.clamp(max=N - 1)], -1)
    return table.int().contiguous(), _counts(table, held, N)


def _counts(table, held, N):
    """How many table entries hold each page."""
    mine = torch.arange(table.shape[1], device="cuda") < held[:, None]
    return torch.bincount(table[mine].long(), minlength=N).int()


def _pages_state(case, g):
    B, N, P = case["B"], case["N"], case["page"]
    lens = _lens(case, g, B)
    wide = -(-(case["ctx"] + case.get("T", 1)) // P) + 1
    if case["op"] == "resize":
        # rows hold pages for what was drafted; `keep` of it was accepted
        keep = (lens - torch.randint(0, case["T"] + 1, (B,), generator=g, device="cuda")).clamp(min=0).int()
        held = -(-lens // P)
        table, refs = _held_table(g, B, N, held, wide)
        return dict(case=case, keep=keep, lens=keep + case["T"], table=table, held=held.int(), refs=refs,
                    copies=_int([[0, 0]] * B))
    if case["op"] == "fork":
        # sources first; a row of a branch may still hold a page from before
        F = case["F"]
        held = torch.cat([-(-lens // P), torch.randint(0, 2, (B * F,), generator=g, device="cuda")]).int()
        table, refs = _held_table(g, B * (1 + F), N, held, wide)
        src = torch.arange(B, device="cuda").repeat_interleave(F).int()
        dst = (B + torch.randperm(B * F, generator=g, device="cuda")).int()
        keep = torch.zeros(B * (1 + F), dtype=torch.int32, device="cuda")
        keep[:B] = lens
        keep[dst.long()] = lens[src.long()]
        more = dict(src=src, dst=dst, keep=keep, lens=keep + case["T"], copies=_int([[0, 0]] * (B * (1 + F))))
    else:
        # rows that hold pages all over the cache; every other row shares the first half of the
        # pages of the one before it
        held = (-(-lens // P)).int()
        table, _ = _held_table(g, B, N, held, wide)
        half = held[0:B - 1:2] // 2
        half = torch.minimum(half, held[1::2])
        part = torch.arange(wide, device="cuda") < half[:, None]
        table[1::2] = torch.where(part, table[0:B - 1:2], table[1::2])
        more = dict(table0=table.clone(), moves=_int([[0, 0]] * (N // 2)).view(N // 2, 2), n_moves=_int([0]))
        refs = _counts(table, held, N)
        more["refs0"] = refs.clone()
    shape = (N, P, case["H"], case["D"])
    return dict(case=case, table=table, held=held, refs=refs, k=_normal(g, shape, torch.bfloat16),
                v=_normal(g, shape, torch.bfloat16)) | more


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("resize", "fork", "compact"):
        return _pages_state(case, g)
    dt, H, Hkv, D, B, P = (DTYPES[case["dtype"]], case["H"], case["Hkv"], case["D"], case["B"], case["page"])
    if case["op"] == "append":
        T = case["T"]
        longest = case["ctx"] + T
        pages, table = _table(g, B, -(-longest // P))
        start = torch.randint(0, case["ctx"] + 1, (B,), generator=g, device="cuda")
        pos = (start[:, None] + torch.arange(T, device="cuda")).reshape(-1).to(torch.int32)
        # one projection gives a token's queries, keys and values side by side
        qkv = _normal(g, (B * T, H + 2 * Hkv, D), dt)

        def weight():
            return (1 + _normal(g, (D,), torch.float32, 0.1)).to(dt) if case["norm"] else None
        return dict(case=case, q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:], q_norm=weight(),
                    k_norm=weight(), cos_sin=_angles(longest, case["R"]),
                    row=torch.arange(B, device="cuda", dtype=torch.int32).repeat_interleave(T),
                    positions=pos, table=table, q_out=torch.empty(B * T, H, D, dtype=dt, device="cuda"),
                    k_cache=_normal(g, (pages, P, Hkv, D), dt), v_cache=_normal(g, (pages, P, Hkv, D), dt))
    n = torch.tensor(_rows(case), dtype=torch.int32, device="cuda")
    n = n[torch.randperm(B, generator=g, device="cuda")]
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1:] = n[:, 0].cumsum(0)
    pages, table = _table(g, B, -(-(case["hi"] + case["ctx"]) // P))
    return dict(case=case, cu=cu, kv_len=n.sum(1).int(), table=table, scale=D ** -0.5,
                q=_normal(g, (int(cu[-1]), H, D), dt), k_cache=_normal(g, (pages, P, Hkv, D), dt),
                v_cache=_normal(g, (pages, P, Hkv, D), dt))


# ---------------------------------------------------------------- one pass

def _rotate(x, cos, sin, pairs):
    """The rotation of the last axis by (neighbouring or half-way) pairs, in x's type."""
    if pairs:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_append(s):
    case, P, R = s["case"], s["case"]["page"], s["case"]["R"]
    pos = s["positions"].long()
    cos, sin = s["cos_sin"][pos][:, None].chunk(2, -1)

    def heads(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
        return torch.cat([_rotate(x[..., :R], cos, sin, case["pairs"]), x[..., R:]], -1)
    page = s["table"][s["row"].long(), pos // P].long()
    s["k_cache"][page, pos % P] = heads(s["k"], s["k_norm"]).to(s["k_cache"].dtype)
    s["v_cache"][page, pos % P] = s["v"]
    s["q_out"].copy_(heads(s["q"], s["q_norm"]))
    return {"k": s["k_cache"], "v": s["v_cache"], "q": s["q_out"]}


def _plain_attn(s):
    case, q, cu = s["case"], s["q"], s["cu"].long()
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    G = case["H"] // Hkv
    mq, kv_len = case["hi"], s["kv_len"].long()
    new = cu.diff()
    i = torch.arange(mq, device="cuda")
    mine = i < new[:, None]                                                       # [B, mq]
    tok = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    keys = s["k_cache"][s["table"].long()].reshape(B, -1, Hkv, D).float()
    vals = s["v_cache"][s["table"].long()].reshape(B, -1, Hkv, D).float()
    at = torch.arange(keys.shape[1], device="cuda")
    vals = vals.masked_fill((at >= kv_len[:, None])[..., None, None], 0.0)
    qp = q.float()[tok].view(B, mq, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, mq * G, D)
    sc = qp @ keys.permute(0, 2, 3, 1)                                            # [B, Hkv, mq*G, n]
    sc *= s["scale"]
    pos = (kv_len - new)[:, None] + i                                             # [B, mq]
    hidden = at > pos[..., None]
    if case["window"]:
        hidden |= (at <= pos[..., None] - case["window"]) & (at >= case["sinks"])
    hidden = hidden.repeat_interleave(G, 1)[:, None]
    sc.masked_fill_(hidden, -math.inf)
    top = sc.amax(-1, keepdim=True)
    sc -= torch.where(top > -math.inf, top, 0.0)
    p = sc.exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ vals.transpose(1, 2)) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).view(B, Hkv, mq, G).transpose(1, 2).reshape(B, mq, case["H"])
    o = o.view(B, Hkv, mq, G, D).transpose(1, 2).reshape(B, mq, case["H"], D)
    return {"out": o[mine].to(q.dtype), "lse": lse[mine]}


def _plain_resize(s):
    """Every row keeps the pages of its first `keep` positions, has the last of them for itself if
    it is partly filled, and takes pages for `lens` positions: the lowest free ones, row by row."""
    table, held, refs, P = s["table"], s["held"], s["refs"], s["case"]["page"]
    B, wide = table.shape
    N = refs.shape[0]
    rows, at = torch.arange(B, device="cuda"), torch.arange(wide, device="cuda")
    kept = (s["keep"] + (P - 1)) // P
    want = (s["lens"] + (P - 1)) // P
    gone = (at >= kept[:, None]) & (at < held[:, None])
    refs.index_add_(0, table[gone], torch.full_like(table[gone], -1))
    table[gone] = -1
    # the last kept page, partly filled and held by others too: the lowest of its rows keeps it
    # if all of them are such rows, the others leave it
    last = table.gather(1, (kept - 1).clamp(min=0).long()[:, None])[:, 0].long()
    partly = (kept > 0) & (s["keep"] % P != 0)
    shared = partly & (refs[last.clamp(min=0)] > 1)
    page = torch.where(shared, last, N)                                           # N: none
    writers = torch.zeros(N + 1, dtype=torch.int32, device="cuda").index_add_(0, page, shared.int())
    first = torch.full((N + 1,), B, device="cuda").scatter_reduce(0, page, rows, "amin")
    all_write = writers[:N] == refs
    leaves = shared & ~(all_write[last.clamp(min=0)] & (first[page] == rows))
    need = (want - kept).clamp(min=0) + leaves
    end = need.cumsum(0)
    free = (refs == 0).nonzero()[:, 0].int()
    got = end <= free.shape[0]
    leaves = leaves & got
    refs.index_add_(0, last[leaves], torch.full_like(last[leaves], -1, dtype=torch.int32))
    grown = (at >= kept[:, None]) & (at < want[:, None]) & got[:, None]
    take = grown | ((at == kept[:, None] - 1) & leaves[:, None])
    place = (end - need)[:, None] + take.cumsum(1) - 1
    fresh = free[place[take]] if free.shape[0] else free[:0]
    table[take] = fresh
    refs[fresh.long()] = 1
    mine = table.gather(1, (kept - 1).clamp(min=0).long()[:, None])[:, 0]
    s["copies"].copy_(torch.where(leaves[:, None], torch.stack([last.int(), mine], 1), -1))
    held.copy_(torch.where(got, torch.maximum(kept, want), kept))


def _plain_fork(s):
    """Every dst row leaves its pages and shares those of its src row."""
    table, held, refs, src, dst = s["table"], s["held"], s["refs"], s["src"].long(), s["dst"].long()
    at = torch.arange(table.shape[1], device="cuda")
    old = table[dst][at < held[dst][:, None]]
    refs.index_add_(0, old, torch.full_like(old, -1))
    mine = at < held[src][:, None]
    table[dst] = torch.where(mine, table[src], -1)
    held[dst] = held[src]
    new = table[dst][mine]
    refs.index_add_(0, new, torch.ones_like(new))


def _plain_copy(s, pairs):
    pairs = pairs[pairs[:, 0] >= 0].long()
    s["k"][pairs[:, 1]] = s["k"][pairs[:, 0]]
    s["v"][pairs[:, 1]] = s["v"][pairs[:, 0]]


def _plain_compact(s):
    """The pages above the number of live ones move into the holes below it, in order."""
    table, refs, moves = s["table"], s["refs"], s["moves"]
    live = refs > 0
    L = live.sum()
    ids = torch.arange(refs.shape[0], device="cuda")
    holes, movers = (~live & (ids < L)).nonzero()[:, 0], (live & (ids >= L)).nonzero()[:, 0]
    n = holes.shape[0]
    moves.fill_(-1)
    moves[:n, 0] = movers.int()
    moves[:n, 1] = holes.int()
    s["n_moves"].fill_(n)
    to = ids.int()
    to[movers] = holes.int()
    mine = torch.arange(table.shape[1], device="cuda") < s["held"][:, None]
    table.copy_(torch.where(mine, to[table.clamp(min=0).long()], table))
    refs[holes] = refs[movers]
    refs[movers] = 0


def _own_buffers(s, lib):
    """The outputs and the workspace that a program keeps from call to call."""
    if "out" not in s:
        q, c = s["q"], s["case"]
        s["out"] = torch.empty_like(q)
        s["lse"] = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
        n = lib.mtp_heads_attn_workspace_bytes(c["B"], q.shape[0], c["H"], c["Hkv"], c["D"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s["out"], s["lse"], s["workspace"]


def _own(s):
    import verify_spec_greedy_gb300 as lib
    case = s["case"]
    if case["op"] == "append":
        lib.mtp_heads_append(s["k"], s["v"], s["cos_sin"], s["row"], s["positions"], s["table"],
                             s["k_cache"], s["v_cache"], k_norm_w=s["k_norm"], q=s["q"],
                             q_out=s["q_out"], q_norm_w=s["q_norm"], eps=EPS, interleaved=case["pairs"])
        return {"k": s["k_cache"], "v": s["v_cache"], "q": s["q_out"]}
    if case["op"] == "attn":
        out, lse, workspace = _own_buffers(s, lib)
        lib.mtp_heads_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"], out,
                           s["scale"], window=case["window"], sinks=case["sinks"], lse=lse,
                           workspace=workspace)
        return {"out": out, "lse": lse}
    if case["op"] == "compact":
        lib.mtp_pages_compact(s["table"], s["held"], s["refs"], s["moves"], s["n_moves"])
        lib.mtp_pages_copy([s["k"], s["v"]], s["moves"], n_pairs=s["n_moves"])
        return None
    if case["op"] == "fork":
        lib.mtp_pages_fork(s["src"], s["dst"], s["table"], s["held"], s["refs"])
    lib.mtp_pages_resize(s["keep"], s["lens"], s["table"], s["held"], s["refs"], case["page"], s["copies"])
    if case["op"] == "fork":
        lib.mtp_pages_copy([s["k"], s["v"]], s["copies"])
    return None


def run(state):
    s, op = state, state["case"]["op"]
    if op == "compact":  # a pass moves together what the pass before it left moved together
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
    if own:
        out = _own(s)
    elif op == "append":
        out = _plain_append(s)
    elif op == "attn":
        out = _plain_attn(s)
    else:
        out = None
        if op == "compact":
            _plain_compact(s)
            _plain_copy(s, s["moves"])
        else:
            if op == "fork":
                _plain_fork(s)
            _plain_resize(s)
            if op == "fork":
                _plain_copy(s, s["copies"])
    if out is None:
        names = {"resize": ("table", "held", "refs", "copies"), "fork": ("table", "held", "refs", "copies", "k", "v"),
                 "compact": ("table", "refs", "moves", "n_moves", "k", "v")}[op]
        out = {n: s[n] for n in names}
    return out


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    B, P = case["B"], case["page"]
    if case["op"] == "append":
        n, H, Hkv, D, R = B * case["T"], case["H"], case["Hkv"], case["D"], case["R"]
        # queries, keys and values in and out, the angles of each position, its row, position and page
        return {"bytes": n * (2 * 2 * (H + 2 * Hkv) * D + 4 * R + 12),
                "flops": n * (H + Hkv) * (4 * D * case["norm"] + 3 * R)}
    if case["op"] == "attn":
        D, w, pairs, keys, toks = case["D"], case["window"], 0, 0, 0
        for new, before in _rows(case):
            toks += new
            # the last query sees the most; with a window, `w` keys and the first ones
            first, sinks = (max(0, before + 1 - w), case["sinks"]) if w else (0, 0)
            keys += before + new - first + min(first, sinks)
            for i in range(new):
                at = before + i + 1
                pairs += min(at, w + min(sinks, max(0, at - w))) if w else at
        return {"bytes": int(toks * case["H"] * (4 * D + 4) + keys * case["Hkv"] * 4 * D + 8 * B + 4 * keys // P),
                "flops": int(pairs * case["H"] * 4 * D)}
    # the pages' lengths depend on the seed: half of the longest each, on average
    per = case["ctx"] // 2 // P + 1
    page_bytes = 2 * 2 * P * case.get("H", 0) * case.get("D", 0)
    if case["op"] == "resize":
        return {"bytes": 4 * (B * 5 + case["N"] + B * 2 * (case["T"] // P + 1)), "flops": B}
    if case["op"] == "fork":
        n = B * case["F"]
        return {"bytes": n * (2 * page_bytes + 4 * 4 * per) + 4 * (case["N"] + 7 * (n + B)), "flops": n}
    live = B * per * 3 // 4
    moved = live * max(0, case["N"] - live) // case["N"]
    return {"bytes": moved * (2 * page_bytes + 16) + 4 * (2 * case["N"] + 2 * B * per), "flops": case["N"]}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_rotation(x, angle_row, pairs):
    """Complex multiplication by e^(i angle), the angle's cosine and sine as tabulated."""
    half = x.shape[-1] // 2
    turn = torch.complex(angle_row[..., :half].double(), angle_row[..., half:].double())
    z = x.double()
    z = torch.view_as_complex(z.unflatten(-1, (half, 2)).contiguous()) if pairs else \
        torch.complex(z[..., :half].contiguous(), z[..., half:].contiguous())
    z = torch.view_as_real(z * turn)
    return z.flatten(-2) if pairs else torch.cat([z[..., 0], z[..., 1]], -1)


def _exact_append(s):
    case, P, R, B, Hkv, D = (s["case"], *(s["case"][k] for k in ("page", "R", "B", "Hkv", "D")))
    turn = s["cos_sin"].index_select(0, s["positions"])[:, None]

    def heads(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
        turned = _exact_rotation(x[..., :R], turn.expand(-1, x.shape[1], -1), case["pairs"])
        return torch.cat([turned, x[..., R:]], -1)
    flat = s["table"].long().gather(1, (s["positions"].long() // P).reshape(B, -1)).reshape(-1) * P \
        + s["positions"].long() % P
    k, v = s["k_cache"].double(), s["v_cache"].double()
    k.view(-1, Hkv, D)[flat] = heads(s["k"], s["k_norm"])
    v.view(-1, Hkv, D)[flat] = s["v"].double()
    return {"k": k, "v": v, "q": heads(s["q"], s["q_norm"])}


def _exact_attn(s):
    case, G = s["case"], s["case"]["H"] // s["case"]["Hkv"]
    outs, sums = [], []
    for b in range(case["B"]):
        q = s["q"][s["cu"][b]:s["cu"][b + 1]]
        n = int(s["kv_len"][b])
        pages = s["table"][b].long()
        keys, vals = (s[c][pages].flatten(0, 1)[:n].double() for c in ("k_cache", "v_cache"))
        pos = torch.arange(n - len(q), n, device="cuda")
        back = pos[:, None] - torch.arange(n, device="cuda")        # how far back a key lies
        seen = back >= 0
        if case["window"]:
            seen &= (back < case["window"]) | (torch.arange(n, device="cuda") < case["sinks"])
        o, l = [], []
        for h in range(case["H"]):
            sc = torch.where(seen, q[:, h].double() @ keys[:, h // G].T * s["scale"], -math.inf)
            lse = torch.logsumexp(sc, -1)
            o.append(torch.exp(sc - lse[:, None]) @ vals[:, h // G])
            l.append(lse)
        outs.append(torch.stack(o, 1))
        sums.append(torch.stack(l, 1))
    return {"out": torch.cat(outs), "lse": torch.cat(sums)}


def _exact_pages(s):
    """One page after another, on the host."""
    case, op, P = s["case"], s["case"]["op"], s["case"]["page"]
    table, refs, held = s["table"].tolist(), s["refs"].tolist(), s["held"].tolist()
    pairs = []

    def leave(b, i):
        refs[table[b][i]] -= 1
        table[b][i] = -1
    if op == "compact":
        live = sum(r > 0 for r in refs)
        movers = [i for i, r in enumerate(refs) if r > 0 and i >= live]
        holes = [i for i in range(live) if refs[i] == 0]
        to = dict(zip(movers, holes))
        table = [[to.get(p, p) for p in t] for t in table]
        for a, b in to.items():
            refs[b], refs[a] = refs[a], 0
        pairs = list(to.items())
        out = {"moves": pairs + [(-1, -1)] * (case["N"] // 2 - len(pairs)), "n_moves": [len(pairs)]}
    else:
        if op == "fork":
            for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
                for i in range(held[b]):
                    leave(b, i)
                held[b] = held[a]
                for i in range(held[a]):
                    table[b][i] = table[a][i]
                    refs[table[a][i]] += 1
        keep, lens = s["keep"].tolist(), s["lens"].tolist()
        kept = [-(-k // P) for k in keep]
        for b, k in enumerate(kept):
            for i in range(k, held[b]):
                leave(b, i)
            held[b] = k
        writers = {}
        for b, k in enumerate(keep):
            if k % P:
                writers.setdefault(table[b][kept[b] - 1], []).append(b)
        leaving = {b for p, w in writers.items() if refs[p] > 1 for b in (w[1:] if len(w) == refs[p] else w)}
        free = [i for i, r in enumerate(refs) if r == 0]
        used, copies, short = 0, [], False
        for b in range(len(table)):
            need = max(0, -(-lens[b] // P) - kept[b]) + (b in leaving)
            short |= used + need > len(free)
            copy = (-1, -1)
            if not short:
                new = free[used:used + need]
                used += need
                if b in leaving:
                    old = table[b][kept[b] - 1]
                    refs[old] -= 1
                    table[b][kept[b] - 1] = new[0]
                    refs[new[0]] = 1
                    copy = (old, new.pop(0))
                for i, p in enumerate(new):
                    table[b][kept[b] + i] = p
                    refs[p] = 1
                held[b] = kept[b] + len(new)
            copies.append(copy)
        pairs = [c for c in copies if c[0] >= 0]
        out = {"copies": copies, "held": held}
    out |= {"table": table, "refs": refs}
    out = {n: torch.tensor(x, dtype=torch.int32, device="cuda").view(s[n].shape) for n, x in out.items()}
    if op != "resize":
        for n in ("k", "v"):
            out[n] = s[n].clone()
            if pairs:
                out[n][[b for _, b in pairs]] = s[n][[a for a, _ in pairs]]
            out[n] = out[n].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn}.get(case["op"], _exact_pages)(s)
