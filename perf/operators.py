"""Timed cases of the draft head's latent attention: the paged cache's append, the attention
over that cache (absorbed form) and the attention over a prompt (expanded form).

A token keeps one latent vector of L values, shared by every head, and R values that carry
its position; the cache holds the L + R values of a token in one row, in pages.  The cases
run from one drafted token of one row to a serving batch with D + 1 verified positions a
row, and from short prompts to long ones.

`run` computes a case with elementary torch operations in 32 bits, or, where `own` is set,
with the library's entry points on the same inputs; `exact` has the same results in 64 bits.
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
        dict(name="append_b1_t1_h16", op="append", B=1, T=1, H=16, L=512, R=64, page=64,
             ctx=200, dtype="bf16", norm=True, pairs=True),
        # the verify step of a serving batch (256 rows, 3 drafts): 1024 tokens, 128 heads'
        # queries rotated on the way
        dict(name="append_b256_t4_h128", op="append", B=256, T=4, H=128, L=512, R=64, page=64,
             ctx=500, dtype="bf16", norm=True, pairs=True),
        # a prompt written whole, rotated by halves; lengths that fill no page
        dict(name="append_b6_t1999_h32_f16", op="append", B=6, T=1999, H=32, L=512, R=64,
             page=32, ctx=0, dtype="f16", norm=True, pairs=False),
        # one drafted token of one row over a short text: the attention's latency
        dict(name="attn_b1_t1_h16_n600", op="attn", B=1, T=1, H=16, L=512, R=64, page=64,
             lo=600, hi=600, dtype="bf16"),
        # the 8-row verify workload, 3 drafts, ragged texts
        dict(name="attn_b8_t4_h16_n2k", op="attn", B=8, T=4, H=16, L=512, R=64, page=16,
             lo=301, hi=2047, dtype="bf16"),
        # the 256-row serving batch with 3 drafts and few heads: bound by the cache's bytes
        dict(name="attn_b256_t4_h16_n4k", op="attn", B=256, T=4, H=16, L=512, R=64, page=64,
             lo=500, hi=4000, dtype="bf16"),
        # 64 rows, one draft, all 128 heads on one GPU: bound by the products
        dict(name="attn_b64_t2_h128_n8k", op="attn", B=64, T=2, H=128, L=512, R=64, page=64,
             lo=1000, hi=8000, dtype="f16"),
        # one row with 6 drafts deep in a long text
        dict(name="attn_b1_t7_h24_n100k", op="attn", B=1, T=7, H=24, L=512, R=64, page=128,
             lo=100001, hi=100001, dtype="bf16"),
        # the draft head's first pass over a short prompt: latency
        dict(name="prefill_b1_h16_n300", op="prefill", B=1, H=16, N=128, R=64, V=128,
             lo=300, hi=300, prefix=0, dtype="bf16"),
        # ragged prompts of a serving batch, admitted together
        dict(name="prefill_b8_h32_n1500", op="prefill", B=8, H=32, N=128, R=64, V=128,
             lo=77, hi=1500, prefix=0, dtype="bf16"),
        # a prompt's next chunk behind what is already cached
        dict(name="prefill_b2_h16_n1000_p7k", op="prefill", B=2, H=16, N=128, R=64, V=128,
             lo=900, hi=1000, prefix=7001, dtype="f16"),
        # one long prompt
        dict(name="prefill_b1_h32_n8k", op="prefill", B=1, H=32, N=128, R=64, V=128,
             lo=8192, hi=8192, prefix=0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "attn", "attn", "prefill"])
        c = dict(op=op, H=rng.choice([_log(rng, 1, 128), 16, 32, 128]), R=rng.choice([64, 64, 32]),
                 dtype=rng.choice(["bf16", "f16"]))
        if op == "append":
            c |= dict(B=_log(rng, 1, 256), T=_log(rng, 1, 1999), L=rng.choice([512, 512, 256]),
                      page=rng.choice([16, 32, 64, 128]), ctx=rng.randrange(0, 700),
                      norm=rng.random() < 0.7, pairs=rng.random() < 0.5)
            if c["B"] * c["T"] <= 6 * 1999 and c["B"] * c["T"] * c["H"] <= 6 * 1999 * 32:
                return c
        elif op == "attn":
            hi = _log(rng, 1, 100000)
            c |= dict(B=_log(rng, 1, 256), T=rng.choice([1, 2, 3, 4, 5, 7]),
                      L=rng.choice([512, 512, 256]), page=rng.choice([16, 32, 64, 128, 48]),
                      lo=max(1, int(hi * rng.random())), hi=hi)
            if c["B"] * c["T"] * c["H"] * c["hi"] <= 64 * 2 * 128 * 8000 and \
                    c["B"] * c["hi"] <= 256 * 4000:
                return c
        else:
            hi = _log(rng, 2, 8192)
            c |= dict(B=_log(rng, 1, 16), N=rng.choice([128, 128, 64]), V=rng.choice([128, 128, 64]),
                      lo=max(1, int(hi * rng.random())), hi=hi,
                      prefix=rng.choice([0, 0, rng.randrange(1, 7002)]))
            if c["B"] * c["H"] * c["hi"] * (c["hi"] + c["prefix"]) <= 32 * 8192 * 8192:
                return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _lengths(case):
    """The rows' lengths: the same ones for every seed, which shuffles them."""
    r = random.Random(case["B"] * 65537 + case["lo"] * 257 + case["hi"])
    return [case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(case["B"] - 1)]


def _shuffled_lengths(g, case):
    n = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    return n[torch.randperm(case["B"], generator=g, device="cuda")]


def _table(g, B, per_row):
    """A block table of B rows over shuffled pages, with a few pages that no row holds."""
    pages = B * per_row + 3
    order = torch.randperm(pages, generator=g, device="cuda")[:B * per_row]
    return pages, order.reshape(B, per_row).to(torch.int32)


def _angles(n, R):
    """[n, R]: the cosines, then the sines, of every position's R / 2 angles."""
    f = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    H, R = case["H"], case["R"]
    if case["op"] == "append":
        B, T, L, P = case["B"], case["T"], case["L"], case["page"]
        longest = case["ctx"] + T
        pages, table = _table(g, B, -(-longest // P))
        start = torch.randint(0, case["ctx"] + 1, (B,), generator=g, device="cuda")
        pos = (start[:, None] + torch.arange(T, device="cuda")).reshape(-1).to(torch.int32)
        row = torch.arange(B, device="cuda", dtype=torch.int32).repeat_interleave(T)
        # the down-projection's output holds a token's latent and its rotated part in one
        # row; the query's rotated part is a slice of the query projection's output
        down = _normal(g, (B * T, L + R), dt)
        qproj = _normal(g, (B * T, H, 128 + R), dt)
        return dict(case=case, latent=down[:, :L], rot=down[:, L:], q_rot=qproj[..., 128:],
                    norm_w=(1 + _normal(g, (L,), torch.float32, 0.1)).to(dt) if case["norm"] else None,
                    cos_sin=_angles(longest, R), tok_row=row, positions=pos, table=table,
                    cache=_normal(g, (pages, P, L + R), dt),
                    q_out=_normal(g, (B * T, H, L + R), dt))
    if case["op"] == "attn":
        B, T, L, P = case["B"], case["T"], case["L"], case["page"]
        kv_len = _shuffled_lengths(g, case)
        pages, table = _table(g, B, -(-case["hi"] // P))
        return dict(case=case, kv_len=kv_len, table=table, scale=(128 + R) ** -0.5,
                    cache=_normal(g, (pages, P, L + R), dt),
                    q=_normal(g, (B, T, H, L + R), dt))
    n = _shuffled_lengths(g, case)
    cu_q = torch.zeros(case["B"] + 1, dtype=torch.int32, device="cuda")
    cu_q[1:] = n.cumsum(0)
    cu_k = torch.zeros_like(cu_q)
    cu_k[1:] = (n + case["prefix"]).cumsum(0)
    nq, nk = int(cu_q[-1]), int(cu_k[-1])
    return dict(case=case, cu_q=cu_q, cu_k=cu_k, scale=(case["N"] + R) ** -0.5,
                q=_normal(g, (nq, H, case["N"] + R), dt),
                kv=_normal(g, (nk, H, case["N"] + case["V"]), dt),
                rot=_normal(g, (nk, R), dt))


# ---------------------------------------------------------------- one pass

def _rotate(x, cos, sin, pairs):
    """The rotation of the last axis by (neighbouring or half-way) pairs, in x's type."""
    if pairs:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_append(s):
    case, cache, q_out = s["case"], s["cache"], s["q_out"]
    L, R, P = case["L"], case["R"], case["page"]
    c = s["latent"].float()
    if s["norm_w"] is not None:
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["norm_w"].float()
    pos = s["positions"].long()
    cos, sin = s["cos_sin"][pos].chunk(2, -1)
    k = _rotate(s["rot"].float(), cos, sin, case["pairs"])
    page = s["table"][s["tok_row"].long(), pos // P].long()
    cache[page, pos % P] = torch.cat([c, k], -1).to(cache.dtype)
    q_out[..., L:] = _rotate(s["q_rot"].float(), cos[:, None], sin[:, None], case["pairs"]).to(q_out.dtype)
    return {"cache": cache, "q": q_out}


def _softmax_rows(s, hidden):
    """(weights, sum, log of the sum) of the scores' last axis; empty rows weigh nothing."""
    s = s.masked_fill(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    return p, torch.where(total > 0, total, 1.0), (top + torch.log(total)).squeeze(-1)


def _plain_attn(s):
    case, q = s["case"], s["q"]
    B, T, H, W = q.shape
    L = case["L"]
    keys = s["cache"][s["table"].long()].reshape(B, -1, W).float()
    at = torch.arange(keys.shape[1], device="cuda")
    keys = keys.masked_fill((at >= s["kv_len"][:, None])[..., None], 0.0)
    seen = s["kv_len"][:, None] - (T - 1 - torch.arange(T, device="cuda"))        # [B, T]
    hidden = (at >= seen[..., None]).repeat_interleave(H, 1)                      # [B, T*H, n]
    p, total, lse = _softmax_rows(q.float().reshape(B, T * H, W) @ keys.transpose(1, 2) * s["scale"], hidden)
    out = (p @ keys[..., :L]) / total
    return {"out": out.reshape(B, T, H, L).to(q.dtype), "lse": lse.reshape(B, T, H)}


def _plain_prefill(s):
    case, q = s["case"], s["q"]
    N, B, H = case["N"], case["B"], case["H"]
    nq, nk = s["cu_q"].diff(), s["cu_k"].diff()
    mq, mk = case["hi"], case["hi"] + case["prefix"]
    iq, ik = torch.arange(mq, device="cuda"), torch.arange(mk, device="cuda")
    tq = (s["cu_q"][:-1, None] + iq).clamp(max=q.shape[0] - 1).long()             # [B, mq]
    tk = (s["cu_k"][:-1, None] + ik).clamp(max=s["kv"].shape[0] - 1).long()       # [B, mk]
    qp = q.float()[tq].transpose(1, 2)                                            # [B, H, mq, N+R]
    kv = s["kv"].float()[tk].transpose(1, 2)                                      # [B, H, mk, N+V]
    rot = s["rot"].float()[tk][:, None]                                           # [B, 1, mk, R]
    sc = qp[..., :N] @ kv[..., :N].transpose(2, 3)
    sc += qp[..., N:] @ rot.transpose(2, 3)
    sc *= s["scale"]
    hidden = ik > iq[:, None] + (nk - nq)[:, None, None]                          # [B, mq, mk]
    hidden = hidden | (ik >= nk[:, None])[:, None]
    p, total, lse = _softmax_rows(sc, hidden[:, None])
    o = (p @ kv[..., N:]) / total
    mine = iq < nq[:, None]                                                       # [B, mq]
    return {"out": o.transpose(1, 2)[mine].to(q.dtype), "lse": lse.transpose(1, 2)[mine]}


def _buffers(s, lib):
    """The outputs and workspace that a program keeps from call to call."""
    case = s["case"]
    if "out" not in s:
        q = s["q"]
        wide = case["L"] if case["op"] == "attn" else case["V"]
        s["out"] = torch.empty(q.shape[:-1] + (wide,), dtype=q.dtype, device="cuda")
        s["lse"] = torch.empty(q.shape[:-1], dtype=torch.float32, device="cuda")
        if case["op"] == "attn":
            B, T, H, _ = q.shape
            n = lib.mtp_latent_attn_workspace_bytes(B, T, H, case["L"], case["R"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s["out"], s["lse"], s.get("workspace")


def _own(s):
    import verify_spec_greedy_gb300 as lib
    case = s["case"]
    if case["op"] == "append":
        L = case["L"]
        lib.mtp_latent_append(s["latent"], s["rot"], s["cos_sin"], s["tok_row"], s["positions"],
                              s["table"], s["cache"], norm_w=s["norm_w"], eps=EPS,
                              interleaved=case["pairs"], q_rot=s["q_rot"], q_out=s["q_out"][..., L:])
        return {"cache": s["cache"], "q": s["q_out"]}
    out, lse, workspace = _buffers(s, lib)
    if case["op"] == "attn":
        lib.mtp_latent_attn(s["q"], s["cache"], s["table"], s["kv_len"], out, s["scale"], lse=lse,
                            workspace=workspace)
    else:
        lib.mtp_latent_prefill(s["q"], s["kv"], s["rot"], s["cu_q"], s["cu_k"], out, s["scale"],
                               lse=lse)
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attn": _plain_attn,
            "prefill": _plain_prefill}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    H, R, B = case["H"], case["R"], case["B"]
    if case["op"] == "append":
        L, n = case["L"], case["B"] * case["T"]
        # latent and rotated part in and out, the queries' rotated parts in and out, the
        # angles of each position, row and position of each token and its page
        return {"bytes": n * (2 * 2 * (L + R) + 2 * 2 * H * R + 4 * R + 12),
                "flops": n * (4 * L * case["norm"] + 3 * R * (1 + H))}
    lengths = _lengths(case)
    total = sum(lengths)
    if case["op"] == "attn":
        L, T = case["L"], case["T"]
        return {"bytes": int(total * 2 * (L + R) + B * T * H * (2 * (L + R) + 2 * L + 4)),
                "flops": int(T * H * total * 2 * (2 * L + R))}
    N, V, p = case["N"], case["V"], case["prefix"]
    # every query's products with the keys that it sees: its own and those before it
    seen = sum(n * (n + 1) / 2 + n * p for n in lengths)
    return {"bytes": int(total * H * (2 * (N + R) + 2 * V + 4) + (total + B * p) * 2 * (H * (N + V) + R)),
            "flops": int(H * seen * 2 * (N + R + V))}


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


def _exact_rows(scores, values, seen):
    """Softmax-weighted sums of one row's values; query i sees the first seen[i] keys."""
    scores = torch.where(torch.arange(scores.shape[-1], device="cuda") < seen[..., None], scores, -math.inf)
    lse = torch.logsumexp(scores, -1)
    w = torch.where(lse[..., None] > -math.inf, torch.exp(scores - lse[..., None]), 0.0)
    return torch.nan_to_num(w) @ values, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        L, P = case["L"], case["page"]
        cache, q_out = s["cache"].double(), s["q_out"].double()
        c = s["latent"].double()
        if s["norm_w"] is not None:
            c = c / (c.pow(2).sum(-1, keepdim=True) / L + EPS).sqrt() * s["norm_w"].double()
        turn = s["cos_sin"].index_select(0, s["positions"])
        flat = s["table"].long().gather(1, (s["positions"].long() // P).reshape(case["B"], -1)).reshape(-1) * P \
            + s["positions"].long() % P
        cache.view(-1, L + case["R"])[flat] = torch.cat([c, _exact_rotation(s["rot"], turn, case["pairs"])], 1)
        q_out[..., L:] = _exact_rotation(s["q_rot"], turn[:, None].expand(-1, case["H"], -1), case["pairs"])
        return {"cache": cache, "q": q_out}
    outs, sums = [], []
    if case["op"] == "attn":
        L, T, H = case["L"], case["T"], case["H"]
        for b in range(case["B"]):
            n = int(s["kv_len"][b])
            keys = s["cache"][s["table"][b].long()].flatten(0, 1)[:n].double()
            seen = n - torch.arange(T - 1, -1, -1, device="cuda").repeat_interleave(H)
            o, lse = _exact_rows(s["q"][b].flatten(0, 1).double() @ keys.T * s["scale"], keys[:, :L], seen)
            outs.append(o.view(T, H, L))
            sums.append(lse.view(T, H))
        return {"out": torch.stack(outs), "lse": torch.stack(sums)}
    N = case["N"]
    for b in range(case["B"]):
        q = s["q"][s["cu_q"][b]:s["cu_q"][b + 1]]
        kv = s["kv"][s["cu_k"][b]:s["cu_k"][b + 1]]
        rot = s["rot"][s["cu_k"][b]:s["cu_k"][b + 1]].double()
        seen = torch.arange(q.shape[0], device="cuda") + (kv.shape[0] - q.shape[0] + 1)
        heads = []
        for h in range(case["H"]):
            key = torch.cat([kv[:, h, :N].double(), rot], 1)
            heads.append(_exact_rows(q[:, h].double() @ key.T * s["scale"], kv[:, h, N:].double(), seen))
        outs.append(torch.stack([o for o, _ in heads], 1))
        sums.append(torch.stack([l for _, l in heads], 1))
    return {"out": torch.cat(outs), "lse": torch.cat(sums)}
