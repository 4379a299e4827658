"""A draft head whose block is attention with grouped heads over a paged cache, with several drafts a
row, random weights:

    python examples/heads_draft.py [--rows 6] [--branches 3] [--drafts 4] [--hidden 1024]

1. The first pass over the prompts: mtp_pages_resize gives every row its pages, mtp_heads_append norms
   and turns queries and keys and writes the cache, mtp_heads_attn attends.
2. Each row branches: mtp_lm_head_topk proposes a first token a branch, mtp_pages_fork shares the
   prompt's pages, mtp_pages_resize gives each branch a last page of its own and room for its drafts,
   and mtp_pages_copy fills that page.
3. Each draft step runs one token a branch.
4. A stand-in for the main model gives target logits, spec_verify_greedy accepts a prefix of every
   branch, and the row goes on from the longest: its pages become the row's, cut to what was
   accepted, and all others are free again.

Nothing is read back in between; the projections are plain matrix products.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import verify_spec_greedy_gb300 as lib  # noqa: E402

BF, I32 = torch.bfloat16, torch.int32
EPS = 1e-6


def ints(x):
    return x.to(I32).contiguous()


class HeadsBlock:
    """The weights of one block with Hq query heads and Hkv key heads of D elements, of which R are
    turned; and the paged cache of `rows` rows up to `length` positions."""

    def __init__(self, hidden, rows, length, pages, Hq=16, Hkv=4, D=128, R=64, page=16, window=0, sinks=0,
                 seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape, fan):
            return (torch.randn(*shape, generator=g, device="cuda") * fan ** -0.5).to(BF)
        self.Hq, self.Hkv, self.D, self.page, self.window, self.sinks = Hq, Hkv, D, page, window, sinks
        self.w_qkv = w((Hq + 2 * Hkv) * D, hidden, fan=hidden)
        self.w_out = w(hidden, Hq * D, fan=Hq * D)
        self.q_norm = self.k_norm = torch.ones(D, dtype=BF, device="cuda")
        a = torch.arange(length, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float()
        self.k, self.v = (torch.zeros(pages, page, Hkv, D, dtype=BF, device="cuda") for _ in range(2))
        self.table = torch.full((rows, -(-length // page)), -1, dtype=I32, device="cuda")
        self.held, self.refs = torch.zeros(rows, dtype=I32, device="cuda"), torch.zeros(pages, dtype=I32, device="cuda")
        self.copies = torch.empty(rows, 2, dtype=I32, device="cuda")
        self.status = torch.zeros(1, dtype=I32, device="cuda")

    def room(self, keep, lens):
        """Every row keeps its first positions and gets pages for `lens`; pages that a branch must not
        share any more are copied."""
        lib.mtp_pages_resize(ints(keep), ints(lens), self.table, self.held, self.refs, self.page, self.copies,
                             status=self.status)
        lib.mtp_pages_copy([self.k, self.v], self.copies, status=self.status)

    def __call__(self, x, row, pos, cu, kv_len, hook=None):
        """x [T, hidden]: the last tokens of the rows of the table, bounded by cu."""
        T, B = len(x), self.table.shape[0]
        qkv = (x @ self.w_qkv.T).view(T, self.Hq + 2 * self.Hkv, self.D)
        q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], 1)
        lib.mtp_heads_append(k, v, self.cos_sin, row, pos, self.table, self.k, self.v, k_norm_w=self.k_norm, q=q,
                             q_out=q, q_norm_w=self.q_norm, eps=EPS, status=self.status)
        out = torch.empty(T, self.Hq, self.D, dtype=BF, device="cuda")
        n = lib.mtp_heads_attn_workspace_bytes(B, T, self.Hq, self.Hkv, self.D)
        lib.mtp_heads_attn(q, self.k, self.v, self.table, cu, kv_len, out, self.D ** -0.5, window=self.window,
                           sinks=self.sinks, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"),
                           status=self.status)
        if hook:
            hook(self, q, cu, kv_len, out)
        return x + out.view(T, -1) @ self.w_out.T


def run(rows=6, branches=3, drafts=4, hidden=1024, vocab=32768, longest=200, seed=0, hook=None, **block):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)

    def w(*shape, std):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF)
    embed, head_w = w(vocab, hidden, std=1.0), w(vocab, hidden, std=hidden ** -0.5)
    norm = torch.ones(hidden, dtype=BF, device="cuda")
    eh_proj = w(hidden, 2 * hidden, std=(2 * hidden) ** -0.5)
    # rows 0 .. rows - 1 hold the prompts, the others the branches
    total_rows = rows * (1 + branches)
    page = block.setdefault("page", 16)
    pages = rows * -(-longest // page) + total_rows * (drafts // page + 2)
    b = HeadsBlock(hidden, total_rows, longest + drafts + 1, pages, seed=seed, **block)

    def draft_input(tokens, h):
        M = len(tokens)
        n = lib.mtp_draft_input_workspace_bytes(M, hidden)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        out = torch.empty(M, hidden, dtype=BF, device="cuda")
        return lib.mtp_draft_input(embed[tokens.long()], h, norm, norm, eh_proj, out, EPS, workspace=ws)

    # 1. the first pass over ragged prompts
    lens = torch.randint(1, longest + 1, (rows,), generator=g, device="cuda")
    lens[0] = longest
    none = torch.zeros(total_rows - rows, dtype=torch.long, device="cuda")
    b.room(torch.zeros(total_rows, device="cuda"), torch.cat([lens, none]))
    cu = torch.zeros(total_rows + 1, dtype=I32, device="cuda")
    cu[1:] = torch.cat([lens, none]).cumsum(0)
    T = int(lens.sum())
    row = ints(torch.arange(rows, device="cuda").repeat_interleave(lens))
    pos = ints(torch.arange(T, device="cuda") - cu[:rows].long().repeat_interleave(lens))
    x = draft_input(torch.randint(0, vocab, (T,), generator=g, device="cuda"), w(T, hidden, std=1.0))
    h = b(x, row, pos, cu, ints(torch.cat([lens, none])), hook)[(cu[1:rows + 1] - 1).long()].contiguous()

    # 2. the branches: the best first tokens, a row of pages each
    n = lib.mtp_lm_head_topk_workspace_bytes(rows, hidden, vocab)
    first = torch.empty(rows, branches, dtype=I32, device="cuda")
    lib.mtp_lm_head_topk(h, head_w, first, norm_w=norm, eps=EPS,
                         workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    src = torch.arange(rows, device="cuda").repeat_interleave(branches)
    dst = torch.arange(rows, total_rows, device="cuda")
    lib.mtp_pages_fork(ints(src), ints(dst), b.table, b.held, b.refs, status=b.status)
    at = lens[src]
    b.room(torch.cat([lens, at]), torch.cat([lens, at + drafts]))

    # 3. the drafts, one token a branch and step
    M = len(dst)
    ids = torch.empty(M, drafts, dtype=I32, device="cuda")
    ids[:, 0] = first.flatten()
    h = h[src].contiguous()
    nws = torch.empty(lib.mtp_lm_head_greedy_workspace_bytes(M, hidden, vocab), dtype=torch.uint8, device="cuda")
    one = torch.zeros(total_rows + 1, dtype=I32, device="cuda")
    one[rows + 1:] = torch.arange(1, M + 1, device="cuda")
    for d in range(1, drafts):
        x = draft_input(ids[:, d - 1].contiguous(), h)
        h = b(x, ints(dst), ints(at + d - 1), one, ints(torch.cat([lens, at + d])), hook)
        pick = torch.empty(M, dtype=I32, device="cuda")
        lib.mtp_lm_head_greedy(h, head_w, pick, norm_w=norm, eps=EPS, workspace=nws)
        ids[:, d] = pick

    # 4. verification of every branch: the stand-in agrees with each draft three times in four
    target = torch.randn(M, drafts + 1, vocab, generator=g, device="cuda")
    agree = torch.rand(M, drafts, generator=g, device="cuda") < 0.75
    top = target[:, :drafts].amax(-1, keepdim=True) + 1
    target[:, :drafts].scatter_(2, ids.long()[..., None], torch.where(agree[..., None], top, top - 20))
    tokens = torch.empty(M, drafts + 1, dtype=I32, device="cuda")
    accepted = torch.empty(M, dtype=I32, device="cuda")
    lib.spec_verify_greedy(target, ids, tokens, accepted)
    best = accepted.view(rows, branches).argmax(1)
    # the cache holds the drafts but the last: what of them was accepted stays
    kept = lens + accepted.view(rows, branches).gather(1, best[:, None])[:, 0].clamp(max=drafts - 1)
    lib.mtp_pages_fork(ints(rows + torch.arange(rows, device="cuda") * branches + best),
                       ints(torch.arange(rows, device="cuda")), b.table, b.held, b.refs, status=b.status)
    b.room(torch.cat([kept, none]), torch.cat([kept, none]))
    return dict(block=b, lens=lens, kept=kept, ids=ids, tokens=tokens, accepted=accepted, best=best, agree=agree,
                rows=rows)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("rows", 6), ("branches", 3), ("drafts", 4), ("hidden", 1024)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    r = run(a.rows, a.branches, a.drafts, a.hidden)
    torch.cuda.synchronize()
    print("prompt lengths   ", r["lens"].tolist())
    print("accepted, by row ", r["accepted"].view(a.rows, -1).tolist())
    print("cut to           ", r["kept"].tolist())
    print("pages held       ", r["block"].held[:a.rows].tolist(), "in use", int((r["block"].refs > 0).sum()))


if __name__ == "__main__":
    main()
