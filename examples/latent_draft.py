"""A draft head whose block is latent attention, from its first pass over the prompts to the
verification of its drafts, with random weights:

    python examples/latent_draft.py [--rows 8] [--drafts 3] [--hidden 1024] [--heads 16]

1. The first pass pairs every prompt position with its next token: mtp_draft_input, then
   mtp_latent_append writes the latents into the paged cache and rotates keys and queries, and
   mtp_latent_prefill attends in the expanded form.
2. Each draft step runs one token a row: mtp_draft_input, mtp_latent_append, mtp_latent_attn in
   the absorbed form over the cache, mtp_lm_head_greedy.
3. A stand-in for the main model gives target logits, spec_verify_greedy accepts a prefix of
   the drafts, and mtp_state_fixup cuts the draft head's cache back to it (its pages stay).

The projections between the library's calls are plain matrix products.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import verify_spec_greedy_gb300 as lib  # noqa: E402

BF = torch.bfloat16
EPS = 1e-6


class LatentBlock:
    """The weights of one block: N key and V value columns a head, R rotated ones, a latent of
    L values; and the paged cache of `rows` rows up to `length` positions."""

    def __init__(self, hidden, heads, rows, length, L=512, R=64, N=128, V=128, page=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape, fan):
            return (torch.randn(*shape, generator=g, device="cuda") * fan ** -0.5).to(BF)
        self.H, self.L, self.R, self.N, self.V, self.page = heads, L, R, N, V, page
        self.w_q, self.w_down = w(heads * (N + R), hidden, fan=hidden), w(L + R, hidden, fan=hidden)
        self.w_k, self.w_v = w(heads, N, L, fan=L), w(heads, V, L, fan=L)
        self.w_out = w(hidden, heads * V, fan=heads * V)
        self.norm_w = torch.ones(L, dtype=BF, device="cuda")
        self.scale = (N + R) ** -0.5
        a = torch.arange(length, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float()
        per_row = -(-length // page)
        order = torch.randperm(rows * per_row, generator=g, device="cuda")
        self.table = order.reshape(rows, per_row).int()
        self.cache = torch.zeros(rows * per_row, page, L + R, dtype=BF, device="cuda")
        self.workspace = torch.empty(lib.mtp_latent_attn_workspace_bytes(rows, 8, heads, L, R),
                                     dtype=torch.uint8, device="cuda")

    def project(self, x, row, pos):
        """The tokens' latents into the cache; their queries [T, H, N + R], rotated."""
        q = (x @ self.w_q.T).view(len(x), self.H, self.N + self.R)
        down = x @ self.w_down.T
        lib.mtp_latent_append(down[:, :self.L], down[:, self.L:], self.cos_sin, row, pos, self.table,
                              self.cache, norm_w=self.norm_w, eps=EPS, q_rot=q[..., self.N:],
                              q_out=q[..., self.N:])
        return q

    def prompt(self, x, row, pos, cu):
        """Whole prompts, one after another, in the expanded form."""
        q = self.project(x, row, pos)
        at = pos.long()
        kept = self.cache[self.table[row.long(), at // self.page].long(), at % self.page]
        up = torch.cat([self.w_k, self.w_v], 1).view(-1, self.L)        # a head's keys, its values
        kv = (kept[:, :self.L] @ up.T).view(len(x), self.H, self.N + self.V)
        out = torch.empty(len(x), self.H, self.V, dtype=BF, device="cuda")
        lib.mtp_latent_prefill(q, kv, kept[:, self.L:], cu, cu, out, self.scale)
        return x + out.view(len(x), -1) @ self.w_out.T

    def step(self, x, row, pos, kv_len, T=1):
        """T tokens of every row, in the absorbed form over the cache."""
        B = kv_len.numel()
        q = self.project(x, row, pos)
        latent = torch.einsum("thn,hnl->thl", q[..., :self.N], self.w_k)
        qa = torch.cat([latent, q[..., self.N:]], -1).view(B, T, self.H, self.L + self.R)
        out = torch.empty(B, T, self.H, self.L, dtype=BF, device="cuda")
        lib.mtp_latent_attn(qa, self.cache, self.table, kv_len, out, self.scale,
                            workspace=self.workspace)
        heads = torch.einsum("thl,hvl->thv", out.view(B * T, self.H, self.L), self.w_v)
        return x + heads.reshape(B * T, -1) @ self.w_out.T


def run(rows=8, drafts=3, hidden=1024, heads=16, vocab=32768, longest=300, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)

    def w(*shape, std):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF)
    embed, head_w = w(vocab, hidden, std=1.0), w(vocab, hidden, std=hidden ** -0.5)
    enorm, hnorm = torch.ones(hidden, dtype=BF, device="cuda"), torch.ones(hidden, dtype=BF, device="cuda")
    eh_proj = w(hidden, 2 * hidden, std=(2 * hidden) ** -0.5)
    block = LatentBlock(hidden, heads, rows, longest + drafts + 1, seed=seed)

    def draft_input(tokens, h):
        M = len(tokens)
        out = torch.empty(M, hidden, dtype=BF, device="cuda")
        n = lib.mtp_draft_input_workspace_bytes(M, hidden)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        return lib.mtp_draft_input(embed[tokens.long()], h, enorm, hnorm, eh_proj, out, EPS, workspace=ws)

    def pick(h, ids):
        n = lib.mtp_lm_head_greedy_workspace_bytes(len(h), hidden, vocab)
        return lib.mtp_lm_head_greedy(h, head_w, ids, norm_w=hnorm, eps=EPS,
                                      workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))

    # 1. the first pass over ragged prompts
    lens = torch.randint(1, longest + 1, (rows,), generator=g, device="cuda")
    lens[0] = longest
    cu = torch.zeros(rows + 1, dtype=torch.int32, device="cuda")
    cu[1:] = lens.cumsum(0)
    total = int(cu[-1])
    row = torch.arange(rows, device="cuda").repeat_interleave(lens).int()
    pos = (torch.arange(total, device="cuda") - cu[:-1].long().repeat_interleave(lens)).int()
    next_tokens = torch.randint(0, vocab, (total,), generator=g, device="cuda")
    main_hidden = w(total, hidden, std=1.0)
    x0 = draft_input(next_tokens, main_hidden)
    h = block.prompt(x0, row, pos, cu)
    last = (cu[1:] - 1).long()
    h = h[last].contiguous()
    kv_len = lens.int()
    ids = torch.empty(rows, dtype=torch.int32, device="cuda")
    pick(h, ids)

    # 2. the drafts: D tokens, the first from the prompt's last position
    draft_ids = torch.empty(rows, drafts, dtype=torch.int32, device="cuda")
    draft_ids[:, 0] = ids
    all_rows = torch.arange(rows, dtype=torch.int32, device="cuda")
    inputs = []
    for d in range(1, drafts):
        x = draft_input(ids, h)
        inputs.append(x)
        at = kv_len.clone()
        kv_len = kv_len + 1
        h = block.step(x, all_rows, at, kv_len)
        pick(h, ids)
        draft_ids[:, d] = ids

    # 3. verification: the stand-in agrees with each draft three times in four
    target = torch.randn(rows, drafts + 1, vocab, generator=g, device="cuda")
    agree = torch.rand(rows, drafts, generator=g, device="cuda") < 0.75
    top = target[:, :drafts].amax(-1, keepdim=True) + 1
    target[:, :drafts].scatter_(2, draft_ids.long()[..., None],
                                torch.where(agree[..., None], top, top - 20))
    tokens = torch.empty(rows, drafts + 1, dtype=torch.int32, device="cuda")
    accepted = torch.empty(rows, dtype=torch.int32, device="cuda")
    lib.spec_verify_greedy(target, draft_ids, tokens, accepted)
    main_len = torch.empty(rows, dtype=torch.int32, device="cuda")
    draft_len = kv_len.clone()
    lib.mtp_state_fixup(accepted, drafts, lens.int(), main_len, draft_kv_len=draft_len)
    return dict(block=block, x0=x0, inputs=inputs, last_hidden=h, lens=lens, kv_len=kv_len, cu=cu, row=row,
                pos=pos, draft_ids=draft_ids, tokens=tokens, accepted=accepted, main_len=main_len,
                draft_len=draft_len, agree=agree)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("rows", 8), ("drafts", 3), ("hidden", 1024), ("heads", 16)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    r = run(a.rows, a.drafts, a.hidden, a.heads)
    torch.cuda.synchronize()
    print("prompt lengths", r["lens"].tolist())
    print("drafts        ", r["draft_ids"].tolist())
    print("accepted      ", r["accepted"].tolist())
    print("draft cache   ", r["kv_len"].tolist(), "cut to", r["draft_len"].tolist())


if __name__ == "__main__":
    main()
