"""Attention with grouped heads over a paged cache in 64 bits, with the bounds of
latent_reference (weights rounded to the inputs' type, fp32 sums), for any set of visible keys."""
import torch

from latent_reference import E32, half_step


def attend(q, keys, values, seen, scale, dtype):
    """Rows q[m, D] over keys[n, D] and values[n, D], row i seeing the keys where seen[m, n]:
    (out, lse, bound on out, bound on lse), float64.  The bounds are latent_reference's."""
    q, keys, values = q.double(), keys.double(), values.double()
    n, D = keys.shape
    if n == 0:
        z = q.new_zeros(len(q), D)
        inf = q.new_full((len(q),), -torch.inf)
        return z, inf, z, torch.zeros_like(inf)
    s = (q @ keys.T * scale).masked_fill(~seen, -torch.inf)
    size = (q.abs() @ keys.abs().T * scale).masked_fill(~seen, 0.0)
    e_s = E32 * D * size.amax(1)
    lse = torch.logsumexp(s, 1)
    p = torch.where(seen, torch.exp(s - torch.where(lse > -torch.inf, lse, 0.0)[:, None]), 0.0)
    out, A = p @ values, p @ values.abs()
    u = half_step(dtype)
    wobble = (n + 16) * E32
    tol = u * out.abs() + (u + 2 * e_s[:, None] + wobble) * 1.01 * A
    lse_tol = e_s + wobble + E32 * torch.where(lse > -torch.inf, lse.abs(), 0.0)
    return out, lse, tol, lse_tol


def visible(n_queries, length, window, sinks, device):
    """seen[i, j] for a row's last n_queries positions over its first `length`."""
    pos = torch.arange(length - n_queries, length, device=device)[:, None]
    j = torch.arange(length, device=device)
    seen = j <= pos
    if window:
        seen = seen & ((j > pos - window) | (j < sinks))
    return seen


class Batch:
    """Rows (new tokens, length) over a cache whose unwritten slots hold NaN and whose table has
    nonsense where no page is needed.  layout: "slots" [pages, P, Hkv, D], "heads" [pages, Hkv, P, D]
    or "both" (keys and values of a page side by side)."""

    def __init__(self, rows, Hq, Hkv, D, P, dtype, seed=0, layout="slots", std=1.0, spare=2, pad=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def rnd(*shape):
            return (torch.randn(*shape, generator=g, device=device) * std).to(dtype)
        self.rows, self.Hq, self.Hkv, self.D, self.P, self.dtype = rows, Hq, Hkv, D, P, dtype
        B = len(rows)
        need = [-(-n // P) for _, n in rows]
        pages = sum(need) + spare
        wide = max(need + [1]) + 1
        order = torch.randperm(pages, generator=g, device=device).int()
        self.table = torch.full((B, wide), -12345, dtype=torch.int32, device=device)
        nan = float("nan")
        if layout == "slots":
            k, v = (torch.full((pages, P, Hkv, D), nan, dtype=dtype, device=device) for _ in range(2))
        elif layout == "heads":
            k, v = (torch.full((pages, Hkv, P, D), nan, dtype=dtype, device=device).transpose(1, 2)
                    for _ in range(2))
        else:
            kv = torch.full((pages, 2, P, Hkv, D + 8), nan, dtype=dtype, device=device)
            k, v = kv[:, 0, ..., :D], kv[:, 1, ..., :D]
        self.k, self.v, self.keys, self.values = k, v, [], []
        at = 0
        for b, (_, n) in enumerate(rows):
            mine = order[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = mine
            keys, values = rnd(n, Hkv, D), rnd(n, Hkv, D)
            if n:
                i = torch.arange(n, device=device)
                k[mine.long()[i // P], i % P] = keys
                v[mine.long()[i // P], i % P] = values
            self.keys.append(keys)
            self.values.append(values)
        new = torch.tensor([r[0] for r in rows], device=device)
        self.cu = torch.zeros(B + 1, dtype=torch.int32, device=device)
        self.cu[1:] = new.cumsum(0)
        self.kv_len = torch.tensor([r[1] for r in rows], dtype=torch.int32, device=device)
        self.Tq = int(self.cu[-1])
        self.pad = pad
        wide_q = rnd(self.Tq + pad, Hq, D + 16)
        self.q = wide_q[..., 8:8 + D] if layout == "both" else wide_q[..., :D].contiguous()
        self.scale = D ** -0.5

    def run(self, lib, window=0, sinks=0, stream=None, **changes):
        dev = self.q.device
        self.out = torch.full((self.Tq + self.pad, self.Hq, self.D), 7.0, dtype=self.dtype, device=dev)
        self.lse = torch.full((self.Tq + self.pad, self.Hq), 7.0, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        n = lib.mtp_heads_attn_workspace_bytes(len(self.rows), self.Tq + self.pad, self.Hq, self.Hkv, self.D)
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device=dev)  # NaN, whatever it is read as
        a = dict(q=self.q, k_cache=self.k, v_cache=self.v, block_table=self.table, cu_q=self.cu,
                 kv_len=self.kv_len, out=self.out, scale=self.scale, window=window, sinks=sinks,
                 lse=self.lse, workspace=self.ws, status=self.status, stream=stream) | changes
        lib.mtp_heads_attn(**a)
        return self.out, self.lse

    def want(self, b, h, window=0, sinks=0):
        """(out, lse, bounds) of row b's queries of head h."""
        n, length = self.rows[b]
        g = h // (self.Hq // self.Hkv)
        q = self.q[self.cu[b]:self.cu[b + 1], h]
        return attend(q, self.keys[b][:, g], self.values[b][:, g],
                      visible(n, length, window, sinks, q.device), self.scale, self.dtype)

    def check(self, window=0, sinks=0, heads=None, status=0):
        from latent_reference import check, check_lse
        assert int(self.status) == status
        for b, (n, length) in enumerate(self.rows):
            lo, hi = int(self.cu[b]), int(self.cu[b + 1])
            for h in heads if heads is not None else range(self.Hq):
                out, lse, tol, lse_tol = self.want(b, h, window, sinks)
                check(self.out[lo:hi, h], out, tol, f"out of row {b} {self.rows[b]}, head {h}")
                check_lse(self.lse[lo:hi, h], lse, lse_tol, f"lse of row {b} {self.rows[b]}, head {h}")
        if self.pad:
            assert (self.out[self.Tq:] == 7).all() and (self.lse[self.Tq:] == 7).all()
