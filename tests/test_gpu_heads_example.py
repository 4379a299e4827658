"""The grouped heads' operators together, as examples/heads_draft.py runs them: every attention of the
run against its formula over what the cache holds, and the pages' counts at the end."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import heads_draft  # noqa: E402
from heads_reference import attend, visible  # noqa: E402
from latent_reference import check  # noqa: E402

pytestmark = pytest.mark.gpu


def against_the_formula(block, q, cu, kv_len, out):
    for b in range(block.table.shape[0]):
        lo, hi, n = int(cu[b]), int(cu[b + 1]), int(kv_len[b])
        if hi == lo:
            continue
        pages = block.table[b, :int(block.held[b])].long()
        keys, values = (c[pages].flatten(0, 1)[:n] for c in (block.k, block.v))
        seen = visible(hi - lo, n, block.window, block.sinks, q.device)
        for h in (0, block.Hq - 1):
            g = h // (block.Hq // block.Hkv)
            want, _, tol, _ = attend(q[lo:hi, h], keys[:, g], values[:, g], seen, block.D ** -0.5, q.dtype)
            check(out[lo:hi, h], want, tol, f"row {b}, head {h}")


@pytest.mark.parametrize("kw", [dict(), dict(rows=3, branches=4, drafts=6, window=40, sinks=4, page=8),
                                dict(rows=2, branches=2, drafts=20, Hq=8, Hkv=8, D=64, R=32, page=32),
                                dict(rows=4, branches=1, drafts=2, Hq=8, Hkv=1, D=256, R=64)])
def test_a_round_of_branched_drafts(kw):
    r = heads_draft.run(hidden=256, vocab=4096, seed=len(kw), hook=against_the_formula, **kw)
    b, rows = r["block"], r["rows"]
    assert int(b.status) == 0
    # the accepted drafts are the agreed ones, and every row goes on from its longest branch
    want = r["agree"].int().cumprod(1).sum(1)
    assert torch.equal(r["accepted"].long(), want.long())
    longest = want.view(rows, -1).amax(1).clamp(max=r["ids"].shape[1] - 1)
    assert torch.equal(r["kept"], r["lens"] + longest)
    # the rows hold what they kept, the branches nothing, and the counts are the table's
    assert torch.equal(b.held[:rows].long(), -(-r["kept"] // b.page)) and (b.held[rows:] == 0).all()
    held = b.table[b.table >= 0].long()
    assert torch.equal(torch.bincount(held, minlength=len(b.refs)).int(), b.refs)
    assert held.numel() == int(b.held.sum()) and int(b.refs.max()) == 1


def test_the_command_runs(capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["heads_draft.py", "--rows", "2", "--hidden", "128"])
    heads_draft.main()
    assert "pages held" in capsys.readouterr().out
