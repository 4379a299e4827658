"""examples/latent_draft.py runs the three latent operators with the draft head's other calls.
Its draft steps (absorbed form, one token at a time over the paged cache) give what one pass
over prompt and drafts together gives in the expanded form, and in the absorbed form with
several tokens a row; lengths and counts fit together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("latent_draft", os.path.join(ROOT, "examples", "latent_draft.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("rows,drafts,hidden,heads,longest", [(1, 2, 256, 4, 5), (5, 4, 512, 16, 150)])
def test_the_forms_agree_along_a_draft(example, rows, drafts, hidden, heads, longest):
    r = example.run(rows, drafts, hidden, heads, vocab=4096, longest=longest, seed=rows)
    lens, steps = r["lens"], drafts - 1
    assert torch.equal(r["kv_len"], lens.int() + steps)
    # prompt and drafted positions as one text, in the expanded form
    new = [torch.cat([r["x0"][int(r["cu"][b]):int(r["cu"][b + 1])], torch.stack([x[b] for x in r["inputs"]])])
           for b in range(rows)]
    n = [len(x) for x in new]
    cu = torch.tensor([0] + n, device="cuda").cumsum(0).int()
    row = torch.arange(rows, device="cuda").repeat_interleave(torch.tensor(n, device="cuda")).int()
    pos = torch.cat([torch.arange(k, device="cuda") for k in n]).int()
    block = r["block"]
    whole = block.prompt(torch.cat(new), row, pos, cu)
    last = whole[(cu[1:] - 1).long()].float()
    # both round latents, heads' keys and values, weights and outputs to bf16 on the way: some
    # 2^-8 of values of size one each
    assert (last - r["last_hidden"].float()).abs().max() < 8 * 2.0 ** -8
    # the drafted positions again, all of a row's in one call
    x = torch.stack(r["inputs"], 1).reshape(rows * steps, hidden)
    at = (lens[:, None] + torch.arange(steps, device="cuda")).reshape(-1).int()
    rows_of = torch.arange(rows, device="cuda").repeat_interleave(steps).int()
    again = block.step(x, rows_of, at, r["kv_len"], T=steps).view(rows, steps, hidden)
    assert (again[:, -1].float() - r["last_hidden"].float()).abs().max() < 8 * 2.0 ** -8


def test_lengths_after_the_verification(example):
    r = example.run(6, 3, 256, 4, vocab=4096, longest=40, seed=3)
    prefix = r["agree"].int().cumprod(1).sum(1)
    assert torch.equal(r["accepted"], prefix.int())
    assert torch.equal(r["main_len"], r["lens"].int() + 1 + prefix.int())
    assert torch.equal(r["draft_len"], torch.minimum(r["kv_len"], r["main_len"]))
