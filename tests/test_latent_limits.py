"""The latent attention's limits, on the host: what include/libmtpspec/latent.h states is what the
entry points check.  A call at a limit goes through to the next check (the first pointer, which is
missing); one step beyond it is refused."""
import os
import re

import pytest

import verify_spec_greedy_gb300 as pkg
from test_latent_abi import APPEND, ATTN, PREFILL, ROOT, so  # noqa: F401

ARG, SHAPE = -1, -3
IDS = (1 << 31) - 1
WIDE = dict(L=64, q_row=1 << 38, q_tok=1 << 20, q_head=128, page_stride=64 * 128, out_row=1 << 38,
            out_tok=1 << 20, out_head=64, q=None)


@pytest.mark.parametrize("good,bad", [
    # 65536 query rows a sequence: the rows of all sequences are the limit
    (dict(B=32767, T=64, Hq=1024), dict(B=32768, T=64, Hq=1024)),
    (dict(B=1 << 20, T=2, Hq=1023), dict(B=1 << 20, T=2, Hq=1024)),
    (dict(B=1 << 20, T=1, Hq=16), dict(B=(1 << 20) + 1, T=1, Hq=16)),
    (dict(B=1, T=256, Hq=256), dict(B=1, T=256, Hq=257)),
    (dict(B=1, num_pages=IDS), dict(B=1, num_pages=IDS + 1)),
    (dict(B=1, max_pages=IDS), dict(B=1, max_pages=IDS + 1)),
    (dict(B=2, q_row=(1 << 39) - 8), dict(B=2, q_row=1 << 39)),
])
def test_attn(so, good, bad):  # noqa: F811
    good, bad = {**ATTN, **WIDE, **good}, {**ATTN, **WIDE, **bad}
    assert so.mtp_latent_attn(*good.values()) == ARG
    assert so.mtp_latent_attn(*bad.values()) == SHAPE
    rows = [(a["B"], a["T"], a["Hq"], a["L"], a["R"]) for a in (good, bad)]
    assert pkg.mtp_latent_attn_workspace_bytes(*rows[0]) > 0
    if rows[0] != rows[1]:
        assert pkg.mtp_latent_attn_workspace_bytes(*rows[1]) == 0


@pytest.mark.parametrize("good,bad", [
    (dict(T=1 << 20), dict(T=(1 << 20) + 1)), (dict(B=1 << 20), dict(B=(1 << 20) + 1)),
    (dict(Hq=1024), dict(Hq=1025)), (dict(max_pos=IDS), dict(max_pos=IDS + 1)),
    (dict(page_size=1 << 24, page_stride=576 << 24), dict(page_size=(1 << 24) + 8, page_stride=577 << 24)),
])
def test_append(so, good, bad):  # noqa: F811
    base = {**APPEND, "T": 1, "q_rot_tok": 1 << 20, "q_out_tok": 1 << 20, "latent": None}
    assert so.mtp_latent_append(*{**base, **good}.values()) == ARG
    assert so.mtp_latent_append(*{**base, **bad}.values()) == SHAPE


@pytest.mark.parametrize("good,bad", [
    (dict(Tq=1 << 24), dict(Tq=(1 << 24) + 1)), (dict(Tk=1 << 24), dict(Tk=(1 << 24) + 1)),
    (dict(B=65536), dict(B=65537)), (dict(Hq=1024), dict(Hq=1025)), (dict(Tk=1), dict(Tk=0)),
])
def test_prefill(so, good, bad):  # noqa: F811
    base = {**PREFILL, "Tq": 1, "Tk": 1, "q_tok": 1 << 20, "kv_tok": 1 << 20, "out_tok": 1 << 20, "q": None}
    assert so.mtp_latent_prefill(*{**base, **good}.values()) == ARG
    assert so.mtp_latent_prefill(*{**base, **bad}.values()) == SHAPE


def test_the_header_states_them():
    text = re.sub(r"\n \* *", " ", open(os.path.join(ROOT, "include", "libmtpspec", "latent.h")).read())
    for limit in ("B * T * Hq <= 2^31 - 1", "T * Hq <= 65536", "num_pages, max_pages and max_pos from 1 to 2^31 - 1",
                  "below 2^39", "0 <= Tq, Tk <= 2^24", "1 <= B <= 65536", "0 <= T <= 2^20, 1 <= B <= 2^20",
                  "up to 2^24"):
        assert limit in text, limit
