"""mtp_heads_attn_workspace_bytes: a workspace made for a batch serves every smaller one (no GPU)."""
import ctypes as C

import pytest

import verify_spec_greedy_gb300 as pkg
from test_heads_abi import ATTN, OK, WORKSPACE, so  # noqa: F401


@pytest.mark.parametrize("D", [16, 48, 64, 80, 128, 144, 256])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (32, 8), (1, 1), (128, 1)])
def test_a_batchs_workspace_serves_smaller_ones(so, Hq, Hkv, D):  # noqa: F811
    ws = pkg.mtp_heads_attn_workspace_bytes
    sizes = [(B, T) for B in (1, 2, 9, 256, 1024, 65536) for T in (1, 4, 31, 256, 5000, 65536)]
    for B, T in sizes:
        n = ws(B, T, Hq, Hkv, D)
        assert n > 0 and all(ws(b, t, Hq, Hkv, D) <= n for b, t in sizes if b <= B and t <= T)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T", [(1, 256), (256, 256), (256, 1)])
def test_less_is_refused_at_every_size(so, D, B, T):  # noqa: F811
    n = pkg.mtp_heads_attn_workspace_bytes(B, T, 16, 4, D)
    a = ATTN | dict(B=B, Tq=T, D=D, page_stride=64 * 4 * D, slot_stride=4 * D, head_stride=D, q_tok=16 * D, q_head=D,
                    out_tok=16 * D, out_head=D)
    assert so.mtp_heads_attn(*(a | dict(Tq=0)).values()) == OK
    assert so.mtp_heads_attn(*(a | dict(workspace=C.c_void_p(4096), workspace_bytes=n - 1)).values()) == WORKSPACE
