"""The latent attention's C entry points on the host: exported as declared, sizes, types,
strides, alignment and workspaces refused before any CUDA call; and the binding's checks."""
import ctypes as C
import os
import re

import pytest
import torch

import verify_spec_greedy_gb300 as pkg
from verify_spec_greedy_gb300 import _binding as b
from verify_spec_greedy_gb300 import build as cuda_build
from test_binding_checks import dev, lib  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ARG, DTYPE, SHAPE, WORKSPACE = 0, -1, -2, -3, -4
BF, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
P = C.c_void_p(4096)


@pytest.fixture(scope="module")
def so():
    cuda_build.build()
    return pkg.load()


def test_every_declared_symbol_is_exported(so):
    src = open(os.path.join(ROOT, "include", "libmtpspec", "latent.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"^(?:int|size_t)\s+(\w+)\s*\(", src, flags=re.M))
    assert names == {"mtp_latent_append", "mtp_latent_attn", "mtp_latent_attn_workspace_bytes",
                     "mtp_latent_prefill"}
    for n in names:
        assert hasattr(so, n) and hasattr(pkg, n)


def test_the_main_header_brings_the_new_one():
    src = open(os.path.join(ROOT, "include", "libmtpspec.h")).read()
    assert '#include "libmtpspec/latent.h"' in src


APPEND = dict(latent=P, latent_stride=512, rot=P, rot_stride=64, norm_w=None, eps=0.0, cos_sin=P,
              max_pos=100, interleaved=1, tok_row=P, positions=P, T=0, L=512, R=64, block_table=P,
              B=1, max_pages=2, cache=P, num_pages=2, page_size=64, page_stride=64 * 576, q_rot=P,
              q_rot_tok=64 * 4, q_rot_head=64, q_out=P, q_out_tok=64 * 4, q_out_head=64, Hq=4,
              dtype=1, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    ({}, OK), (dict(dtype=0), DTYPE), (dict(dtype=3), DTYPE), (dict(dtype=2), OK),
    (dict(T=-1), SHAPE), (dict(T=(1 << 20) + 1), SHAPE), (dict(L=0), SHAPE), (dict(L=500), SHAPE),
    (dict(L=576), SHAPE), (dict(R=0), SHAPE), (dict(R=24), SHAPE), (dict(R=80), SHAPE),
    (dict(B=0), SHAPE), (dict(max_pages=0), SHAPE), (dict(num_pages=0), SHAPE),
    (dict(page_size=4), SHAPE), (dict(page_size=12), SHAPE), (dict(page_stride=64 * 576 - 8), SHAPE),
    (dict(page_stride=64 * 576 + 4), SHAPE), (dict(max_pos=0), SHAPE),
    (dict(T=2, latent_stride=504), SHAPE), (dict(T=2, latent_stride=516), SHAPE),
    (dict(T=2, rot_stride=-64), SHAPE), (dict(Hq=0), SHAPE), (dict(Hq=1025), SHAPE),
    (dict(q_rot_head=32), SHAPE), (dict(q_out_head=4), SHAPE), (dict(T=2, q_out_tok=63), SHAPE),
    (dict(q_out=None), ARG), (dict(q_rot=None), ARG), (dict(q_rot=None, q_out=None, Hq=0), OK),
    (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(T=1, latent=None), ARG), (dict(T=1, cache=None), ARG), (dict(T=1, cos_sin=None), ARG),
    (dict(T=1, tok_row=None), ARG), (dict(T=1, block_table=None), ARG),
    (dict(T=1, latent=C.c_void_p(4104)), ARG), (dict(T=1, cache=C.c_void_p(4098)), ARG),
    (dict(T=1, norm_w=C.c_void_p(4104)), ARG), (dict(T=1, cos_sin=C.c_void_p(4100)), ARG),
    (dict(T=1, positions=C.c_void_p(4097)), ARG), (dict(T=1, q_out=C.c_void_p(4104)), ARG),
    (dict(T=1, status=C.c_void_p(4098)), ARG),
])
def test_append_refusals(so, change, code):
    assert so.mtp_latent_append(*{**APPEND, **change}.values()) == code


ATTN = dict(q=P, q_row=16 * 576, q_tok=16 * 576, q_head=576, cache=P, num_pages=2, page_size=64,
            page_stride=64 * 576, block_table=P, max_pages=2, kv_len=P, B=0, T=1, Hq=16, L=512, R=64,
            scale=0.1, out=P, out_row=16 * 512, out_tok=16 * 512, out_head=512, lse=None, dtype=1,
            workspace=None, workspace_bytes=0, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    ({}, OK), (dict(dtype=0), DTYPE), (dict(dtype=2), OK), (dict(B=-1), SHAPE),
    (dict(B=(1 << 20) + 1), SHAPE), (dict(T=0), SHAPE), (dict(T=257), SHAPE), (dict(Hq=0), SHAPE),
    (dict(T=256, Hq=1024), SHAPE), (dict(L=520), SHAPE), (dict(R=8), SHAPE),
    (dict(B=1 << 20, T=128, Hq=128), SHAPE), (dict(page_size=63), SHAPE),
    (dict(q_head=568), SHAPE), (dict(q_head=577), SHAPE), (dict(B=2, q_row=0), SHAPE),
    (dict(out_head=504), SHAPE), (dict(T=2, out_tok=8), SHAPE), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (dict(scale=0.0), ARG), (dict(scale=-0.1), ARG),
    (dict(B=1, q=None), ARG), (dict(B=1, out=None), ARG), (dict(B=1, kv_len=None), ARG),
    (dict(B=1, block_table=None), ARG), (dict(B=1, cache=None), ARG),
    (dict(B=1, q=C.c_void_p(4104)), ARG), (dict(B=1, out=C.c_void_p(4104)), ARG),
    (dict(B=1, lse=C.c_void_p(4097)), ARG), (dict(B=1), WORKSPACE),
    (dict(B=1, workspace=P, workspace_bytes=1000), WORKSPACE),
    (dict(B=1, workspace=C.c_void_p(4112), workspace_bytes=1 << 30), ARG),
])
def test_attn_refusals(so, change, code):
    assert so.mtp_latent_attn(*{**ATTN, **change}.values()) == code


def test_attn_workspace(so):
    ws = pkg.mtp_latent_attn_workspace_bytes
    assert ws(1, 1, 16, 512, 64) > 0 and ws(1, 1, 16, 512, 64) % 256 == 0
    assert ws(4, 2, 128, 512, 64) >= ws(4, 1, 16, 512, 64)
    for bad in ((0, 1, 16, 512, 64), (1, 0, 16, 512, 64), (1, 1, 16, 513, 64), (1, 1, 16, 512, 72),
                (-1, 1, 16, 512, 64), (1, 1, 1025, 512, 64)):
        assert ws(*bad) == 0


PREFILL = dict(q=P, q_tok=2 * 192, q_head=192, kv=P, kv_tok=2 * 256, kv_head=256, rot=P, rot_stride=64,
               cu_q=P, cu_k=P, B=1, Tq=0, Tk=0, Hq=2, N=128, R=64, V=128, scale=0.1, out=P,
               out_tok=2 * 128, out_head=128, lse=None, dtype=1, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    ({}, OK), (dict(dtype=0), DTYPE), (dict(dtype=2), OK), (dict(B=0), SHAPE), (dict(Tq=-1), SHAPE),
    (dict(Tq=5), SHAPE), (dict(Tq=1 << 25, Tk=5), SHAPE), (dict(Tk=-1), SHAPE), (dict(Hq=0), SHAPE),
    (dict(N=96), SHAPE), (dict(V=256), SHAPE), (dict(R=12), SHAPE), (dict(R=128), SHAPE),
    (dict(q_head=184), SHAPE), (dict(kv_head=252), SHAPE), (dict(Tq=2, Tk=2, rot_stride=16), SHAPE),
    (dict(out_head=64), SHAPE), (dict(Tq=2, Tk=2, out_tok=4), SHAPE), (dict(scale=0.0), ARG),
    (dict(scale=float("nan")), ARG), (dict(Tq=1, Tk=1, q=None), ARG), (dict(Tq=1, Tk=1, kv=None), ARG),
    (dict(Tq=1, Tk=1, rot=None), ARG), (dict(Tq=1, Tk=1, cu_q=None), ARG),
    (dict(Tq=1, Tk=1, out=C.c_void_p(4100)), ARG), (dict(Tq=1, Tk=1, rot=C.c_void_p(4104)), ARG),
    (dict(Tq=1, Tk=1, cu_k=C.c_void_p(4098)), ARG), (dict(Tq=1, Tk=1, lse=C.c_void_p(4098)), ARG),
])
def test_prefill_refusals(so, change, code):
    assert so.mtp_latent_prefill(*{**PREFILL, **change}.values()) == code


# ---------------------------------------------------------------- the binding

def append_args(T=3, L=64, R=16, dtype=BF):
    down = dev(T, L + R, dtype=dtype)
    return dict(latent=down[:, :L], rot=down[:, L:], cos_sin=dev(9, R), tok_row=dev(T, dtype=I32),
                positions=dev(T, dtype=I32), block_table=dev(2, 4, dtype=I32),
                cache=dev(5, 8, L + R, dtype=dtype), norm_w=dev(L, dtype=dtype), eps=0.5,
                q_rot=dev(T, 2, 40, dtype=dtype)[..., 24:], q_out=dev(T, 2, R, dtype=dtype))


def test_append_passes_strides(lib):  # noqa: F811
    a = append_args()
    b.mtp_latent_append(**a)
    (name, args), = lib.calls
    assert name == "mtp_latent_append"
    assert args[1] == args[3] == 80 and args[2] - args[0] == 128
    assert args[11:14] == (3, 64, 16) and args[15:17] == (2, 4)
    assert args[18:21] == (5, 8, 640) and args[22:24] == (80, 40) and args[25:29] == (32, 16, 2, b.BF16)


def test_append_refuses(lib):  # noqa: F811
    for change, err in ((dict(latent=torch.zeros(3, 64, dtype=BF)), ValueError),
                        (dict(latent=dev(3, 64)), TypeError), (dict(rot=dev(3, 16, dtype=F16)), TypeError),
                        (dict(rot=dev(2, 16, dtype=BF)), ValueError), (dict(cos_sin=dev(9, 8)), ValueError),
                        (dict(cos_sin=dev(9, 16, dtype=BF)), TypeError),
                        (dict(tok_row=dev(2, dtype=I32)), ValueError),
                        (dict(positions=dev(3, dtype=torch.int64)), TypeError),
                        (dict(cache=dev(5, 8, 79, dtype=BF)), ValueError),
                        (dict(cache=dev(5, 8, 80, dtype=F16)), TypeError),
                        (dict(cache=dev(5, 16, 80, dtype=BF)[:, ::2]), ValueError),
                        (dict(norm_w=dev(64, dtype=F16)), TypeError), (dict(norm_w=dev(32, dtype=BF)), ValueError),
                        (dict(q_out=None), ValueError), (dict(q_out=dev(3, 1, 16, dtype=BF)), ValueError),
                        (dict(q_rot=dev(3, 16, 2, dtype=BF).transpose(1, 2)), ValueError)):
        with pytest.raises(err):
            b.mtp_latent_append(**{**append_args(), **change})
    assert lib.calls == []


def test_attn_checks(lib):  # noqa: F811
    ok = dict(q=dev(2, 1, 3, 80, dtype=F16), cache=dev(5, 8, 80, dtype=F16),
              block_table=dev(2, 4, dtype=I32), kv_len=dev(2, dtype=I32),
              out=dev(2, 1, 3, 64, dtype=F16), scale=0.5, lse=dev(2, 1, 3),
              workspace=dev(512, dtype=torch.uint8))
    b.mtp_latent_attn(**ok)
    (name, args), = lib.calls
    assert name == "mtp_latent_attn" and args[1:4] == (240, 0, 80)     # one token: no stride
    assert args[5:8] == (5, 8, 640) and args[9] == 4 and args[11:16] == (2, 1, 3, 64, 16)
    assert args[22] == b.F16 and args[24] == 512
    for change, err in ((dict(q=dev(2, 1, 3, 80)), TypeError), (dict(out=dev(2, 1, 3, 64, dtype=BF)), TypeError),
                        (dict(out=dev(2, 1, 2, 64, dtype=F16)), ValueError),
                        (dict(block_table=dev(3, 4, dtype=I32)), ValueError),
                        (dict(block_table=dev(8, dtype=I32)), ValueError),
                        (dict(kv_len=dev(1, dtype=I32)), ValueError), (dict(lse=dev(5)), ValueError),
                        (dict(cache=dev(5, 8, 64, dtype=F16)), ValueError), (dict(cache=None), ValueError),
                        (dict(workspace=torch.zeros(512, dtype=torch.uint8)), ValueError)):
        with pytest.raises(err):
            b.mtp_latent_attn(**{**ok, **change})
    assert len(lib.calls) == 1


def test_prefill_checks(lib):  # noqa: F811
    ok = dict(q=dev(6, 3, 80, dtype=BF), kv=dev(9, 3, 128, dtype=BF), rot=dev(9, 16, dtype=BF),
              cu_q=dev(3, dtype=I32), cu_k=dev(3, dtype=I32), out=dev(6, 3, 64, dtype=BF), scale=0.5)
    b.mtp_latent_prefill(**ok)
    (name, args), = lib.calls
    assert name == "mtp_latent_prefill" and args[1:3] == (240, 80) and args[4:6] == (384, 128)
    assert args[10:17] == (2, 6, 9, 3, 64, 16, 64)
    for change, err in ((dict(kv=dev(9, 3, 127, dtype=BF)), ValueError), (dict(kv=dev(9, 2, 128, dtype=BF)), ValueError),
                        (dict(rot=dev(9, 16)), TypeError), (dict(cu_k=dev(2, dtype=I32)), ValueError),
                        (dict(cu_q=dev(3)), TypeError), (dict(out=dev(5, 3, 64, dtype=BF)), ValueError),
                        (dict(lse=dev(17)), ValueError)):
        with pytest.raises(err):
            b.mtp_latent_prefill(**{**ok, **change})
    assert len(lib.calls) == 1
