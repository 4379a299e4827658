"""The grouped heads' and the pages' C entry points on the host: exported as declared, sizes, types,
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


@pytest.mark.parametrize("header,want", [
    ("heads.h", {"mtp_heads_append", "mtp_heads_attn", "mtp_heads_attn_workspace_bytes"}),
    ("pages.h", {"mtp_pages_resize", "mtp_pages_fork", "mtp_pages_compact", "mtp_pages_copy"})])
def test_every_declared_symbol_is_exported(so, header, want):
    src = open(os.path.join(ROOT, "include", "libmtpspec", header)).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"^(?:int|size_t)\s+(\w+)\s*\(", src, flags=re.M))
    assert names == want
    for n in names:
        assert hasattr(so, n) and hasattr(pkg, n)
    main = open(os.path.join(ROOT, "include", "libmtpspec.h")).read()
    assert f'#include "libmtpspec/{header}"' in main


def test_the_new_status_bit():
    src = open(os.path.join(ROOT, "include", "libmtpspec", "pages.h")).read()
    assert int(re.search(r"MTPSPEC_STATUS_NO_PAGES (0x\w+)", src)[1], 16) == pkg.STATUS_NO_PAGES
    assert pkg.STATUS_NO_PAGES & (pkg.STATUS_BAD_DRAFT_ID | pkg.STATUS_BAD_PARAM | pkg.STATUS_TIMEOUT) == 0


APPEND = dict(k=P, k_tok=512, k_head=128, v=P, v_tok=512, v_head=128, k_norm_w=None, cos_sin=P, max_pos=100,
              R=64, interleaved=0, tok_row=P, positions=P, T=0, Hkv=4, D=128, block_table=P, B=1, max_pages=2,
              k_cache=P, v_cache=P, num_pages=2, page_size=64, page_stride=64 * 512, slot_stride=512,
              head_stride=128, q=P, q_tok=16 * 128, q_head=128, q_norm_w=None, q_out=P, q_out_tok=16 * 128,
              q_out_head=128, Hq=16, eps=0.0, dtype=1, status=None, stream=None)
ONE = dict(T=1)


@pytest.mark.parametrize("change,code", [
    ({}, OK), (dict(dtype=0), DTYPE), (dict(dtype=3), DTYPE), (dict(dtype=2), OK), (dict(T=-1), SHAPE),
    (dict(T=(1 << 20) + 1), SHAPE), (dict(D=8), SHAPE), (dict(D=120), SHAPE), (dict(D=272), SHAPE),
    (dict(R=8), SHAPE), (dict(R=144), SHAPE), (dict(R=24), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hkv=3), SHAPE),
    (dict(Hq=2), SHAPE), (dict(Hq=1028), SHAPE), (dict(Hq=0, q=None, q_out=None), OK), (dict(B=0), SHAPE),
    (dict(B=(1 << 20) + 1), SHAPE), (dict(max_pos=0), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(num_pages=0), SHAPE), (dict(page_size=4), SHAPE), (dict(page_size=12), SHAPE),
    (dict(slot_stride=384), SHAPE), (dict(slot_stride=516), SHAPE), (dict(head_stride=64), SHAPE),
    (dict(page_stride=64 * 512 - 8), SHAPE), (dict(page_stride=-8), SHAPE),
    (dict(slot_stride=128, head_stride=64 * 128), OK), (dict(slot_stride=128, head_stride=63 * 128), SHAPE),
    (dict(T=2, k_tok=64), SHAPE), (dict(k_head=-128), SHAPE), (dict(T=2, v_tok=516), SHAPE),
    (dict(q_head=64), SHAPE), (dict(T=2, q_out_tok=16 * 128 - 8), SHAPE), (dict(q_out=None), ARG),
    (dict(q=None), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (ONE | dict(k=None), ARG), (ONE | dict(v=None), ARG), (ONE | dict(cos_sin=None), ARG),
    (ONE | dict(tok_row=None), ARG), (ONE | dict(positions=None), ARG), (ONE | dict(block_table=None), ARG),
    (ONE | dict(k_cache=None), ARG), (ONE | dict(v_cache=C.c_void_p(4104)), ARG),
    (ONE | dict(k=C.c_void_p(4104)), ARG), (ONE | dict(q_norm_w=C.c_void_p(4104)), ARG),
    (ONE | dict(cos_sin=C.c_void_p(4100)), ARG), (ONE | dict(positions=C.c_void_p(4097)), ARG),
    (ONE | dict(q_out=C.c_void_p(4104)), ARG), (ONE | dict(status=C.c_void_p(4098)), ARG),
])
def test_append_refusals(so, change, code):
    assert so.mtp_heads_append(*{**APPEND, **change}.values()) == code


ATTN = dict(q=P, q_tok=16 * 128, q_head=128, k_cache=P, v_cache=P, num_pages=2, page_size=64,
            page_stride=64 * 512, slot_stride=512, head_stride=128, block_table=P, max_pages=2, cu_q=P,
            kv_len=P, B=1, Tq=0, Hq=16, Hkv=4, D=128, window=0, sinks=0, scale=0.1, out=P, out_tok=16 * 128,
            out_head=128, lse=None, dtype=1, workspace=None, workspace_bytes=0, status=None, stream=None)
Q1 = dict(Tq=1)


@pytest.mark.parametrize("change,code", [
    ({}, OK), (dict(dtype=0), DTYPE), (dict(dtype=2), OK), (dict(B=0), SHAPE), (dict(B=65537), SHAPE),
    (dict(Tq=-1), SHAPE), (dict(Tq=(1 << 24) + 1), SHAPE), (dict(Tq=1 << 24, Hq=128), SHAPE),
    (dict(Hq=15), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hq=512, Hkv=2), SHAPE), (dict(D=250), SHAPE),
    (dict(D=272), SHAPE), (dict(page_size=63), SHAPE), (dict(num_pages=0), SHAPE),
    (dict(slot_stride=400), SHAPE), (dict(Tq=2, q_tok=64), SHAPE), (dict(q_head=132), SHAPE),
    (dict(out_head=64), SHAPE), (dict(Tq=2, out_tok=8), SHAPE), (dict(window=-1), ARG), (dict(sinks=-1), ARG),
    (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (Q1 | dict(q=None), ARG), (Q1 | dict(k_cache=None), ARG),
    (Q1 | dict(v_cache=None), ARG), (Q1 | dict(block_table=None), ARG), (Q1 | dict(cu_q=None), ARG),
    (Q1 | dict(kv_len=None), ARG), (Q1 | dict(out=None), ARG), (Q1 | dict(q=C.c_void_p(4104)), ARG),
    (Q1 | dict(out=C.c_void_p(4104)), ARG), (Q1 | dict(cu_q=C.c_void_p(4098)), ARG),
    (Q1 | dict(lse=C.c_void_p(4098)), ARG), (Q1, WORKSPACE),
    (Q1 | dict(workspace=P, workspace_bytes=1000), WORKSPACE),
    (Q1 | dict(workspace=C.c_void_p(4112), workspace_bytes=1 << 40), ARG),
])
def test_attn_refusals(so, change, code):
    assert so.mtp_heads_attn(*{**ATTN, **change}.values()) == code


def test_attn_workspace():
    ws = pkg.mtp_heads_attn_workspace_bytes
    for good in ((1, 1, 1, 1, 16), (256, 1024, 32, 8, 128), (1, 8192, 16, 2, 256), (65536, 65536, 8, 8, 64)):
        n = ws(*good)
        assert 0 < n <= 64 << 20 and n % 256 == 0
    for bad in ((0, 1, 16, 4, 128), (1, 0, 16, 4, 128), (1, -1, 16, 4, 128), (1, 1, 16, 3, 128), (1, 1, 16, 4, 24),
                (1, 1 << 24, 128, 8, 128)):
        assert ws(*bad) == 0


RESIZE = dict(keep=P, lens=P, block_table=P, held=P, refs=P, B=4, max_pages=8, num_pages=100, page_size=16,
              copies=P, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(B=0), SHAPE), (dict(B=16385), SHAPE), (dict(max_pages=0), SHAPE), (dict(num_pages=0), SHAPE),
    (dict(num_pages=1 << 31), SHAPE), (dict(B=16384, max_pages=1 << 27), SHAPE), (dict(page_size=0), SHAPE),
    (dict(page_size=(1 << 24) + 1), SHAPE), (dict(keep=None), ARG), (dict(lens=None), ARG),
    (dict(block_table=None), ARG), (dict(held=None), ARG), (dict(refs=None), ARG),
    (dict(copies=C.c_void_p(4098)), ARG), (dict(refs=C.c_void_p(4097)), ARG), (dict(status=C.c_void_p(2)), ARG)])
def test_resize_refusals(so, change, code):
    assert so.mtp_pages_resize(*{**RESIZE, **change}.values()) == code


FORK = dict(src=P, dst=P, n=0, block_table=P, held=P, refs=P, B=4, max_pages=8, num_pages=100, status=None,
            stream=None)


@pytest.mark.parametrize("change,code", [
    ({}, OK), (dict(n=-1), SHAPE), (dict(n=1025), SHAPE), (dict(B=0), SHAPE), (dict(n=1, src=None), ARG),
    (dict(n=1, dst=None), ARG), (dict(n=1, refs=None), ARG), (dict(n=1, held=C.c_void_p(4097)), ARG)])
def test_fork_refusals(so, change, code):
    assert so.mtp_pages_fork(*{**FORK, **change}.values()) == code


COMPACT = dict(block_table=P, held=P, refs=P, B=4, max_pages=8, num_pages=100, moves=P, n_moves=P, status=None,
               stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(B=0), SHAPE), (dict(num_pages=0), SHAPE), (dict(moves=None), ARG), (dict(n_moves=None), ARG),
    (dict(block_table=None), ARG), (dict(moves=C.c_void_p(4098)), ARG)])
def test_compact_refusals(so, change, code):
    assert so.mtp_pages_compact(*{**COMPACT, **change}.values()) == code


def copy_args(caches=(4096, 8192), **change):
    a = dict(caches=(C.c_void_p * len(caches))(*caches) if caches else None, n_caches=len(caches or (0,)),
             num_pages=10,
             page_bytes=256, page_stride=256, pairs=P, n=0, n_pairs=None, status=None, stream=None) | change
    return a.values()


@pytest.mark.parametrize("change,code", [
    ({}, OK), (dict(n_caches=0), SHAPE), (dict(n_caches=65), SHAPE), (dict(num_pages=0), SHAPE),
    (dict(page_bytes=8), SHAPE), (dict(page_bytes=264), SHAPE), (dict(page_stride=264), SHAPE),
    (dict(page_stride=128), SHAPE), (dict(n=-1), SHAPE), (dict(n=(1 << 30) + 1), SHAPE),
    (dict(n=1, pairs=None), ARG), (dict(n=1, caches=None), ARG), (dict(n=1, pairs=C.c_void_p(4098)), ARG),
    (dict(n=1, n_pairs=C.c_void_p(4098)), ARG)])
def test_copy_refusals(so, change, code):
    assert so.mtp_pages_copy(*copy_args(**change)) == code


def test_copy_refuses_a_cache(so):
    assert so.mtp_pages_copy(*copy_args((4096, 0), n=1)) == ARG
    assert so.mtp_pages_copy(*copy_args((4096, 4104), n=1)) == ARG


# ---------------------------------------------------------------- the binding

def append_args(T=3, Hq=4, Hkv=2, D=64, dtype=BF):
    qkv = dev(T, Hq + 2 * Hkv, D + 16, dtype=dtype)[..., :D]
    return dict(k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], cos_sin=dev(9, 32), tok_row=dev(T, dtype=I32),
                positions=dev(T, dtype=I32), block_table=dev(2, 4, dtype=I32),
                k_cache=dev(5, 8, Hkv, D, dtype=dtype), v_cache=dev(5, 8, Hkv, D, dtype=dtype),
                k_norm_w=dev(D, dtype=dtype), q=qkv[:, :Hq], q_out=dev(T, Hq, D, dtype=dtype),
                q_norm_w=dev(D, dtype=dtype), eps=0.5, interleaved=True)


def test_append_passes_strides(lib):  # noqa: F811
    b.mtp_heads_append(**append_args())
    (name, a), = lib.calls
    assert name == "mtp_heads_append"
    assert a[1:3] == a[4:6] == (8 * 80, 80) and a[8:11] == (9, 32, 1) and a[13:16] == (3, 2, 64)
    assert a[17:19] == (2, 4) and a[21:26] == (5, 8, 1024, 128, 64)
    assert a[27:29] == (8 * 80, 80) and a[31:34] == (256, 64, 4) and a[35] == b.BF16


def test_append_refuses(lib):  # noqa: F811
    for change, err in ((dict(k=torch.zeros(3, 2, 64, dtype=BF)), ValueError), (dict(k=dev(3, 2, 64)), TypeError),
                        (dict(v=dev(3, 2, 64, dtype=F16)), TypeError), (dict(v=dev(3, 3, 64, dtype=BF)), ValueError),
                        (dict(k=None), ValueError), (dict(k_cache=None), ValueError),
                        (dict(k_cache=dev(5, 8, 2, 80, dtype=BF)), ValueError),
                        (dict(v_cache=dev(5, 8, 2, 64, dtype=F16)), TypeError),
                        (dict(v_cache=dev(5, 2, 8, 64, dtype=BF).transpose(1, 2)), ValueError),
                        (dict(k_norm_w=dev(64)), TypeError), (dict(q_norm_w=dev(32, dtype=BF)), ValueError),
                        (dict(q=None), ValueError), (dict(q_out=None), ValueError),
                        (dict(q_out=dev(3, 4, 48, dtype=BF)), ValueError),
                        (dict(cos_sin=dev(9, 32, dtype=BF)), TypeError), (dict(tok_row=dev(2, dtype=I32)), ValueError),
                        (dict(positions=dev(3)), TypeError),
                        (dict(q=dev(3, 64, 4, dtype=BF).transpose(1, 2)), ValueError)):
        with pytest.raises(err):
            b.mtp_heads_append(**{**append_args(), **change})
    assert lib.calls == []


def test_attn_checks(lib):  # noqa: F811
    ok = dict(q=dev(6, 4, 64, dtype=F16), k_cache=dev(5, 2, 8, 64, dtype=F16).transpose(1, 2),
              v_cache=dev(5, 2, 8, 64, dtype=F16).transpose(1, 2), block_table=dev(3, 4, dtype=I32),
              cu_q=dev(4, dtype=I32), kv_len=dev(3, dtype=I32), out=dev(6, 4, 64, dtype=F16), scale=0.5, window=7,
              sinks=2, lse=dev(6, 4), workspace=dev(512, dtype=torch.uint8))
    b.mtp_heads_attn(**ok)
    (name, a), = lib.calls
    assert name == "mtp_heads_attn" and a[1:3] == (256, 64) and a[5:10] == (5, 8, 1024, 64, 512)
    assert a[11] == 4 and a[14:21] == (3, 6, 4, 2, 64, 7, 2) and a[26] == b.F16 and a[28] == 512
    for change, err in ((dict(q=dev(6, 4, 64)), TypeError), (dict(q=None), ValueError),
                        (dict(out=dev(6, 4, 64, dtype=BF)), TypeError), (dict(out=dev(6, 4, 48, dtype=F16)), ValueError),
                        (dict(k_cache=dev(5, 8, 2, 64, dtype=F16)), ValueError),
                        (dict(v_cache=None), ValueError), (dict(cu_q=dev(3, dtype=I32)), ValueError),
                        (dict(kv_len=dev(2, dtype=I32)), ValueError), (dict(kv_len=dev(3)), TypeError),
                        (dict(lse=dev(23)), ValueError), (dict(block_table=dev(12, dtype=I32)), ValueError),
                        (dict(workspace=torch.zeros(512, dtype=torch.uint8)), ValueError)):
        with pytest.raises(err):
            b.mtp_heads_attn(**{**ok, **change})
    assert len(lib.calls) == 1


def test_pages_checks(lib):  # noqa: F811
    table, held, refs = dev(4, 8, dtype=I32), dev(4, dtype=I32), dev(100, dtype=I32)
    keep, lens, copies = dev(4, dtype=I32), dev(4, dtype=I32), dev(4, 2, dtype=I32)
    b.mtp_pages_resize(keep, lens, table, held, refs, 16, copies)
    b.mtp_pages_fork(dev(3, dtype=I32), dev(3, dtype=I32), table, held, refs)
    b.mtp_pages_compact(table, held, refs, dev(50, 2, dtype=I32), dev(1, dtype=I32))
    caches = [dev(10, 16, 2, 64, dtype=BF) for _ in range(3)]
    b.mtp_pages_copy(caches, copies)
    b.mtp_pages_copy([dev(10, 40, dtype=BF)[:, :32]], copies, n_pairs=dev(1, dtype=I32))
    calls = dict((n, a) for n, a in lib.calls[:3])
    assert calls["mtp_pages_resize"][5:9] == (4, 8, 100, 16)
    assert calls["mtp_pages_fork"][2] == 3 and calls["mtp_pages_fork"][6:9] == (4, 8, 100)
    assert calls["mtp_pages_compact"][3:6] == (4, 8, 100)
    assert lib.calls[3][1][1:5] == (3, 10, 16 * 2 * 64 * 2, 16 * 2 * 64 * 2) and lib.calls[3][1][6] == 4
    assert lib.calls[4][1][1:5] == (1, 10, 64, 80)
    n = len(lib.calls)
    host = torch.zeros(4, dtype=I32)
    for call in (lambda: b.mtp_pages_resize(host, lens, table, held, refs, 16),
                 lambda: b.mtp_pages_resize(dev(3, dtype=I32), lens, table, held, refs, 16),
                 lambda: b.mtp_pages_resize(keep, lens, dev(32, dtype=I32), held, refs, 16),
                 lambda: b.mtp_pages_resize(keep, lens, table, dev(3, dtype=I32), refs, 16),
                 lambda: b.mtp_pages_resize(keep, lens, table, held, refs, 16, dev(4, dtype=I32)),
                 lambda: b.mtp_pages_fork(dev(3, dtype=I32), dev(2, dtype=I32), table, held, refs),
                 lambda: b.mtp_pages_compact(table, held, refs, dev(49, 2, dtype=I32), dev(1, dtype=I32)),
                 lambda: b.mtp_pages_copy([], copies), lambda: b.mtp_pages_copy(caches, dev(8, dtype=I32)),
                 lambda: b.mtp_pages_copy([dev(10, 2, 16, dtype=BF).transpose(1, 2)], copies),
                 lambda: b.mtp_pages_copy([caches[0], dev(10, 16, 2, 32, dtype=BF)], copies),
                 lambda: b.mtp_pages_copy([torch.zeros(10, 16, dtype=BF)], copies)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        b.mtp_pages_resize(dev(4), lens, table, held, refs, 16)
    assert len(lib.calls) == n
