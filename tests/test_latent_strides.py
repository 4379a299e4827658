"""Outputs whose axes overlap are refused on the host: strides that are each as long as an item,
but with which two items share elements.  Layouts in any order of their axes go through, to the
next check (the first pointer, which is missing)."""
import ctypes as C
import itertools

import pytest

from test_latent_abi import APPEND, ATTN, PREFILL, so  # noqa: F401

ARG, SHAPE = -1, -3


def overlaps(item, axes):
    """By setting every element's place down."""
    seen = set()
    for at in itertools.product(*(range(n) for _, n in axes)):
        first = sum(i * s for i, (s, _) in zip(at, axes))
        place = set(range(first, first + item))
        if seen & place:
            return True
        seen |= place
    return False


def nested(item, axes):
    span = item
    for s, n in sorted(a for a in axes if a[1] > 1):
        if s < span:
            return False
        span += s * (n - 1)
    return True


TWO = [(64, 64), (128, 64), (64, 192), (192, 64), (64, 184), (128, 128), (72, 216), (208, 72), (64, 128)]


@pytest.mark.parametrize("tok,head", TWO)
def test_append_and_prefill(so, tok, head):  # noqa: F811
    want = ARG if nested(64, [(tok, 3), (head, 3)]) else SHAPE
    assert (want == SHAPE) >= overlaps(64, [(tok, 3), (head, 3)])
    a = {**APPEND, "T": 3, "Hq": 3, "q_rot_tok": 192, "q_out_tok": tok, "q_out_head": head, "latent": None}
    assert so.mtp_latent_append(*a.values()) == want
    a = {**PREFILL, "Tq": 3, "Tk": 3, "Hq": 3, "q_tok": 576, "kv_tok": 768, "V": 64, "out_tok": tok,
         "out_head": head, "q": None}
    assert so.mtp_latent_prefill(*a.values()) == want


@pytest.mark.parametrize("strides", [(384, 192, 64), (64, 128, 384), (192, 64, 384), (64, 64, 64), (384, 64, 64),
                                     (384, 128, 64), (376, 192, 64), (128, 384, 64), (400, 200, 72), (192, 384, 64)])
def test_attn(so, strides):  # noqa: F811
    axes = list(zip(strides, (2, 2, 3)))
    want = ARG if nested(64, axes) else SHAPE
    assert (want == SHAPE) >= overlaps(64, axes)
    a = {**ATTN, "B": 2, "T": 2, "Hq": 3, "L": 64, "q_row": 2 * 3 * 128, "q_tok": 3 * 128, "q_head": 128,
         "page_stride": 64 * 128, "out_row": strides[0], "out_tok": strides[1], "out_head": strides[2], "q": None}
    assert so.mtp_latent_attn(*a.values()) == want


def test_an_axis_of_one_may_have_any_stride(so):  # noqa: F811
    a = {**ATTN, "B": 2, "T": 1, "Hq": 3, "L": 64, "q_row": 3 * 128, "q_tok": 0, "q_head": 128,
         "page_stride": 64 * 128, "out_row": 192, "out_tok": 0, "out_head": 64, "q": None}
    assert so.mtp_latent_attn(*a.values()) == ARG
    assert so.mtp_latent_attn(*{**a, "out_row": 128}.values()) == SHAPE
    big = (1 << 39) - 8                             # the longest stride: nothing overflows
    assert so.mtp_latent_attn(*{**a, "B": 1 << 20, "q_row": big, "out_row": big}.values()) == ARG
    assert so.mtp_latent_append(*{**APPEND, "T": 1, "Hq": 1, "q_out_tok": 0, "q_out_head": 0,
                                  "latent": C.c_void_p(None)}.values()) == ARG
