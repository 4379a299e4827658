"""mtp_heads_attn against its formulas in 64 bits: head layouts, lengths from none to thousands,
pages of any height, windows and first tokens, empty rows, refused lengths and pages."""
import pytest
import torch

import verify_spec_greedy_gb300 as lib
from heads_reference import Batch

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("Hq,Hkv,D,P,dtype,layout", [
    (1, 1, 128, 64, BF, "slots"), (32, 8, 128, 64, BF, "slots"), (10, 2, 128, 48, F16, "heads"),
    (3, 3, 64, 8, F16, "both"), (128, 1, 64, 16, BF, "slots"), (14, 2, 96, 24, BF, "both"),
    (6, 2, 256, 128, F16, "heads"), (12, 4, 16, 256, BF, "slots"), (8, 1, 80, 1024, F16, "both"),
    (5, 1, 192, 16, BF, "heads"), (48, 2, 144, 40, F16, "slots"), (16, 2, 256, 8, BF, "both"),
])
def test_heads_and_pages(Hq, Hkv, D, P, dtype, layout):
    rows = [(1, 1), (1, 130), (4, 257), (0, 50), (3, 3), (130, 130), (7, 300), (1, 128), (65, 900)]
    x = Batch(rows, Hq, Hkv, D, P, dtype, seed=D + P, layout=layout, pad=3)
    x.run(lib)
    x.check(heads=sorted({0, Hq // 2, Hq - 1}))


@pytest.mark.parametrize("rows", [
    [(1, 1)], [(1, 600)], [(4, 4)], [(1, 5000)], [(257, 257)], [(1000, 1000)], [(33, 20000)],
    [(300, 4000), (1, 9000)], [(1, n) for n in range(1, 200)], [(4, 100 + 7 * i) for i in range(64)],
    [(16, 128), (17, 129), (15, 127), (32, 256), (31, 255), (33, 257)],
    [(0, 0), (0, 7), (2, 2), (0, 0)], [(700, 1500), (1, 3000), (64, 64), (1, 1)],
])
@pytest.mark.parametrize("D", [128, 256])
def test_lengths(rows, D):
    x = Batch(rows, 8, 2, D, 16, BF, seed=len(rows))
    x.run(lib)
    x.check(heads=[0, 7])


@pytest.mark.parametrize("window,sinks", [
    (1, 0), (1, 1), (5, 3), (64, 0), (127, 4), (128, 128), (129, 200), (300, 4), (1000, 1), (1, 5000),
    (100000, 4), (2 ** 31 - 1, 2 ** 31 - 1), (130, 100000)])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, BF), (10, 2, 64, F16), (4, 1, 256, BF)])
def test_windows(window, sinks, Hq, Hkv, D, dtype):
    rows = [(1, 1), (1, 1000), (200, 1300), (3, 128), (520, 520), (2, 257), (0, 9)]
    x = Batch(rows, Hq, Hkv, D, 16, dtype, seed=window % 1000 + sinks)
    x.run(lib, window, sinks)
    x.check(window, sinks, heads=[0, Hq - 1])


def test_a_query_before_the_first_position_sees_nothing():
    """More queries than the row's length: the first ones lie before position 0."""
    x = Batch([(5, 5), (1, 7)], 4, 2, 64, 16, BF)
    x.run(lib, kv_len=torch.tensor([2, 0], dtype=torch.int32, device="cuda"))
    assert (x.out[:3] == 0).all() and (x.lse[:3] == -torch.inf).all()
    assert (x.out[5] == 0).all() and (x.lse[5] == -torch.inf).all()
    y = Batch([(2, 2)], 4, 2, 64, 16, BF)
    y.k, y.v, y.table = x.k, x.v, x.table[:1].contiguous()
    y.q = x.q[3:5].contiguous()
    y.run(lib)
    assert torch.equal(y.out, x.out[3:5]) and torch.equal(y.lse, x.lse[3:5])


def test_rows_are_their_own():
    """Each row of a mixed batch as if it were alone: the same keys whatever the others are."""
    rows = [(300, 800), (1, 2000), (4, 64), (65, 65), (1, 40)]
    x = Batch(rows, 16, 4, 128, 32, BF, seed=9)
    x.run(lib)
    x.check(heads=[0, 5, 15])


def test_bad_lengths_and_pages_are_taken_as_documented():
    rows = [(1, 64), (2, 100), (1, 40)]
    x = Batch(rows, 4, 2, 128, 16, BF, seed=3)
    # a length beyond the table counts as the table's end, a negative one as none
    far = torch.tensor([64, 100, -5], dtype=torch.int32, device="cuda")
    x.run(lib, kv_len=far)
    assert int(x.status) == lib.STATUS_BAD_PARAM
    assert (x.out[3] == 0).all() and (x.lse[3] == -torch.inf).all()
    # pages out of range are read as zeros
    y = Batch(rows, 4, 2, 128, 16, BF, seed=3)
    y.table[1, 2], y.table[1, 4] = 10 ** 6, -1
    y.keys[1][32:48] = y.values[1][32:48] = 0
    y.keys[1][64:80] = y.values[1][64:80] = 0
    y.run(lib)
    y.check(status=lib.STATUS_BAD_PARAM)


@pytest.mark.parametrize("cu,like", [([0, 4, 2, 9], [0, 4, 4, 9]), ([-3, 5, 6, 100], [0, 5, 6, 9]),
                                     ([2, 3, 3, 8], [2, 3, 3, 8])])
def test_bounds_out_of_order(cu, like):
    x = Batch([(3, 40), (3, 50), (3, 60)], 4, 2, 64, 16, BF, seed=5)
    x.run(lib, cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    got, lse, status = x.out.clone(), x.lse.clone(), int(x.status)
    x.run(lib, cu_q=torch.tensor(like, dtype=torch.int32, device="cuda"))
    assert torch.equal(got, x.out) and torch.equal(lse, x.lse)
    assert status == (lib.STATUS_BAD_PARAM if cu != like else 0) and int(x.status) == 0
    assert (x.out[:like[0]] == 7).all() and (x.out[like[-1]:] == 7).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [[(1, 700), (1, 30)], [(300, 700), (20, 20)]])
def test_nan_and_infinite_queries_stay_alone(D, rows):
    x = Batch(rows, 8, 2, D, 16, BF, seed=1)
    x.q[0, 3, 0] = float("nan")
    x.q[0, 4, 1] = float("inf")
    x.run(lib)
    assert x.out[0, 3].isnan().all() and x.lse[0, 3].isnan()
    assert x.out[0, 4].isnan().all() and x.lse[0, 4].isnan()
    x.q[0, 3:5] = 0
    out, lse = x.out.clone(), x.lse.clone()
    x.run(lib)
    out[0, 3:5], lse[0, 3:5] = x.out[0, 3:5], x.lse[0, 3:5]
    assert torch.equal(out, x.out) and torch.equal(lse, x.lse)
    x.check(heads=[0, 3, 4, 7])


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("rows", [[(1, 2000)], [(200, 2000)]])
def test_scores_far_apart(dtype, rows):
    """Scores of some +-200: the weights' exponents span the whole range, and the maximum rises
    late."""
    x = Batch(rows, 4, 1, 128, 32, dtype, seed=4, std=4.0)
    x.run(lib)
    x.check()


def test_the_same_call_twice_and_in_a_graph():
    x = Batch([(4, 900 + 31 * i) for i in range(40)], 16, 4, 128, 16, BF, seed=6)
    x.run(lib)
    out, lse = x.out.clone(), x.lse.clone()
    x.run(lib)
    assert torch.equal(out, x.out) and torch.equal(lse, x.lse)
    args = dict(out=x.out, lse=x.lse, workspace=x.ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lib.mtp_heads_attn(x.q, x.k, x.v, x.table, x.cu, x.kv_len, scale=x.scale, **args)
    x.kv_len -= 300  # the graph reads the lengths when it runs
    x.rows = [(n, m - 300) for n, m in x.rows]
    x.keys, x.values = [k[:-300] for k in x.keys], [v[:-300] for v in x.values]
    x.out.fill_(7.0)
    for _ in range(3):
        graph.replay()
    x.check(heads=[0, 15])


def test_two_streams_with_a_workspace_each():
    a = Batch([(1, 3000), (4, 500)], 8, 2, 128, 16, BF, seed=7)
    b = Batch([(64, 700), (1, 1)], 8, 2, 128, 16, BF, seed=8)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        with torch.cuda.stream(s):
            a.run(lib)
        with torch.cuda.stream(t):
            b.run(lib)
    torch.cuda.synchronize()
    a.check(heads=[0, 7])
    b.check(heads=[0, 7])


def test_without_lse_and_status():
    x = Batch([(3, 200), (70, 70)], 4, 2, 96, 24, F16, seed=2)
    x.run(lib)
    out = x.out.clone()
    x.run(lib, lse=None, status=None)
    assert torch.equal(out, x.out)


def test_pages_past_32_bit_offsets():
    """A cache of 2^31 elements and more: the last pages' offsets need 64 bits."""
    P, Hkv, D = 128, 8, 128
    pages = 2 ** 31 // (P * Hkv * D) + 40
    k = torch.zeros(pages, P, Hkv, D, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    x = Batch([(2, 500), (130, 300)], 16, 8, D, P, BF, seed=11)
    n = x.k.shape[0]
    k[-n:], v[-n:] = x.k, x.v
    x.k, x.v = k, v
    x.table = torch.where(x.table >= 0, x.table + (pages - n), x.table)
    x.run(lib)
    x.check(heads=[0, 15])


# Heads of up to 64 elements with few (token, head) rows a row: units of 32 rows.
SMALL = [
    (4, 4, 64, 16, BF), (64, 8, 64, 16, F16), (10, 2, 48, 24, BF), (32, 1, 64, 64, F16), (40, 1, 16, 8, BF),
    (128, 1, 64, 128, BF), (12, 4, 32, 48, F16),
]


@pytest.mark.parametrize("Hq,Hkv,D,P,dtype", SMALL)
@pytest.mark.parametrize("rows", [
    [(1, 1)], [(1, 5000)], [(1, 1), (0, 40), (1, 128), (0, 0), (1, 129), (1, 1000), (0, 3), (0, 1)],
    [(1, n) for n in range(1, 150)], [(2, 3), (0, 8), (0, 9), (5, 700)] + [(0, 1)] * 40, [(0, 5)] * 3 + [(1, 2)],
])
def test_few_rows_of_small_heads(Hq, Hkv, D, P, dtype, rows):
    x = Batch(rows, Hq, Hkv, D, P, dtype, seed=len(rows) + D)
    x.run(lib)
    x.check(heads=sorted({0, Hq // 2, Hq - 1}))


@pytest.mark.parametrize("window,sinks", [
    (1, 0), (1, 1), (5, 3), (127, 4), (128, 128), (129, 200), (300, 4), (1, 5000), (2 ** 31 - 1, 2 ** 31 - 1),
    (130, 100000)])
@pytest.mark.parametrize("Hq,Hkv,D,P,dtype", SMALL[:3])
def test_windows_of_few_rows_of_small_heads(window, sinks, Hq, Hkv, D, P, dtype):
    rows = [(1, 1), (1, 1000), (3, 1300), (3, 128), (1, 520), (2, 257), (0, 9), (4, 4), (1, 129)]
    x = Batch(rows, Hq, Hkv, D, P, dtype, seed=window % 1000 + sinks)
    x.run(lib, window, sinks)
    x.check(window, sinks, heads=[0, Hq - 1])
