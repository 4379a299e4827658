"""mtp_heads_attn with outputs of any layout, in graphs and on streams of its own, and run after
run: both kernels (heads of 64 elements and few tokens a row, and others)."""
import pytest
import torch

import verify_spec_greedy_gb300 as lib
from heads_reference import Batch

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16
FEW = ([(1, 700), (3, 64), (1, 1), (2, 3000), (0, 9), (1, 130)], 8, 2)
MANY = ([(130, 300), (1, 700), (64, 64), (3, 3000), (0, 9), (200, 201)], 8, 2)


def batch(few, D, dtype=BF, **kw):
    rows, Hq, Hkv = FEW if few else MANY
    return Batch(rows, Hq, Hkv, D, 16, dtype, seed=D, **kw)


@pytest.mark.parametrize("layout", ["heads outside", "wide rows", "16-byte rows", "wide heads"])
@pytest.mark.parametrize("few,D", [(True, 64), (True, 48), (True, 16), (False, 64), (False, 128), (False, 144),
                                   (False, 256)])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_outputs_of_any_layout(few, D, layout, dtype):
    x = batch(few, D, dtype)
    T, H = x.Tq, x.Hq
    if layout == "heads outside":
        whole = torch.full((H, T, D), 7.0, dtype=dtype, device="cuda")
        out = whole.transpose(0, 1)
    elif layout == "wide rows":
        whole = torch.full((T, H * D + 8), 7.0, dtype=dtype, device="cuda")
        out = whole[:, :H * D].unflatten(1, (H, D))
    elif layout == "16-byte rows":  # no row starts at a multiple of 32 bytes
        whole = torch.full((T, H, D + 16), 7.0, dtype=dtype, device="cuda")
        out = whole[..., 8:8 + D]
    else:
        whole = torch.full((T, H, D + 8), 7.0, dtype=dtype, device="cuda")
        out = whole[..., :D]
    x.run(lib)
    want = x.out.clone()
    x.check(heads=[0, H - 1])
    written = torch.zeros_like(whole, dtype=torch.bool)
    view = written.as_strided(out.shape, out.stride(), out.storage_offset())
    view.fill_(True)
    x.run(lib, out=out)
    assert torch.equal(out, want)
    assert (whole[~written] == 7).all()  # nothing beside the rows was written


@pytest.mark.parametrize("few", [True, False])
def test_in_a_graph(few):
    x = batch(few, 64)
    x.run(lib)
    x.check(heads=[0, 7])
    want, lse = x.out.clone(), x.lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(3):
            lib.mtp_heads_attn(x.q, x.k, x.v, x.table, x.cu, x.kv_len, x.out, x.scale, lse=x.lse, workspace=x.ws)
    for _ in range(3):
        x.out.fill_(7.0)
        x.lse.fill_(7.0)
        graph.replay()
        assert torch.equal(want, x.out) and torch.equal(lse, x.lse)


@pytest.mark.parametrize("few", [True, False])
def test_on_two_streams(few):
    a, b = batch(few, 64), batch(few, 48, F16)
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


@pytest.mark.parametrize("few,D", [(True, 64), (False, 64), (False, 128), (False, 256)])
def test_the_same_bits_run_after_run(few, D):
    x = batch(few, D)
    x.run(lib)
    out, lse = x.out.clone(), x.lse.clone()
    for i in range(30):
        if i % 3 == 0:  # other work beside it changes when its parts end
            torch.randn(1 << 22, device="cuda").sort()
        x.run(lib)
        assert torch.equal(out, x.out) and torch.equal(lse, x.lse)
