"""mtp_heads_attn at the largest length, 2^31 - 256 positions: pages that many entries of the table share,
and a few keys, next to both ends, whose scores stand 60 above all others.

Those keys' scores are equal, so that their weights are the same power of two and the output is the mean
of their values: off by a rounding (half a step), by some roundings in fp32, and by the weights of all
other keys, 2^31 e^-60 < 2^-55 of it."""
import pytest
import torch

import verify_spec_greedy_gb300 as lib
from latent_reference import half_step

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16
P, LEN = 1 << 22, (1 << 31) - 256


@pytest.mark.parametrize("window,sinks", [(0, 0), (2000, 0), (2000, 6), (2, 1), (LEN - 1, 0), (LEN - 4, 3),
                                          (LEN - 100, 200), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("D,dtype", [(16, BF), (16, F16), (80, BF), (144, F16)])  # both kernels, all tiles
def test_the_largest_length(D, dtype, window, sinks):
    entries, T = (1 << 31) // P, 3
    g = torch.Generator(device="cuda").manual_seed(D)
    k = torch.zeros(3, P, 1, D, dtype=dtype, device="cuda")
    v = torch.randn(3, P, 1, D, generator=g, device="cuda").to(dtype)
    table = torch.zeros(1, entries, dtype=torch.int32, device="cuda")  # page 0 but at the ends
    table[0, 0], table[0, -1] = 2, 1
    high = [0, 2, 5, 127, 150, LEN - 1999, LEN - 700, LEN - 3, LEN - 2, LEN - 1]
    page = {0: 2, entries - 1: 1}
    for n in high:
        k[page[n // P], n % P, 0, 0] = 1
    k[1, LEN % P:], v[1, LEN % P:] = float("nan"), float("nan")
    q = torch.zeros(T, 2, D, dtype=dtype, device="cuda")
    q[:, :, 0] = 64
    out = torch.empty_like(q)
    lse = torch.empty(T, 2, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(lib.mtp_heads_attn_workspace_bytes(1, T, 2, 1, D), dtype=torch.uint8, device="cuda")
    lib.mtp_heads_attn(q, k, v, table, torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                       torch.tensor([LEN], dtype=torch.int32, device="cuda"), out, 60 / 64, window=window,
                       sinks=sinks, lse=lse, workspace=ws, status=status)
    assert int(status) == 0
    for i in range(T):
        n = LEN - T + i
        seen = [j for j in high if j <= n and (window == 0 or j > n - window or j < sinks)]
        values = torch.stack([v[page[j // P], j % P, 0] for j in seen]).double()
        mean, size = values.mean(0), values.abs().mean(0)
        tol = half_step(dtype) * mean.abs() + 2.0 ** -18 * size + torch.finfo(dtype).tiny
        for h in range(2):
            assert ((out[i, h].double() - mean).abs() <= tol).all()
            want = 60 + torch.log(torch.tensor(float(len(seen)), dtype=torch.float64)).item()
            assert abs(lse[i, h].item() - want) <= 60 * 2.0 ** -20
