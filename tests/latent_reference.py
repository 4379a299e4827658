"""The latent attention's formulas in 64 bits (torch on the CPU or the GPU), with bounds on
what 16-bit inputs, fp32 sums and weights rounded to the inputs' type may differ by.

u = finfo(type).eps / 2 is the relative error of one rounding.  An output is sum_n p_n v_n:
  - each weight is rounded once:                      u * A,  A = sum_n p_n |v_n|
  - a score's fp32 sum of K products is off by at most e_s = 2^-22 * K * scale * sum |q k|
    (2^-22 a step: the tensor cores' additions may truncate), which moves a weight and the
    sum below it by a factor of e^(2 e_s):            2 e_s * A
  - n additions of fp32 in numerator and denominator, and the exponential's own error
    (a few 2^-23):                                    (n + 16) * 2^-22 * A
  - the output is rounded once:                       u * |out|
and ln sum_n e^(s_n) by e_s + (n + 16) * 2^-22 + 2^-22 |lse|."""
import torch

E32 = 2.0 ** -22


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rotate(x, cos_sin, interleaved):
    """x[..., R] (float64) turned by the angles of cos_sin[..., R]."""
    R = x.shape[-1]
    c, s = cos_sin[..., :R // 2].double(), cos_sin[..., R // 2:].double()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :R // 2], x[..., R // 2:])
    y0, y1 = a * c - b * s, a * s + b * c
    out = torch.empty_like(x)
    if interleaved:
        out[..., 0::2], out[..., 1::2] = y0, y1
    else:
        out[..., :R // 2], out[..., R // 2:] = y0, y1
    return out


def rms_norm(x, w, eps):
    x = x.double()
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def attend(q, keys, values, seen, scale, dtype):
    """Rows q[m, K] over keys[n, K] and values[n, V], row i seeing the first seen[i] keys:
    (out, lse, bound on out, bound on lse), float64."""
    q, keys, values = q.double(), keys.double(), values.double()
    n, K = keys.shape
    hidden = torch.arange(n, device=q.device) >= seen[:, None]
    s = (q @ keys.T * scale).masked_fill(hidden, -torch.inf)
    size = (q.abs() @ keys.abs().T * scale).masked_fill(hidden, 0.0)
    e_s = E32 * K * (size.amax(1) if n else torch.zeros(len(q), device=q.device).double())
    lse = torch.logsumexp(s, 1) if n else torch.full((len(q),), -torch.inf, device=q.device).double()
    p = torch.where(hidden, 0.0, torch.exp(s - torch.where(lse > -torch.inf, lse, 0.0)[:, None]))
    out, A = p @ values, p @ values.abs()
    u = half_step(dtype)
    wobble = (n + 16) * E32
    tol = u * out.abs() + (u + 2 * e_s[:, None] + wobble) * 1.01 * A
    lse_tol = e_s + wobble + E32 * torch.where(lse > -torch.inf, lse.abs(), 0.0)
    return out, lse, tol, lse_tol


def check(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - tol
    assert (over <= 0).all(), f"{what}: off by {over.max().item():.3e} more than allowed"


def check_lse(got, want, tol, what):
    got = got.double()
    empty = want == -torch.inf
    assert torch.equal(got == -torch.inf, empty), f"{what}: empty rows"
    check(torch.where(empty, 0.0, got), torch.where(empty, 0.0, want), tol, what)
