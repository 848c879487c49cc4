"""Plain 64-bit forms of the attention operators, and bounds on the error that the
kernels' stated arithmetic allows (not collected: no test_ prefix).

Bounds.  With x the scores in natural units, a score is off by at most
  dx = gamma(d) * scale * sum |q||k| + 2^-21 |x|
(fp32 sums as in serving_ref.gamma, then at most six rounded factors), which is the
relative error of its probability before the exponential's own (two units in the last
place, 2^-22) and the rounding to the product's type (half a step: 2^-11 for fp16, 2^-8
for bf16; fp16 also 2^-25 of the largest, in its subnormals).  Both sums over n keys are
off by gamma(n); the output is rounded to bf16, half a step, 2^-8.
"""
import math

import torch

from serving_ref import gamma

MAG = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def rope(x, positions, inv_freq, sections, interleaved):
    """float64 [t, heads, d]."""
    y = x.double().clone()
    n = sum(sections)
    i = 0
    for a, count in enumerate(sections):
        for _ in range(count):
            ang = positions[a].double() * inv_freq[i].double()
            c, s = ang.cos()[:, None], ang.sin()[:, None]
            p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            x1, x2 = x[..., p].double(), x[..., q].double()
            y[..., p], y[..., q] = x1 * c - x2 * s, x2 * c + x1 * s
            i += 1
    return y


def rows(kv, kv_sf, which, slots):
    """The cache's rows in `slots` (valid ones) before the global scale: float64 [t, heads, d]."""
    page = kv.shape[3]
    at, off = slots.long() // page, slots.long() % page
    codes = kv[at, which, :, off].long()
    sf = kv_sf.view(torch.float8_e4m3fn)[at, which, :, :, off].double()
    mag = torch.tensor(MAG + [-v for v in MAG], dtype=torch.float64, device=kv.device)
    v = torch.stack([mag[codes & 15], mag[codes >> 4]], -1).flatten(-2)
    return v * sf.repeat_interleave(16, -1)


def attend(q, k, v, scale, seen, half_step, tiny):
    """q [rows, d], k, v [keys, d] float64; seen [rows, keys].  Returns out, lse, and bounds on both."""
    d, n = q.shape[1], max(1, k.shape[0])
    x = q @ k.t() * scale
    dx = (gamma(d) * (q.abs() @ k.abs().t()) * scale + 2.0 ** -21 * x.abs()).masked_fill(~seen, 0).amax(-1, keepdim=True) \
        if k.shape[0] else torch.zeros(q.shape[0], 1, dtype=torch.float64, device=q.device)
    x = x.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None])
    va = torch.where(v.isfinite(), v, torch.zeros_like(v))
    out = p @ va
    rel = half_step + 2 * (2 * dx + gamma(n) + 2.0 ** -20)
    err = (p @ va.abs()) * rel + tiny * (seen.double() @ va.abs())
    bound = err + (out.abs() + err) * 2.0 ** -8 + 1e-37
    dl = dx[:, 0] + gamma(n) + 2.0 ** -20 + 2.0 ** -21 * lse.abs().masked_fill(lse == -math.inf, 0)
    return out, lse, bound, dl


def worst(got, ref, bound):
    return ((got.double() - ref).abs() / bound).max().item() if got.numel() else 0.0


def same_lse(got, ref, bound):
    empty = ref == -math.inf
    if not torch.equal(got == -math.inf, empty):
        return False
    return worst(got[~empty], ref[~empty], bound[~empty]) <= 1.0
