"""Plain 64-bit forms of the serving operators, and bounds on the error that the
kernels' stated arithmetic allows (not collected: no test_ prefix).

Bounds.  A sum of K products in fp32, however it is split over slices, waves and
launches, adds each product in at most K/4 + 64 rounded additions (a matrix
instruction's 32 products count as at most eight levels, then one addition a
slice, then at most 64 partial sums), so it is off by at most
(K/4 + 64) * 2^-24 * sum |products|.  A value that enters the next product as two
bf16 halves is off by 2^-16 of itself; a bf16 output by 2^-8 of itself, half a
unit in the last of its 8 significant bits.
"""
import numpy as np
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def gamma(k):
    return (k / 4 + 64) * 2.0 ** -24


def rand_fp4(gen, *shape, k):
    """Random packed codes [*shape, k/2] on the GPU."""
    return torch.randint(0, 256, (*shape, k // 2), dtype=torch.uint8, device="cuda", generator=gen)


def rand_sf(gen, rows, k, items=None, lo=0x20, hi=0x50):
    """Random swizzled scale bytes (codes lo..hi-1, about 2^-3..2^3) of `items`
    matrices; padding bytes hold the largest scale, which no result may show."""
    rp, cp = (rows + 127) // 128 * 128, (k // 16 + 3) // 4 * 4
    n = 1 if items is None else items
    sf = torch.full((n, rp * cp), 0x7E, dtype=torch.uint8, device="cuda")
    at = sf_index(rows, k).view(-1)
    sf[:, at] = torch.randint(lo, hi, (n, at.numel()), dtype=torch.uint8, device="cuda", generator=gen)
    return sf[0] if items is None else sf


def sf_index(rows, k):
    r = torch.arange(rows, device="cuda")[:, None]
    c = torch.arange(k // 16, device="cuda")[None]
    groups = (k // 16 + 3) // 4
    return ((r // 128) * groups + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4


def dequant(codes, sf):
    """[n, k/2] packed codes and their scale buffer -> float64 [n, k]."""
    n, k = codes.shape[0], codes.shape[1] * 2
    mag = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    v = torch.empty(n, k, dtype=torch.float64, device=codes.device)
    v[:, 0::2] = mag[(codes & 15).long()]
    v[:, 1::2] = mag[(codes >> 4).long()]
    return v * sf.view(torch.float8_e4m3fn)[sf_index(n, k)].double().repeat_interleave(16, 1)


def route(logits, k, score, renorm):
    """Per token the chosen experts in order and their weights, in float64."""
    ids, ws = [], []
    for row in logits.double().cpu().numpy():
        able = [j for j in range(len(row)) if not np.isnan(row[j]) and row[j] > -np.inf]
        best = sorted(able, key=lambda j: (-row[j], j))[:k]
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "softmax":
                top = max((row[j] for j in able), default=0.0)
                den = sum(np.exp(row[j] - top) for j in (best if renorm else able))
                w = [np.exp(row[j] - top) / den for j in best]
            else:
                # log of the sigmoid, so that very negative logits keep their ratios
                log = [min(row[j], 0.0) - np.log1p(np.exp(-abs(row[j]))) for j in best]
                top = max(log, default=0.0) if renorm else 0.0
                w = [np.exp(v - top) for v in log]
                w = [v / sum(w) for v in w] if renorm else w
        ids.append(best)
        ws.append(w)
    return ids, ws


def moe(x, logits, w13, w13_sf, a13, w2, w2_sf, a2, k, score, renorm):
    """(out, bound on |kernel - out|, ids [t, k], weights [t, k]), float64."""
    t, h = x.shape
    inter = w2.shape[2] * 2
    ids, ws = route(logits, k, score, renorm)
    out = torch.zeros(t, h, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(out)
    x64 = x.double()
    for e in sorted({e for row in ids for e in row}):
        rows = [i for i in range(t) if e in ids[i]]
        at = torch.tensor(rows, device="cuda")
        wt = torch.tensor([ws[i][ids[i].index(e)] for i in rows], dtype=torch.float64, device="cuda")[:, None]
        w = dequant(w13[e], w13_sf[e])
        al = a13[e].double()
        gu, sgu = x64[at] @ w.t() * al, x64[at].abs() @ w.abs().t() * al.abs()
        g, u = gu[:, :inter], gu[:, inter:]
        dg, du = gamma(h) * sgu[:, :inter], gamma(h) * sgu[:, inter:]
        silu = g * torch.sigmoid(g)
        act = silu * u
        # |silu'| <= 1.1; the two factors' errors, their product, the split and a
        # few fp32 roundings (exp, division, the products with the weights)
        da = 1.1 * dg * (u.abs() + du) + silu.abs() * du + act.abs() * (2.0 ** -16 + 2.0 ** -19)
        w = dequant(w2[e], w2_sf[e])
        s = a2[e].double() * wt
        out[at] += act @ w.t() * s
        err[at] += (da @ w.abs().t() + gamma(k * inter) * (act.abs() @ w.abs().t())) * s.abs()
    idm = torch.tensor([r + [-1] * (k - len(r)) for r in ids], dtype=torch.int32)
    wm = torch.tensor([list(r) + [0.0] * (k - len(r)) for r in ws], dtype=torch.float64)
    return out, err + out.abs() * 2.0 ** -8 * 1.01 + 1e-30, idm, wm


def adapters(base, base_abs, k, x, la, lb, ids, scaling, bias):
    """base = alpha * A @ W^T and its sum of magnitudes, in float64 -> (out, bound)."""
    out, err = base.clone(), gamma(k) * base_abs
    L, r = la.shape[0], la.shape[1]
    x64 = x.double()
    for a in sorted({int(v) for v in ids.tolist() if 0 <= v < L}):
        at = (ids == a).nonzero()[:, 0]
        s = 1.0 if scaling is None else scaling[a].double()
        A, B = la[a].double(), lb[a].double()
        d, sd = x64[at] @ A.t() * s, x64[at].abs() @ A.abs().t() * abs(s)
        out[at] += d @ B.t()
        # d's own sum and scaling, its split, and the second sum beside the base
        err[at] += ((gamma(k) + 2.0 ** -23) * sd + 2.0 ** -16 * d.abs()) @ B.abs().t() + gamma(k + r) * (
            d.abs() @ B.abs().t() + base_abs[at])
    if bias is not None:
        out = out + bias.double()
    return out, err + (out.abs() + (0 if bias is None else bias.double().abs())) * 2.0 ** -8 * 1.01 + 1e-30


def worst(got, ref, bound):
    """Largest |got - ref| / bound (inf where finiteness differs)."""
    got = got.double()
    same = torch.isnan(got) == torch.isnan(ref)
    assert bool(same.all()), "NaN in other places"
    fin = torch.isfinite(ref)
    assert bool((torch.isfinite(got) == fin).all()), "infinities in other places"
    return float(((got - ref).abs() / bound)[fin].max()) if bool(fin.any()) else 0.0
