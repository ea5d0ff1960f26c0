"""The cache operators in plain 64-bit torch, from their definitions, and the
error bounds that the kernels are held to. Shares no code with the CUDA path.

Bounds (u = 2^-24, half a step of fp32; a rounding to bf16 is off by at most
2^-8 relative). For one output row with weights p_j and A = sum_j p_j |v_j|:

* a logit is a sum of 128 products in fp32, then scaled: off by at most
  dx = (128 + 4) u * scale * sum_d |q_d k_d| in natural units (any order of
  the sum; 4 for the scale's own rounding, the product and the subtraction of
  the maximum);
* a weight is then off by a factor exp(2 dx) at most (numerator and
  denominator), plus 2^-21 for the exponential and its base-2 argument, plus
  the rounding of the sum: c u with c the longest chain of additions;
* products and sums of p v add another c u;
* the bf16 kernels round the weights to bf16 before the product with V
  (2^-8 A) and the result (2^-8 |o|); the fp32 ones round the result (u |o|).
"""
import math

import torch

U = 2.0 ** -24
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2


def seen_mask(n_q, n_k, length, window, sinks, device):
    p = (length - n_q + torch.arange(n_q, device=device))[:, None]
    j = torch.arange(n_k, device=device)[None]
    m = (j <= p) & (p >= 0)
    if window > 0:
        m &= (j < sinks) | (j > p - window)
    return m


def _head(q, k, v, mask, scale, bf16):
    """q [R, d], k/v [n, d], mask [R, n]: outputs, weights, output bounds, relative weight bounds [R]."""
    q, k, v = q.double(), k.double(), v.double()
    k = torch.where(mask.any(0)[:, None], k, torch.zeros_like(k))
    v = torch.where(mask.any(0)[:, None], v, torch.zeros_like(v))
    x = (q @ k.T) * scale
    x = torch.where(mask, x, torch.full_like(x, -math.inf))
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    tot = e.sum(1, keepdim=True)
    p = torch.where(tot > 0, e / torch.where(tot > 0, tot, torch.ones_like(tot)), torch.zeros_like(e))
    o, big = p @ v, p @ v.abs()
    dx = 132 * U * scale * torch.where(mask, q.abs() @ k.abs().T, torch.zeros_like(x)).amax(1)
    chain = 64 + 16 + 2 * (k.shape[0] / 64 + 1) + 128       # inside a tile, its lanes, over tiles, over splits
    rel = torch.expm1(2 * dx) + 2.0 ** -21 + 2 * chain * U
    bound = big * rel[:, None] + (BF16_HALF * (big + o.abs()) if bf16 else U * o.abs())
    return o, p, bound * 1.01, rel * 1.01


def attention(q, k, v, lens, window=0, sinks=0, scale=None, k_prefix=None, v_prefix=None):
    """[b, h, n_q, d] outputs and their bounds, [b, h_kv, n_k] added scores and their bounds."""
    b, hq, nq, d = q.shape
    hkv, nk = k.shape[1], k.shape[2]
    g = hq // hkv
    bf16 = q.dtype == torch.bfloat16
    scale = scale if scale else 1 / math.sqrt(d)
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    add = torch.zeros(b, hkv, nk, dtype=torch.float64, device=q.device)
    add_tol = torch.zeros_like(add)
    for s in range(b):
        mask = seen_mask(nq, nk, int(lens[s]), window, sinks, q.device)
        for kh in range(hkv):
            kk, vv, mm = k[s, kh], v[s, kh], mask
            if k_prefix is not None:
                kk, vv = torch.cat([k_prefix[kh], kk]), torch.cat([v_prefix[kh], vv])
                mm = torch.cat([torch.ones(nq, k_prefix.shape[1], dtype=torch.bool, device=q.device), mm], 1)
            for h in range(kh * g, (kh + 1) * g):
                o, p, t, rel = _head(q[s, h], kk, vv, mm, scale, bf16)
                out[s, h], tol[s, h] = o, t
                if k_prefix is None:
                    add[s, kh] += p.sum(0)
                    add_tol[s, kh] += (p * (rel + 300 * U)[:, None]).sum(0)   # up to 256 rows added in fp32
    return out, tol, add, add_tol


def evict(score, lens, sinks, recent, budget):
    """Per sequence and head the kept indices (lists, ascending)."""
    b, hkv, _ = score.shape
    kept = []
    for s in range(b):
        n = int(lens[s])
        kept.append([])
        for h in range(hkv):
            if n <= budget:
                kept[-1].append(list(range(n)))
                continue
            row = [float(x) for x in score[s, h, :n].cpu()]
            row = [-math.inf if math.isnan(x) else x for x in row]
            nan = [math.isnan(float(x)) for x in score[s, h, :n].cpu()]
            free = range(sinks, n - recent)
            best = sorted(free, key=lambda j: (nan[j], -row[j], j))[:budget - sinks - recent]
            kept[-1].append(sorted(list(range(sinks)) + best + list(range(n - recent, n))))
    return kept
