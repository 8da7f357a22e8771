"""64-bit restatements of the 4-bit products, the routing and the experts' blocks, with the bounds
their kernels are held to."""
import math

import numpy as np
import torch


def matrices(g, count, n, k, group, zeros, device="cuda"):
    """count matrices [n][k]: codes, fp16 scales, zeros or None; padding of scales is NaN, of zeros 255."""
    S, used = (k // group + 7) // 8 * 8, k // group
    codes = torch.randint(0, 256, (count, n, k // 2), generator=g, device=device, dtype=torch.uint8)
    scales = (0.5 + torch.rand(count, n, S, generator=g, device=device)) / (4.6 * math.sqrt(k))
    scales[..., used:] = math.nan
    z = None
    if zeros:
        z = torch.randint(0, 16, (count, n, S), generator=g, device=device, dtype=torch.uint8)
        z[..., used:] = 255
    return codes, scales.half(), z


def weights(codes, scales, zeros, k, group):
    """fp64 weights [..., n, k]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    per = torch.arange(k, device=codes.device) // group
    z = 8.0 if zeros is None else zeros.double()[..., per]
    return (c - z) * scales.double()[..., per]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def product(x, w, dtype, tokens=None):
    """(exact y, bound of an output's error).  For up to eight tokens c - z is exact, x too (fp32: to 22
    bits), and what is left is binary32 addition, cut on the tensor cores: per group 8 steps (16 with two parts)
    that lose below 2^-22 of its magnitudes each, then at most 1024 groups in up to eight chains, 2^-24 each
    of all of it: below 1e-5 of the sum of magnitudes.  More bf16 tokens: weights rounded to 11 bits,
    2^-11 of the magnitudes; fp32: as few tokens.  A row of x is scaled so that its
    largest value lies below 2^15, and fp16's last place is 2^-24 (half of it is lost): 2^-39 of that value."""
    xd = x.double()
    y, mag = xd @ w.t(), xd.abs() @ w.abs().t()
    many = (x.shape[0] if tokens is None else tokens) > 8
    rel = 2.0 ** -11 if dtype == torch.bfloat16 and many else 1e-5
    lost = 2.0 ** -39 * xd.abs().amax(1, keepdim=True) * w.abs().sum(1)
    return y, rel * mag + lost + half_step(dtype) * y.abs() + 1e-30


def experts(x, up, down, group, ids, wts, dtype):
    """(exact y, bound).  The bound of a block: gate and up rows as a product's, silu's slope is below
    1.1, h in at least 16 bits, the down rows as a product's, and the output's rounding."""
    T, H = x.shape
    F = up[0].shape[1] // 2
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    off = torch.zeros_like(y)
    rel = 2.0 ** -11 if dtype == torch.bfloat16 else 1e-5
    for e in range(up[0].shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        wu = weights(*(None if m is None else m[e] for m in up), H, group)
        wd = weights(*(None if m is None else m[e] for m in down), F, group)
        xe = x[t].double()
        both = xe @ wu.t()
        mag = xe.abs() @ wu.abs().t() + 2.0 ** -39 / rel * xe.abs().amax(1, keepdim=True) * wu.abs().sum(1)
        g, u, dg, du = both[:, :F], both[:, F:], rel * mag[:, :F], rel * mag[:, F:]
        s = g * torch.sigmoid(g)
        h = s * u
        dh = 1.1 * dg * (u.abs() + du) + s.abs() * du + 2.0 ** -(11 if dtype == torch.bfloat16 else 22) * h.abs()
        dh = dh + 2.0 ** -39 * h.abs().amax(1, keepdim=True)
        w = wts[t, j].double()[:, None]
        y.index_add_(0, t, w * (h @ wd.t()))
        off.index_add_(0, t, w.abs() * (dh @ wd.abs().t() + rel * (h.abs() + dh) @ wd.abs().t()))
    return y, off + half_step(dtype) * (y.abs() + off) + 1e-30


def route(x, k, sigmoid, bias=None, groups=1, keep=1, best=1, renormalize=True, scale=1.0, live=None):
    """ids, weights (fp64), expert_start and order from logits [T][E] (numpy, any float type)."""
    T, E = x.shape
    ids = np.full((T, k), -1, np.int64)
    wts = np.zeros((T, k))
    big = float(np.finfo(np.float32).max)
    for t in range(T if live is None else min(max(live, 0), T)):
        v = np.minimum(x[t].astype(np.float64), big)
        b = np.zeros(E) if bias is None else bias.astype(np.float64)
        can = (v > -np.inf) & (b > -np.inf)
        if not can.any():
            continue
        m = v[can].max()
        with np.errstate(over="ignore", invalid="ignore"):
            s = 1 / (1 + np.exp(-v)) if sigmoid else np.exp(v - m)
        if not sigmoid:
            s = s / s[can].sum()
        key = v if bias is None and best == 1 else s + b
        n = E // groups
        if groups > 1:
            value = []
            for i in range(groups):
                part = sorted((key[e] for e in range(i * n, i * n + n) if can[e]), reverse=True)
                value.append(sum(part[:best]) if part else -np.inf)
            order = sorted((i for i in range(groups) if value[i] > -np.inf), key=lambda i: (-value[i], i))[:keep]
            can = can & np.isin(np.arange(E) // n, order)
        chosen = sorted((e for e in range(E) if can[e]), key=lambda e: (-key[e], e))[:k]
        ids[t, :len(chosen)] = chosen
        if renormalize:   # with the largest chosen logit's power of e taken out
            c = v[chosen]
            low = min(c.max(), 0.0) if sigmoid else c.max()
            with np.errstate(over="ignore", invalid="ignore"):
                s = np.where(c < 0, np.exp(c - low) / (1 + np.exp(c)), 1 / (1 + np.exp(-c))) if sigmoid else np.exp(c - low)
            wts[t, :len(chosen)] = scale * s / s.sum()
        else:
            wts[t, :len(chosen)] = scale * s[chosen]
    flat = ids.flatten()
    pairs = np.array(sorted((i for i in range(T * k) if flat[i] >= 0), key=lambda i: (flat[i], i)), np.int64)
    order = np.full(T * k, -1, np.int64)
    order[:len(pairs)] = pairs
    start = np.array([(flat[flat >= 0] < e).sum() for e in range(E + 1)])
    return ids, wts, start, order
