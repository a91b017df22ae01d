"""Plain 64-bit implementations of the rotated append, the 8-bit append and the 8-bit attention
(CPU, loops over sequences and pages), and the inputs their tests share."""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3_MAX = 448.0
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}


def cu(lengths):
    c = np.zeros(len(lengths) + 1, dtype=np.int32)
    c[1:] = np.cumsum(lengths)
    return torch.from_numpy(c)


def block_table(sk, P, seed, spare=3, extra_cols=1):
    """(table int32 with -1 past each sequence's pages, number of blocks): shuffled blocks."""
    pages = [(s + P - 1) // P for s in sk]
    nb = sum(pages) + spare
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    bt = torch.full((len(sk), max(pages, default=0) + extra_cols), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt, nb


def tables(max_pos, rot, base=10000.0):
    inv = base ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


def rotate(x, pos, cos, sin, interleaved):
    """(rotated x, sum |products| of each output) of x (tokens, heads, D) in float64."""
    rot = 2 * cos.shape[1]
    y, mag = x.double().clone(), x.double().abs()
    c, s = cos[pos].double()[:, None], sin[pos].double()[:, None]
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia], mag[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, mag


def positions(n, sk):
    return torch.cat([torch.arange(m - k, m) for k, m in zip(n, sk)] + [torch.zeros(0, dtype=torch.long)])


def pow2_scale(absmax):
    """float: the least 2^k, k >= -100, with absmax <= 448 2^k."""
    if absmax <= 0:
        return 2.0 ** -100
    f, e = math.frexp(absmax)
    return 2.0 ** max(-100, e - 9 if f <= 0.875 else e - 8)


def e4m3(x):
    """float64 -> the nearest e4m3 value (ties to even; at most 448 in magnitude), by arithmetic."""
    a = x.abs()
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 1).clamp_min(-6) - 3)
    return torch.sign(x) * torch.round(a / step) * step  # torch.round: ties to even


def append_q8(x, mag, n, sk, bt, codes, scale):
    """Tokens x (total, Hkv, D) float64 into (codes float64 values, scale float64) in place.
    Returns a float64 tensor like ``codes``: how far a value (code x scale) may be off, 0 for slots
    whose code must be exact: half a step of e4m3 at the value, plus the fp32 arithmetic of the
    rotation (three roundings of 2^-24 of the products' magnitudes ``mag``)."""
    P = codes.shape[1]
    slack = torch.zeros_like(codes)
    at = 0
    for b, (k, m) in enumerate(zip(n, sk)):
        for p in range((m - k) // P, (m - 1) // P + 1) if k else ():
            lo, hi, blk = max(m - k, p * P), min(m, p * P + P), int(bt[b, p])
            t = slice(at + lo - (m - k), at + hi - (m - k))
            for h in range(codes.shape[2]):
                v = x[t, h]
                fin = v[torch.isfinite(v)]
                want = pow2_scale(float(fin.abs().max()) if fin.numel() else 0.0)
                if lo > p * P:
                    now = max(float(scale[blk, h]), want)
                    codes[blk, :lo - p * P, h] = e4m3(codes[blk, :lo - p * P, h] * (float(scale[blk, h]) / now))
                else:
                    now = want
                scale[blk, h] = now
                s = slice(lo - p * P, hi - p * P)
                codes[blk, s, h] = torch.where(torch.isfinite(v), e4m3(v / now), torch.nan)
                half = torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, now * 2.0 ** -10))
                slack[blk, s, h] = torch.nan_to_num(half) + 3 * 2.0 ** -24 * torch.nan_to_num(mag[t, h])
        at += k
    return slack


def attention(q, k, v, cu_q, cu_k, bt, scale, wl=-1, wr=-1, slopes=None):
    """Attention in float64 over paged k, v (float64 values (blocks, P, Hkv, D)).  Rows without
    a key: 0 and -inf.  Returns (out (total_q, H, D), lse (H, total_q))."""
    q = q.double()
    H, Hkv, D, P = q.shape[1], k.shape[2], q.shape[2], k.shape[1]
    out = torch.zeros_like(q)
    lse = torch.full((H, q.shape[0]), -math.inf, dtype=torch.float64)
    for b in range(len(cu_q) - 1):
        q0, q1 = int(cu_q[b]), int(cu_q[b + 1])
        n, m = q1 - q0, int(cu_k[b + 1] - cu_k[b])
        if n == 0 or m == 0:
            continue
        used = bt[b, :(m + P - 1) // P].long()
        i = torch.arange(n)[:, None] + (m - n)
        j = torch.arange(m)[None, :]
        ok = torch.ones((n, m), dtype=torch.bool)
        if wl >= 0:
            ok &= j >= i - wl
        if wr >= 0:
            ok &= j <= i + wr
        for h in range(H):
            kk = k[used, :, h * Hkv // H].reshape(-1, D)[:m]
            vv = v[used, :, h * Hkv // H].reshape(-1, D)[:m]
            z = q[q0:q1, h] @ torch.where(ok.any(0)[:, None], kk, torch.zeros_like(kk)).T * scale
            if slopes is not None:
                z = z - float(slopes[h]) * (j - i).abs()
            z = z.masked_fill(~ok, -math.inf)
            l = torch.logsumexp(z, dim=1)
            lse[h, q0:q1] = l
            w = torch.exp(z - torch.where(l == -math.inf, torch.zeros_like(l), l)[:, None])
            out[q0:q1, h] = w @ torch.where(ok.any(0)[:, None], vv, torch.zeros_like(vv))
    return out, lse


def random_pool(nb, P, Hkv, D, seed, kind="pow2", std=1.0):
    """(codes e4m3, scale f32) of N(0, std^2) values.  ``kind``: scales by powers of two, by
    absmax / 448, or "wide" (absmax / 448 of pages whose magnitudes span 2^+-12)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((nb, P, Hkv, D), generator=g) * std
    if kind == "wide":
        x *= torch.exp2(torch.randint(-12, 13, (nb, 1, Hkv, 1), generator=g).float())
    top = x.abs().amax(dim=(1, 3))
    s = top / E4M3_MAX
    if kind == "pow2":
        s = torch.tensor([pow2_scale(float(t)) for t in top.reshape(-1)]).reshape(top.shape).float()
    return (x / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s.float()


def values(codes, scale):
    """The float64 values of an 8-bit pool."""
    return codes.float().double() * scale.double()[:, None, :, None]
