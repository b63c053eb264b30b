"""Plain FP64 forms of the rotary positions and of the quantised paged cache,
for the tests (numpy and torch, nothing of the library)."""
from __future__ import annotations

import math

import numpy as np
import torch

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def frequencies(rot, base=10000.0, scaling=0, factor=1.0, trained=4096.0, fast=32.0, slow=1.0):
    """FP64 frequencies and the factor of the rotated channels."""
    j = np.arange(rot // 2, dtype=np.float64)
    if scaling == 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * j / rot)
    if scaling == 1:
        return f / factor, 1.0
    if scaling == 3:
        at = lambda turns: rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(at(fast))), min(rot - 1, math.ceil(at(slow)))
        ramp = np.clip((j - lo) / max(hi - lo, 1e-3), 0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rope(x, positions, inv_freq, mscale, half, rot, inverse=False):
    """x [B, N, H, D] (any type) -> FP64."""
    x = x.double()
    a = torch.as_tensor(positions).double().to(x.device)[..., None, None] * torch.as_tensor(inv_freq).to(x.device)
    c, s = a.cos() * mscale, a.sin() * (-mscale if inverse else mscale)
    y = x.clone()
    i0 = torch.arange(rot // 2) if half else torch.arange(0, rot, 2)
    i1 = i0 + (rot // 2 if half else 1)
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    return y


def quantise(x, dtype):
    """Rows of BF16 values -> (codes as FP64 values, FP32 scales), the quotient in FP64."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(x).all(-1, keepdim=True)
    top = TOP[dtype]
    q = torch.where((amax > 0) & ~bad, x * top / amax, torch.zeros_like(x))
    if dtype == torch.int8:
        code = q.round()
    else:
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        code = (q / step).round() * step
    scale = (amax / top).float().squeeze(-1)  # one rounding: the FP64 quotient is not half-way between FP32 values
    return code, torch.where(bad.squeeze(-1), torch.full_like(scale, math.nan), scale)


def rows(cache, table, b, slots):
    """Dequantised FP64 K and V [len(slots), H, D] of sequence b."""
    k, ks, v, vs = cache
    page_size = k.shape[2]
    page, off = table[b].long()[slots // page_size], slots % page_size
    return (k[page, :, off].double() * ks[page, :, off].double()[..., None],
            v[page, :, off].double() * vs[page, :, off].double()[..., None])


def seen(mask, b, t, T, n_draft):
    """Drafted tokens that row t of sequence b sees."""
    if mask is None:
        return list(range(min(t + 1, n_draft)))
    w = mask[b, t].tolist()
    return [j for j in range(n_draft) if (w[j // 32] >> (j % 32)) & 1]


def attention(q, cache, table, context, count, mask, scale=None):
    """FP64 (out, lse, bound) of the drafted rows; rows from count on are NaN.

    bound: how far the kernel may be from out.  Each probability times its V
    scale is rounded to FP16 (2^-11, or 2^-25 absolute of the largest, which
    is 1, where that is subnormal); a score is an FP32 sum of D products
    and two more roundings, off by at most (D + 4) 2^-24 sum |q k|, which moves
    a probability and the denominator by that (relative); exp2 and the other
    FP32 steps add 2^-19; the sums over n keys n 2^-24; the result is rounded
    to BF16, 2^-8.  lse moves by the score's error, and 2^-22 of
    itself and of the sum."""
    B, T, Hq, D = q.shape
    H = cache[0].shape[1]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    out = torch.full((B, T, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((B, T, Hq), math.nan, dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        n = int(context[b])
        cnt = T if count is None else int(count[b])
        k, v = rows(cache, table, b, torch.arange(n + cnt, device=q.device))
        for t in range(cnt):
            use = torch.tensor(list(range(n)) + [n + j for j in seen(mask, b, t, T, cnt)], dtype=torch.long,
                               device=q.device)
            for h in range(H):
                hq = slice(h * G, (h + 1) * G)
                if not len(use):
                    out[b, t, hq], lse[b, t, hq] = 0.0, -math.inf
                    continue
                kk, vv, qq = k[use, h], v[use, h], q[b, t, hq].double()
                s = qq @ kk.T * scale
                p = torch.softmax(s, -1)
                out[b, t, hq], lse[b, t, hq] = p @ vv, torch.logsumexp(s, -1)
                ds = ((qq.abs() @ kk.abs().T).amax(-1, keepdim=True) * scale) * (D + 4) * 2.0 ** -24
                spread = p @ vv.abs()
                sub = len(use) * 2.0 ** -25 * vv.abs().amax() * p.amax(-1, keepdim=True)
                tol[b, t, hq] = (spread * (2.0 ** -11 + 2 * ds + 2.0 ** -19 + len(use) * 2.0 ** -24) + sub +
                                 2.0 ** -8 * out[b, t, hq].abs())
                tol_lse[b, t, hq] = ds[:, 0] + 2.0 ** -22 * (lse[b, t, hq].abs() + 1) + len(use) * 2.0 ** -24
    return out, lse, tol, tol_lse


def tree_mask(parents, device):
    """int32 [B, T, words] of the parents [B][T] (-1: grows from the context)."""
    T = len(parents[0])
    words = [[[0] * (-(-T // 32)) for _ in range(T)] for _ in parents]
    for b, pb in enumerate(parents):
        for i, p in enumerate(pb):
            if p >= 0:
                words[b][i] = list(words[b][p])
            words[b][i][i // 32] |= 1 << (i % 32)
    m = torch.tensor(words, dtype=torch.int64)
    return torch.where(m >= 1 << 31, m - (1 << 32), m).to(torch.int32).to(device)
