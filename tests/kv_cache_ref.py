"""Plain fp64 forms of the paged 8-bit cache's operators, from their
definitions, for the tests of the CUDA path."""

from __future__ import annotations

import math

import numpy as np
import torch


def e4m3(x):
    """x (fp64) rounded to the nearest e4m3 value, ties to even, saturating
    at 448; NaN stays NaN."""
    x = np.clip(x, -448.0, 448.0)
    _, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)  # 3 mantissa bits, min 2^-9
    return np.rint(x / step) * step


def decode(codes):
    """fp64 values of float8_e4m3fn codes."""
    return codes.float().double().numpy()


def block_scale(x):
    """2^e, e the smallest integer in [-40, 40] with max |finite x| <=
    448 * 2^e."""
    a = np.abs(x[np.isfinite(x)])
    a = float(a.max()) if a.size else 0.0
    for e in range(-40, 40):
        if a <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 40


def append(pages, scales, table, lens, new, n_new):
    """Appends new [B, H_kv, T, D] (bf16) to fp64 copies of the pages' code
    values [n, H_kv, P, D] and scales [n, H_kv]; returns both."""
    pages, scales = decode(pages).copy(), scales.double().numpy().copy()
    P = pages.shape[2]
    for b in range(len(lens)):
        at, end = int(lens[b]), int(lens[b]) + int(n_new[b])
        while at < end:
            pid, lo = int(table[b, at // P]), at % P
            hi = min(P, lo + end - at)
            for h in range(pages.shape[1]):
                first = at - int(lens[b])
                x = new[b, h, first:first + hi - lo].double().numpy()
                s = block_scale(x)
                if lo > 0:
                    s = max(s, scales[pid, h])
                    if s > scales[pid, h]:
                        pages[pid, h, :lo] = e4m3(pages[pid, h, :lo]
                                                  * (scales[pid, h] / s))
                pages[pid, h, lo:hi] = e4m3(x / s)
                scales[pid, h] = s
            at += hi - lo
    return pages, scales


def attention(q, k_pages, v_pages, k_scale, v_scale, table, lens, scale,
              window=0, softcap=0.0, slopes=None):
    """(out, lse, spread) in fp64 for q [B, H, T, D] on the CPU; spread =
    sum p |v|."""
    B, H, T, D = q.shape
    Hkv, P = k_pages.shape[1], k_pages.shape[2]
    out = torch.zeros(B, H, T, D, dtype=torch.float64)
    spread = torch.zeros_like(out)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        ids = table[b, :(n + P - 1) // P].long()

        def tokens(pages, sc):
            x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn)
            x = x.float().double() * sc.double()[ids][:, :, None, None]
            return x.transpose(0, 1).reshape(Hkv, -1, D)[:, :n]

        k, v = tokens(k_pages, k_scale), tokens(v_pages, v_scale)
        pos = torch.arange(n - T, n)[:, None]
        key = torch.arange(n)[None, :]
        vis = key <= pos
        if window > 0:
            vis &= pos - key < window
        for h in range(H):
            j = h // (H // Hkv)
            x = q[b, h].double() @ k[j].T * scale
            if softcap > 0:
                x = softcap * torch.tanh(x / softcap)
            if slopes is not None:
                x = x - float(slopes[h]) * (pos - key).abs().double()
            x = x.masked_fill(~vis, -math.inf)
            l = torch.logsumexp(x, -1)
            w = torch.exp(x - torch.where(torch.isfinite(l), l,
                                          torch.zeros_like(l))[:, None])
            # a masked key contributes nothing, whatever its value holds
            for t in range(T):
                s = vis[t]
                out[b, h, t] = w[t, s] @ v[j][s]
                spread[b, h, t] = w[t, s] @ v[j][s].abs()
            lse[b, h] = l
    return out, lse, spread


def random_cache(num_pages, Hkv, P, D, seed, spread=3, centre=-7):
    """Random codes and power-of-two scales on the CPU: (k, v, ks, vs)."""
    g = torch.Generator().manual_seed(seed)
    res = []
    for _ in range(2):
        x = torch.randn(num_pages, Hkv, P, D, generator=g) * 110.0
        res.append(x.clamp(-448, 448).to(torch.float8_e4m3fn))
    for _ in range(2):
        e = torch.randint(centre - spread, centre + spread + 1,
                          (num_pages, Hkv), generator=g)
        res.append(torch.exp2(e.float()))
    return res


def random_table(lens, P, width, num_pages, seed):
    """Pages of each sequence, scattered; -1 past its last."""
    perm = torch.randperm(num_pages,
                          generator=torch.Generator().manual_seed(seed))
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        m = (int(n) + P - 1) // P
        table[b, :m] = perm[at:at + m].int()
        at += m
    assert at <= num_pages
    return table
