"""Plain fp64 form of attention of drafted tokens over the paged 8-bit cache,
from its definition, and trees for the tests of the CUDA path."""

from __future__ import annotations

import math

import torch


def random_tree(B, T, seed, empty=0.0):
    """Truth values [B, T, T]: each draft hangs on an earlier one or is a root
    of its own; some rows have no bit."""
    g = torch.Generator().manual_seed(seed)
    bits = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for t in range(T):
            parent = int(torch.randint(max(-1, t - 6), t, (1,), generator=g)) \
                if t else -1
            if parent >= 0:
                bits[b, t] = bits[b, parent]
            bits[b, t, t] = True
        gone = torch.rand(T, generator=g) < empty
        bits[b, gone] = False
    return bits


def pack(bits):
    """Truth values [..., T, T] -> int32 words [..., T, ceil(T / 32)]."""
    n = bits.shape[-1]
    words = (n + 31) // 32
    full = torch.zeros(*bits.shape[:-1], words * 32, dtype=torch.int64)
    full[..., :n] = bits.long()
    v = (full.view(*bits.shape[:-1], words, 32) << torch.arange(32)).sum(-1)
    return torch.where(v >= 2 ** 31, v - 2 ** 32, v).int()


def attention(q, k_pages, v_pages, k_scale, v_scale, table, lens, n_new, bits,
              scale, window=0, softcap=0.0, slopes=None):
    """(out, lse, spread) in fp64 for q [B, H, T, D] on the CPU; spread =
    sum p |v|.  bits None: a chain."""
    B, H, T, D = q.shape
    Hkv, P = k_pages.shape[1], k_pages.shape[2]
    out = torch.zeros(B, H, T, D, dtype=torch.float64)
    spread = torch.zeros_like(out)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64)
    for b in range(B):
        length, n = int(lens[b]), int(n_new[b])
        if n == 0:
            continue
        base = length - n
        ids = table[b, :(length + P - 1) // P].long()

        def tokens(pages, sc):
            x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn)
            x = x.float().double() * sc.double()[ids][:, :, None, None]
            return x.transpose(0, 1).reshape(Hkv, -1, D)[:, :length]

        k, v = tokens(k_pages, k_scale), tokens(v_pages, v_scale)
        mine = torch.ones(n, n, dtype=torch.bool).tril() if bits is None \
            else bits[b, :n, :n]
        depth = mine.sum(-1) - 1
        at = torch.cat([torch.arange(base), base + depth])
        pos = (base + depth)[:, None]
        vis = torch.cat([torch.ones(n, base, dtype=torch.bool), mine], 1)
        vis &= (depth >= 0)[:, None]
        if window > 0:
            vis &= pos - at < window
        for h in range(H):
            j = h // (H // Hkv)
            x = q[b, h, :n].double() @ k[j].T * scale
            if softcap > 0:
                x = softcap * torch.tanh(x / softcap)
            if slopes is not None:
                x = x - float(slopes[h]) * (pos - at).abs().double()
            x = x.masked_fill(~vis, -math.inf)
            l = torch.logsumexp(x, -1)
            w = torch.exp(x - torch.where(l == -math.inf, torch.zeros_like(l),
                                          l)[:, None])
            # a masked key contributes nothing, whatever its value holds
            for t in range(n):
                s = vis[t]
                out[b, h, t] = w[t, s] @ v[j][s]
                spread[b, h, t] = w[t, s] @ v[j][s].abs()
            lse[b, h, :n] = l
    return out, lse, spread
