"""Plain fp64 attention with modified softmax scores (tanh cap, distance
bias), forward and backward, for the tests of the CUDA path."""

from __future__ import annotations

import torch

import oracle


def visible(flags, window, Sq, Skv, B, q_seg=None, kv_seg=None, dense=None):
    """Boolean [B, Sq, Skv] visibility."""
    rows = []
    for b in range(B):
        rows.append(torch.from_numpy(oracle.visibility_matrix(
            flags, window, Sq, Skv,
            None if q_seg is None else q_seg[b],
            None if kv_seg is None else kv_seg[b], dense=dense)))
    return torch.stack(rows)


def logits(q, k, vis, scale, softcap, slopes):
    """fp64 logits [B, H, Sq, Skv] (-inf where masked) and the cap's
    derivative 1 - tanh^2 (or None), as 1 / cosh^2, which does not cancel
    where tanh saturates."""
    H, Hkv = q.shape[1], k.shape[1]
    ke = k.double().repeat_interleave(H // Hkv, 1)
    x = q.double() @ ke.transpose(2, 3) * scale
    t = None
    if softcap > 0:
        t = torch.cosh(x / softcap) ** -2
        x = softcap * torch.tanh(x / softcap)
    if slopes is not None:
        i, j = torch.arange(q.shape[2]), torch.arange(k.shape[2])
        dist = (i[:, None] - j[None, :]).abs().double()
        x = x - slopes.double().view(1, H, 1, 1) * dist
    return x.masked_fill(~vis[:, None], float("-inf")), t


def forward(q, k, v, vis, scale, softcap=0.0, slopes=None):
    """(out, lse, spread) in fp64; spread = sum_k p |v|, which bounds how
    far rounding p moves the output."""
    H, Hkv = q.shape[1], k.shape[1]
    x, _ = logits(q, k, vis, scale, softcap, slopes)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(torch.isfinite(lse), lse,
                                  torch.zeros_like(lse))[..., None])
    ve = v.double().repeat_interleave(H // Hkv, 1)
    return p @ ve, lse, p @ ve.abs()


def backward(q, k, v, do, vis, scale, softcap=0.0, slopes=None,
             bounds=False):
    """(dq, dk, dv) in fp64 from the formulas; with ``bounds`` also how far
    the kernels' roundings may move each element, (bq, bk, bv).

    Bounds, with h = 2^-8 (half a bf16 step) and e = 2^-11 for the f32 work
    (scores, exponentials, the logsumexp): P is off by (h + e) P where it
    multiplies dO and by e P elsewhere; the output that D_q = sum_d dO out is
    taken from by h (sum_k P |V| + |out|), so D_q by h sum_d |dO| (...); dS
    is rounded to bf16, h |dS|; every result to bf16, h |result|.  Sums over
    keys, queries and the heads of a group add the bounds up.
    """
    B, H, Sq, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    G = H // Hkv
    x, bend = logits(q, k, vis, scale, softcap, slopes)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(torch.isfinite(lse), lse,
                                  torch.zeros_like(lse))[..., None])
    ke = k.double().repeat_interleave(G, 1)
    ve = v.double().repeat_interleave(G, 1)
    do = do.double()

    def group(y):
        return y.view(B, Hkv, G, Skv, D).sum(2)

    dp = do @ ve.transpose(2, 3)
    row = (p * dp).sum(-1, keepdim=True)
    if bend is None:
        bend = torch.ones_like(p)
    ds = p * (dp - row) * bend * scale
    dq = ds @ ke
    dk = group(ds.transpose(2, 3) @ q.double())
    dv = group(p.transpose(2, 3) @ do)
    if not bounds:
        return dq, dk, dv
    h, e = 2.0 ** -8, 2.0 ** -11
    out, spread = p @ ve, p @ ve.abs()
    off = h * (do.abs() * (spread + out.abs())).sum(-1, keepdim=True)
    size = dp.abs() + row.abs()
    b = (h + e) * ds.abs() + p * bend * abs(scale) * (off + e * size)
    bq = b @ ke.abs()
    bk = group(b.transpose(2, 3) @ q.double().abs())
    bv = group((h + e) * p.transpose(2, 3) @ do.abs())
    return (dq, dk, dv), tuple(y + h * (y + g.abs()) for y, g in
                               zip((bq, bk, bv), (dq, dk, dv)))
