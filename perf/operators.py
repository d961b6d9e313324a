"""Cases of the attention operators with modified scores and of the 8-bit
paged key/value cache: their inputs, a plain form in elementary torch
operations, the framework's calls, and their definition in 64 bits.

Scores: x = scale q.k, capped to c tanh(x / c) where a cap c is given, then
lowered by slope_h |q - k| where slopes are given; softmax over the visible
keys.  Cache: pages of `page` tokens per key/value head in e4m3 with one
power-of-two scale per (page, head).
"""

import math

import torch

own = False

# ------------------------------------------------------------------- cases


def listed():
    return [
        # one short prompt of a small model: launch and host latency
        dict(name="prefill_short", op="forward", B=1, H=8, Hkv=8, S=256, D=64,
             mask="causal", window=0, softcap=30.0, alibi=False),
        # packed documents, capped scores: the batch of a training or
        # prompt step
        dict(name="prefill_packed", op="forward", B=2, H=16, Hkv=16, S=8192,
             D=128, mask="packed", window=0, softcap=50.0, alibi=False),
        # one long prompt, grouped heads, a bias that falls with distance
        dict(name="prefill_alibi", op="forward", B=1, H=32, Hkv=8, S=8192,
             D=128, mask="causal", window=0, softcap=0.0, alibi=True),
        # sliding window, odd length, both modifications at once
        dict(name="prefill_window", op="forward", B=1, H=12, Hkv=4, S=2999,
             D=128, mask="local", window=1000, softcap=30.0, alibi=True),
        # forward and backward of a short ragged batch row
        dict(name="train_short", op="training", B=1, H=4, Hkv=2, S=300, D=64,
             mask="causal", window=0, softcap=50.0, alibi=True),
        # forward and backward of an ordinary training batch, capped
        dict(name="train_capped", op="training", B=4, H=16, Hkv=16, S=2048,
             D=128, mask="causal", window=0, softcap=50.0, alibi=False),
        # forward and backward over packed documents, grouped heads, biased
        dict(name="train_packed", op="training", B=1, H=32, Hkv=8, S=4096,
             D=128, mask="packed", window=0, softcap=0.0, alibi=True),
        # the keys and values of a batch of prompts go into the cache
        dict(name="append_prompts", op="append", B=8, Hkv=8, D=128, page=64,
             T=2048, new_lo=500, len_lo=0, len_hi=0),
        # one new token for each sequence being served
        dict(name="append_step", op="append", B=64, Hkv=8, D=128, page=64,
             T=1, new_lo=1, len_lo=100, len_hi=1000),
        # one sequence, one new token: latency
        dict(name="decode_one", op="decode", B=1, H=32, Hkv=8, D=128, page=64,
             T=1, len_lo=2000, len_hi=2000, window=0, softcap=50.0,
             alibi=False),
        # a serving batch of unequal lengths
        dict(name="decode_batch", op="decode", B=64, H=32, Hkv=8, D=128,
             page=64, T=1, len_lo=300, len_hi=12000, window=0, softcap=0.0,
             alibi=True),
        # few very long sequences: the cache's bytes are the whole cost
        dict(name="decode_long", op="decode", B=4, H=32, Hkv=8, D=128,
             page=128, T=1, len_lo=100000, len_hi=131072, window=0,
             softcap=50.0, alibi=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "training", "append", "decode"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 6, 8])
    softcap, alibi = rng.choice([(30.0, False), (50.0, False), (0.0, True),
                                 (20.0, True)])
    if op in ("forward", "training"):
        top = 8192 if op == "forward" else 4096
        S = _log(rng, 200, top)
        if rng.random() < 0.5:
            S = max(256, S // 128 * 128)
        G = min(G, max(1, 32 // Hkv))
        B = rng.choice([1, 1, 2, 3]) if S <= 2048 else 1
        mask = rng.choice(["causal", "packed", "local", "full"])
        window = _log(rng, 30, S) if mask == "local" else 0
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, S=S, D=D, mask=mask,
                    window=window, softcap=softcap, alibi=alibi)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        step = rng.random() < 0.5
        T = rng.choice([1, 1, 2, 4]) if step else _log(rng, 20, 2000)
        B = _log(rng, 1, 128) if step else rng.choice([1, 2, 5, 8])
        len_hi = _log(rng, 50, 4000)
        return dict(op=op, B=B, Hkv=Hkv, D=D, page=page, T=T,
                    new_lo=max(1, T // 3), len_lo=rng.choice([0, len_hi // 5]),
                    len_hi=len_hi)
    B = _log(rng, 1, 64)
    len_hi = _log(rng, 200, 400000 // max(B, 4))
    T = rng.choice([1, 1, 1, 2, 4])
    window = rng.choice([0, 0, 0, _log(rng, 50, 4000)])
    return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, D=D, page=page, T=T,
                len_lo=max(T, len_hi // rng.choice([1, 4, 30])),
                len_hi=max(T, len_hi), window=window, softcap=softcap,
                alibi=alibi)


# ------------------------------------------------------------------ inputs


def _segments(case, seed):
    """Ids 0, 1, 2, ... of packed documents, [B, S] int32 on the host."""
    g = torch.Generator().manual_seed(seed * 7 + 5)
    B, S = case["B"], case["S"]
    lo, hi = max(1, S // 32), max(2, S // 4)
    seg = torch.empty(B, S, dtype=torch.int32)
    for b in range(B):
        n = torch.randint(lo, hi + 1, (S // lo + 1,), generator=g)
        ids = torch.repeat_interleave(torch.arange(n.numel()), n)
        seg[b] = ids[:S].int()
    return seg


def _slopes(H):
    """Geometric slopes, 2^(-8 (h + 1) / H): the steepest head looks a few
    tokens back, the flattest a few hundred."""
    h = torch.arange(1, H + 1, dtype=torch.float64)
    return torch.exp2(-8.0 * h / H).float()


def _ints(lo, hi, n, seed):
    g = torch.Generator().manual_seed(seed * 11 + 3)
    return torch.randint(lo, hi + 1, (n,), generator=g).int()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    st = dict(case=case)
    if case["op"] in ("forward", "training"):
        B, H, Hkv, S, D = (case[n] for n in ("B", "H", "Hkv", "S", "D"))
        # queries of spread magnitude, so that capped scores reach the cap's
        # bend in some rows
        row = torch.rand(B, H, S, 1, generator=g, device=dev) * 3.5 + 0.5
        st["q"] = (torch.randn(B, H, S, D, generator=g, device=dev)
                   * row).bfloat16()
        st["k"] = torch.randn(B, Hkv, S, D, generator=g, device=dev).bfloat16()
        st["v"] = torch.randn(B, Hkv, S, D, generator=g, device=dev).bfloat16()
        if case["op"] == "training":
            st["dout"] = torch.randn(B, H, S, D, generator=g,
                                     device=dev).bfloat16()
        st["seg"] = (_segments(case, seed).to(dev)
                     if case["mask"] == "packed" else None)
        st["slopes"] = _slopes(H).to(dev) if case["alibi"] else None
        return st
    B, Hkv, D, P, T = (case[n] for n in ("B", "Hkv", "D", "page", "T"))
    lens = _ints(case["len_lo"], case["len_hi"], B, seed)
    new = (_ints(case["new_lo"], T, B, seed + 1) if case["op"] == "append"
           else torch.zeros(B, dtype=torch.int32))
    pages = (lens + new + P - 1) // P
    width = int((int(case["len_hi"]) + T + P - 1) // P)
    total = int(pages.sum()) if case["op"] == "decode" else B * width
    # the sequences' pages lie scattered in the pool, as after some serving
    perm = torch.randperm(total + 3, generator=torch.Generator().manual_seed(
        seed + 17)).int()
    table = torch.full((B, width), -1, dtype=torch.int32)
    first = torch.cumsum(pages, 0) - pages
    slot = torch.arange(width).expand(B, width)
    used = slot < pages[:, None]
    table[used] = perm[(first[:, None] + slot)[used].long()]
    st["table"], st["lens"] = table.to(dev), lens.to(dev)
    shape = (total + 3, Hkv, P, D)
    for n in ("k", "v"):
        codes = torch.randn(shape, generator=g, device=dev) * 110.0
        st[n + "_pages"] = codes.clamp_(-448, 448).to(torch.float8_e4m3fn)
        st[n + "_scale"] = torch.exp2(torch.randint(
            -8, -5, shape[:2], generator=g, device=dev).float())
        del codes
    if case["op"] == "append":
        st["n_new"] = new.to(dev)
        for n in ("k_new", "v_new"):  # as a projection leaves them
            x = torch.randn(B, T, Hkv, D, generator=g, device=dev)
            st[n] = x.bfloat16().transpose(1, 2)
        return st
    H = case["H"]
    q = torch.randn(B, T, H, D, generator=g, device=dev) * 1.5
    st["q"] = q.bfloat16().transpose(1, 2)
    st["slopes"] = _slopes(H).to(dev) if case["alibi"] else None
    return st


# --------------------------------------------------------------- plain form


def _visible(case, seg, dev):
    """[B or 1, 1, 1, S, S] truth values."""
    S = case["S"]
    q = torch.arange(S, device=dev)[:, None]
    k = torch.arange(S, device=dev)[None, :]
    vis = torch.ones(S, S, dtype=torch.bool, device=dev)
    if case["mask"] != "full":
        vis = k <= q
    if case["mask"] == "local":
        vis = vis & (q - k < case["window"])
    vis = vis[None]
    if seg is not None:
        vis = vis & (seg[:, :, None] == seg[:, None, :])
    return vis[:, None, None]


def _modified(x, case, slopes, dist):
    """(logits, tanh or None) of the scaled scores x [B, Hkv, G, Tq, Tk]."""
    t = None
    if case["softcap"] > 0:
        t = torch.tanh(x / case["softcap"])
        x = t * case["softcap"]
    if slopes is not None:
        s = slopes.view(1, x.shape[1], x.shape[2], 1, 1)
        x = x - s * dist
    return x, t


def _softmax(z, vis):
    """(p, lse) over the visible keys; a row that sees none has p = 0 and
    lse = -inf."""
    z = z.masked_fill(~vis, -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(z - m)
    n = e.sum(-1, keepdim=True)
    lse = (m + torch.log(n)).squeeze(-1)
    return e / torch.where(n > 0, n, torch.ones_like(n)), lse


def _plain_attention(st):
    case = st["case"]
    B, H, Hkv, S, D = (case[n] for n in ("B", "H", "Hkv", "S", "D"))
    G, scale = H // Hkv, 1.0 / math.sqrt(D)
    q = st["q"].float().view(B, Hkv, G * S, D)
    k, v = st["k"].float(), st["v"].float()
    i = torch.arange(S, device=q.device)
    dist = (i[:, None] - i[None, :]).abs().float()
    vis = _visible(case, st["seg"], q.device)
    x = (q @ k.transpose(2, 3) * scale).view(B, Hkv, G, S, S)
    z, t = _modified(x, case, st["slopes"], dist)
    p, lse = _softmax(z, vis)
    p = p.view(B, Hkv, G * S, S)
    out = (p @ v).view(B, H, S, D)
    res = dict(out=out.bfloat16(), lse=lse.reshape(B, H, S))
    if case["op"] == "forward":
        return res
    do = st["dout"].float().view(B, Hkv, G * S, D)
    dp = do @ v.transpose(2, 3)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    if t is not None:
        ds = ds * (1 - t.view(ds.shape) ** 2)
    ds = ds * scale
    res["dq"] = (ds @ k).view(B, H, S, D).bfloat16()
    res["dk"] = (ds.transpose(2, 3) @ q).bfloat16()
    res["dv"] = (p.transpose(2, 3) @ do).bfloat16()
    return res


def _exponent(amax):
    """The smallest e in [-40, 40] with amax <= 448 * 2^e."""
    m, x = torch.frexp(amax)  # amax = m 2^x, m in [0.5, 1); 448 = 0.875 2^9
    e = x - 9 + (m > 0.875).int()
    return torch.where(amax > 0, e, torch.full_like(e, -40)).clamp(-40, 40)


def _codes(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _put(pages, scales, x, pid, live, at, old, new):
    """Writes the tokens of x [B, Hkv, T, D] that `new` marks into the pages
    pid (one per live slot), re-rounding the old tokens of a page whose scale
    grows."""
    B, slots, P = new.shape
    x = x.float().gather(2, at.expand(B, x.shape[1], -1, x.shape[3]))
    x = x.view(B, x.shape[1], slots, P, -1).transpose(1, 2)[live]
    old, new = old[live][:, None, :, None], new[live][:, None, :, None]
    size = torch.where(new & torch.isfinite(x), x.abs(), torch.zeros_like(x))
    want = torch.exp2(_exponent(size.amax((2, 3))).float())
    was, raw = scales[pid], pages[pid]
    scale = torch.where(old.any(2)[:, :, 0], torch.maximum(was, want), want)
    again = _codes(raw.view(torch.float8_e4m3fn).float()
                   * (was / scale)[:, :, None, None]).view(torch.uint8)
    again = torch.where((scale > was)[:, :, None, None], again, raw)
    fresh = _codes(x / scale[:, :, None, None]).view(torch.uint8)
    pages[pid] = torch.where(new, fresh, torch.where(old, again, raw))
    scales[pid] = scale


def _plain_append(st):
    case = st["case"]
    B, P, T = (case[n] for n in ("B", "page", "T"))
    table, lens, n_new = st["table"], st["lens"].long(), st["n_new"].long()
    slots = (T + P - 2) // P + 1  # pages that T tokens can touch
    page = lens[:, None] // P + torch.arange(slots, device=lens.device)
    tok = page[:, :, None] * P + torch.arange(P, device=lens.device)
    old = tok < lens[:, None, None]
    new = ~old & (tok < (lens + n_new)[:, None, None])
    live = new.any(-1)  # [B, slots]
    pid = table.gather(1, page.clamp(max=table.shape[1] - 1))[live].long()
    at = (tok - lens[:, None, None]).clamp(0, T - 1).view(B, 1, -1, 1)
    _put(st["k_pages"].view(torch.uint8), st["k_scale"], st["k_new"], pid,
         live, at, old, new)
    _put(st["v_pages"].view(torch.uint8), st["v_scale"], st["v_new"], pid,
         live, at, old, new)
    return _cache_state(st)


def _cache_state(st):
    return {n: st[n] for n in ("k_pages", "k_scale", "v_pages", "v_scale")}


def _plain_decode(st):
    case = st["case"]
    B, H, Hkv, D, P, T = (case[n] for n in ("B", "H", "Hkv", "D", "page", "T"))
    G, scale = H // Hkv, 1.0 / math.sqrt(D)
    idx = st["table"].clamp(min=0).long()

    def tokens(name):
        x = st[name + "_pages"].view(torch.uint8)[idx].view(
            torch.float8_e4m3fn).float()
        x = x * st[name + "_scale"][idx][:, :, :, None, None]
        return x.transpose(1, 2).reshape(B, Hkv, -1, D)

    k, v = tokens("k"), tokens("v")
    pos = (st["lens"].long()[:, None] - T
           + torch.arange(T, device=idx.device))[:, None, None, :, None]
    key = torch.arange(k.shape[2], device=idx.device)
    vis = key <= pos
    if case["window"] > 0:
        vis = vis & (pos - key < case["window"])
    # what lies behind a sequence's last token is never read
    seen = vis.any(3)[:, 0, 0, :, None][:, None]
    k, v = k.masked_fill(~seen, 0.0), v.masked_fill(~seen, 0.0)
    q = st["q"].float().reshape(B, Hkv, G * T, D)
    x = (q @ k.transpose(2, 3) * scale).view(B, Hkv, G, T, -1)
    z, _ = _modified(x, case, st["slopes"], (pos - key).abs().float())
    p, lse = _softmax(z, vis)
    out = (p.view(B, Hkv, G * T, -1) @ v).view(B, H, T, D)
    return dict(out=out.bfloat16(), lse=lse.reshape(B, H, T))


# ------------------------------------------------------ the framework's calls


def _own_attention(st):
    import block_sparse_masked_build_gb300 as bsm
    case, seg = st["case"], st["seg"]
    B, S = case["B"], case["S"]
    flags = {"causal": bsm.MASK_CAUSAL, "full": 0,
             "local": bsm.MASK_CAUSAL | bsm.MASK_LOCAL,
             "packed": bsm.MASK_CAUSAL | bsm.MASK_SEGMENT}[case["mask"]]
    info = bsm.build_mask_info(flags, B, S, S, window=case["window"],
                               q_segment_ids=seg, kv_segment_ids=seg)
    mods = dict(mask_info=info, q_segment_ids=seg, kv_segment_ids=seg,
                softcap=case["softcap"], alibi_slopes=st["slopes"])
    out, lse = bsm.splash_attention(st["q"], st["k"], st["v"], **mods)
    res = dict(out=out, lse=lse)
    if case["op"] == "training":
        res["dq"], res["dk"], res["dv"] = bsm.splash_attention_bwd(
            st["q"], st["k"], st["v"], out, lse, st["dout"], **mods)
    return res


def _own_cache(st):
    import block_sparse_masked_build_gb300 as bsm
    return bsm.KVCache(st["k_pages"], st["v_pages"], st["k_scale"],
                       st["v_scale"])


def _own_append(st):
    import block_sparse_masked_build_gb300 as bsm
    bsm.kv_append(_own_cache(st), st["table"], st["lens"], st["k_new"],
                  st["v_new"], n_new=st["n_new"])
    return _cache_state(st)


def _own_decode(st):
    import block_sparse_masked_build_gb300 as bsm
    case = st["case"]
    out, lse = bsm.paged_attention(
        st["q"], _own_cache(st), st["table"], st["lens"],
        window=case["window"], softcap=case["softcap"],
        alibi_slopes=st["slopes"])
    return dict(out=out, lse=lse)


def run(state):
    op = state["case"]["op"]
    if op == "append":
        return _own_append(state) if own else _plain_append(state)
    if op == "decode":
        return _own_decode(state) if own else _plain_decode(state)
    return _own_attention(state) if own else _plain_attention(state)


# -------------------------------------------------------------------- work


def _pairs(case):
    """Visible (query, key) pairs of one head, over the batch.  Packed
    documents are counted at their mean length."""
    B, S = case["B"], case["S"]
    if case["mask"] == "full":
        return B * S * S
    if case["mask"] == "causal":
        return B * S * (S + 1) // 2
    if case["mask"] == "local":
        w = min(case["window"], S)
        return B * (w * (w + 1) // 2 + (S - w) * w)
    lo, hi = max(1, S // 32), max(2, S // 4)
    mean = (lo + hi) / 2
    square = mean * mean + (hi - lo) ** 2 / 12
    return int(B * S * (square / mean + 1) / 2)


def work(case):
    if case["op"] in ("forward", "training"):
        B, H, Hkv, S, D = (case[n] for n in ("B", "H", "Hkv", "S", "D"))
        q, kv = B * H * S * D * 2, B * Hkv * S * D * 2
        flops = 4 * D * H * _pairs(case)
        nbytes = 2 * q + 2 * kv + 4 * B * H * S
        if case["op"] == "training":
            flops = 14 * D * H * _pairs(case)
            nbytes += 2 * q + 2 * kv  # dout read, dq, dk, dv written
        return dict(bytes=nbytes, flops=flops)
    B, Hkv, D, P, T = (case[n] for n in ("B", "Hkv", "D", "page", "T"))
    if case["op"] == "append":
        n = B * (case["new_lo"] + T) / 2  # tokens, at their mean
        return dict(bytes=n * Hkv * D * 2 * 3 + 8 * Hkv * (n / P + B),
                    flops=n * Hkv * D * 2 * 2)
    H = case["H"]
    mean = (case["len_lo"] + case["len_hi"]) / 2
    seen = min(mean, case["window"] + T - 1) if case["window"] else mean
    nbytes = B * (seen * Hkv * D * 2 + seen / P * (8 * Hkv + 4)
                  + H * T * (4 * D + 4))
    return dict(bytes=nbytes, flops=4 * D * B * H * T * seen)


# ---------------------------------------------------- definition in 64 bits


def _exact_row(q, k, v, scale, case, slope, qpos, kpos, vis):
    """One head: q [T, D], k and v [L, D] in 64 bits -> (out, lse)."""
    x = (q @ k.T) * scale
    if case["softcap"] > 0:
        c = case["softcap"]
        e = torch.exp(-2.0 * x.abs() / c)
        x = torch.sign(x) * c * (1.0 - e) / (1.0 + e)
    if slope is not None:
        x = x - slope * (qpos[:, None] - kpos[None, :]).abs()
    x = x.masked_fill(~vis, -math.inf)
    lse = torch.logsumexp(x, -1)
    live = torch.isfinite(lse)
    w = torch.exp(x - torch.where(live, lse, torch.zeros_like(lse))[:, None])
    return w @ v, lse


def _exact_attention(case, st):
    B, H, Hkv, S, D = (case[n] for n in ("B", "H", "Hkv", "S", "D"))
    G, train = H // Hkv, case["op"] == "training"
    dev = st["q"].device
    pos = torch.arange(S, device=dev, dtype=torch.float64)
    out = torch.empty(B, H, S, D, dtype=torch.float64, device=dev)
    lse = torch.empty(B, H, S, dtype=torch.float64, device=dev)
    dq = torch.zeros_like(out)
    dk = torch.zeros(B, Hkv, S, D, dtype=torch.float64, device=dev)
    dv = torch.zeros_like(dk)
    for b in range(B):
        vis = torch.ones(S, S, dtype=torch.bool, device=dev)
        if case["mask"] != "full":
            vis = vis.tril()
        if case["mask"] == "local":
            vis = vis.triu(1 - case["window"])
        if st["seg"] is not None:
            vis &= st["seg"][b][:, None] == st["seg"][b][None, :]
        for h in range(H):
            j = h // G
            q = st["q"][b, h].double().requires_grad_(train)
            k = st["k"][b, j].double().requires_grad_(train)
            v = st["v"][b, j].double().requires_grad_(train)
            slope = float(st["slopes"][h]) if case["alibi"] else None
            o, l = _exact_row(q, k, v, D ** -0.5, case, slope, pos, pos, vis)
            out[b, h], lse[b, h] = o.detach(), l.detach()
            if train:
                gq, gk, gv = torch.autograd.grad(
                    o, (q, k, v), st["dout"][b, h].double())
                dq[b, h] = gq
                dk[b, j] += gk
                dv[b, j] += gv
    res = dict(out=out, lse=lse)
    if train:
        res.update(dq=dq, dk=dk, dv=dv)
    return res


def _exact_e4m3(x):
    """x (64 bits) rounded to the nearest e4m3 value, ties to even."""
    x = x.clamp(-448, 448)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30)))
    # log2 may land on the wrong side of a power of two
    e = torch.where(torch.exp2(e) > x.abs(), e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= x.abs(), e + 1, e).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _exact_append(case, st):
    P = case["page"]
    lens, new = st["lens"].tolist(), st["n_new"].tolist()
    table = st["table"].tolist()
    res = {}
    for name in ("k", "v"):
        pages = st[name + "_pages"].double()
        scales = st[name + "_scale"].double()
        for b in range(case["B"]):
            at, end = lens[b], lens[b] + new[b]
            while at < end:
                pid, lo = table[b][at // P], at % P
                hi = min(P, lo + end - at)
                x = st[name + "_new"][b, :, at - lens[b]:
                                      at - lens[b] + hi - lo].double()
                amax = x.abs().amax((1, 2))
                need = torch.exp2(torch.ceil(torch.log2(
                    amax.clamp(min=1e-30) / 448.0)).clamp(-40, 40))
                scale = torch.maximum(scales[pid], need) if lo else need
                if lo:
                    pages[pid, :, :lo] = torch.where(
                        (scale > scales[pid])[:, None, None],
                        _exact_e4m3(pages[pid, :, :lo] * (
                            scales[pid] / scale)[:, None, None]),
                        pages[pid, :, :lo])
                pages[pid, :, lo:hi] = _exact_e4m3(x / scale[:, None, None])
                scales[pid] = scale
                at += hi - lo
        res[name + "_pages"], res[name + "_scale"] = pages, scales
    return res


def _exact_decode(case, st):
    B, H, Hkv, D, P, T = (case[n] for n in ("B", "H", "Hkv", "D", "page", "T"))
    dev = st["q"].device
    out = torch.empty(B, H, T, D, dtype=torch.float64, device=dev)
    lse = torch.empty(B, H, T, dtype=torch.float64, device=dev)
    for b, n in enumerate(st["lens"].tolist()):
        qpos = torch.arange(n - T, n, device=dev, dtype=torch.float64)
        kpos = torch.arange(n, device=dev, dtype=torch.float64)
        gap = qpos[:, None] - kpos[None, :]
        vis = gap >= 0
        if case["window"] > 0:
            vis &= gap < case["window"]
        ids = st["table"][b, :(n + P - 1) // P].long()
        kv = []
        for name in ("k", "v"):
            x = st[name + "_pages"].view(torch.uint8)[ids].view(
                torch.float8_e4m3fn).double()
            x = x * st[name + "_scale"][ids].double()[:, :, None, None]
            kv.append(x.transpose(0, 1).reshape(Hkv, -1, D)[:, :n])
        for h in range(H):
            j = h // (H // Hkv)
            slope = float(st["slopes"][h]) if case["alibi"] else None
            out[b, h], lse[b, h] = _exact_row(
                st["q"][b, h].double(), kv[0][j], kv[1][j], D ** -0.5, case,
                slope, qpos, kpos, vis)
    return dict(out=out, lse=lse)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "decode":
        return _exact_decode(case, st)
    return _exact_attention(case, st)
