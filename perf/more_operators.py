"""Cases of the head norm with position rotation (forward and backward), of
the 8-bit cache's append with both on the way, and of attention of a tree of
drafted tokens over that cache: their inputs, a plain form in elementary torch
operations, the framework's calls, and their definition in 64 bits.

Norm and rotation of a head's row x [D]: y = w x / sqrt(mean(x^2) + eps) where
normalised; of its first `rot` elements the pairs (i, i + rot / 2), or (2 i, 2
i + 1), turn by the angle position[axis of i] * base^(-2 i / rot).

Cache: pages of `page` tokens per key/value head in e4m3 with one power-of-two
scale per (page, head).  Of a sequence's tokens the last n are drafts; draft t
sees all tokens before the drafts and the drafts whose bits its row of `tree`
has; its position is the first draft's plus its depth (bits set, less one).
"""

import functools
import math

import torch

own = False

EPS = 1e-6

# ------------------------------------------------------------------- cases


def listed():
    return [
        # one new token for each of a few sequences: launch and host latency
        dict(name="rotate_step", op="rotate", B=8, H=32, Hkv=8, S=1, D=128,
             rot=128, base=1e6, inter=False, norm=True, wide=False, axes=1,
             where="step", far=30000),
        # one long prompt, grouped heads, norm and rotation
        dict(name="rotate_prompt", op="rotate", B=1, H=32, Hkv=8, S=8192,
             D=128, rot=128, base=1e6, inter=False, norm=True, wide=False,
             axes=1, where="prompt", far=100000),
        # a video between texts: positions of three axes, odd length
        dict(name="rotate_video", op="rotate", B=2, H=16, Hkv=4, S=2999,
             D=128, rot=128, base=1e6, inter=False, norm=False, wide=False,
             axes=3, where="video", far=1000),
        # forward and backward of a short ragged batch row, half of each head
        # rotated, neighbouring elements paired
        dict(name="rotate_train_short", op="training", B=1, H=4, Hkv=2, S=300,
             D=64, rot=32, base=1e4, inter=True, norm=True, wide=True, axes=1,
             where="prompt", far=0),
        # forward and backward of a training batch of packed documents
        dict(name="rotate_train_packed", op="training", B=2, H=16, Hkv=16,
             S=8192, D=128, rot=128, base=1e4, inter=False, norm=True,
             wide=True, axes=1, where="packed", far=0),
        # one new token for each sequence being served, key normalised and
        # rotated on the way
        dict(name="append_step", op="append", B=64, Hkv=8, D=128, page=64,
             T=1, new_lo=1, len_lo=100, len_hi=20000, rot=128, base=1e6,
             inter=False, norm=True, axes=1, drafts=False),
        # the keys and values of a batch of prompts go into the cache
        dict(name="append_prompts", op="append", B=8, Hkv=8, D=128, page=64,
             T=2048, new_lo=500, len_lo=0, len_hi=0, rot=128, base=1e6,
             inter=False, norm=True, axes=1, drafts=False),
        # drafted tokens, positions by their depth in a tree
        dict(name="append_drafts", op="append", B=16, Hkv=8, D=128, page=64,
             T=48, new_lo=20, len_lo=300, len_hi=12000, rot=128, base=1e4,
             inter=False, norm=False, axes=1, drafts=True),
        # one sequence, a few drafts: latency
        dict(name="tree_one", op="tree", B=1, H=32, Hkv=8, D=128, page=64,
             T=8, new_lo=8, len_lo=2000, len_hi=2000, window=0, softcap=0.0,
             alibi=False),
        # a serving batch of unequal lengths, a small tree each
        dict(name="tree_batch", op="tree", B=32, H=32, Hkv=8, D=128, page=64,
             T=16, new_lo=7, len_lo=300, len_hi=12000, window=0, softcap=0.0,
             alibi=False),
        # wide trees: as much a matrix product as a walk over the cache
        dict(name="tree_wide", op="tree", B=16, H=32, Hkv=8, D=128, page=64,
             T=64, new_lo=64, len_lo=2000, len_hi=12000, window=0,
             softcap=0.0, alibi=False),
        # few very long sequences, capped scores
        dict(name="tree_long", op="tree", B=2, H=32, Hkv=8, D=128, page=128,
             T=25, new_lo=25, len_lo=100000, len_hi=131072, window=0,
             softcap=50.0, alibi=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "training", "append", "tree"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 6, 8])
    turn = dict(rot=rng.choice([D, D, D // 2, D - 16]),
                base=rng.choice([1e4, 5e5, 1e6]), inter=rng.random() < 0.3,
                norm=rng.random() < 0.7, axes=rng.choice([1, 1, 1, 2, 3]))
    if op in ("rotate", "training"):
        G = min(G, max(1, 32 // Hkv))
        S = _log(rng, 1, 8192)
        B = max(1, min(_log(rng, 1, 64), 8192 // S))
        where = "video" if turn["axes"] > 1 else rng.choice(
            ["prompt", "packed", "step"])
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, S=S, D=D, where=where,
                    wide=rng.random() < 0.5,
                    far=rng.choice([0, 1000, 100000, 250000]), **turn)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        kind = rng.choice(["step", "prompt", "drafts"])
        T = {"step": rng.choice([1, 1, 2, 4]), "prompt": _log(rng, 20, 2000),
             "drafts": _log(rng, 4, 128)}[kind]
        B = rng.choice([1, 2, 5, 8]) if kind == "prompt" else _log(rng, 1, 64)
        len_hi = _log(rng, 50, 4000)
        if kind == "drafts":
            turn["axes"] = 1
        return dict(op=op, B=B, Hkv=Hkv, D=D, page=page, T=T,
                    new_lo=max(1, T // 3), len_lo=rng.choice([0, len_hi // 5]),
                    len_hi=len_hi, drafts=kind == "drafts", **turn)
    softcap, alibi = rng.choice([(0.0, False), (0.0, False), (50.0, False),
                                 (0.0, True), (30.0, True)])
    T = _log(rng, 1, 128)
    B = _log(rng, 1, 64)
    top = min(131072, 400000 // max(B, 3), int(2.4e8 / (B * T * Hkv * G)))
    len_hi = max(T + 200, _log(rng, 200, max(201, top)))
    return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, D=D, page=page, T=T,
                new_lo=rng.choice([T, max(1, T // 3)]),
                len_lo=max(T, len_hi // rng.choice([1, 4, 30])),
                len_hi=len_hi, softcap=softcap, alibi=alibi,
                window=rng.choice([0, 0, 0, _log(rng, 50, 4000)]))


# ------------------------------------------------------------------ inputs


def _axis_of(rot, axes):
    """The axis of each frequency: thirds (halves) of the frequencies."""
    n = rot // 2
    return [min(i * axes // n, axes - 1) for i in range(n)]


def _positions(case, seed):
    """[B, S], or [axes, B, S] of more than one axis; int32 on the host."""
    g = torch.Generator().manual_seed(seed * 7 + 5)
    B, S, far = case["B"], case["S"], case["far"]
    start = torch.randint(0, far + 1, (B, 1), generator=g)
    s = torch.arange(S).expand(B, S)
    if case["where"] == "step":  # S tokens of sequences of unequal lengths
        return (s + start).int()
    if case["where"] == "prompt":
        return (s + far).int()
    if case["where"] == "packed":  # positions start anew in each document
        lo, hi = max(1, S // 32), max(2, S // 4)
        n = torch.randint(lo, hi + 1, (B, S // lo + 1), generator=g)
        end = torch.cumsum(n, 1)
        doc = torch.searchsorted(end, s.contiguous(), right=True)
        return (s - (end - n).gather(1, doc)).int()
    # video: text, then frames of 12 x 20 patches, and text after them
    head = torch.randint(0, max(1, S // 8) + 1, (B, 1), generator=g)
    count = max(1, S * 3 // 4)
    at = (s - head).clamp(0, count - 1)
    frame, patch = at // 240, at % 240
    inside = (s >= head) & (s < head + count)
    after = s - head - count + 1 + (count - 1) // 240 + 20
    text = torch.where(s < head, s, head + after)
    axis = [head + frame, head + patch // 20, head + patch % 20]
    return torch.stack([torch.where(inside, a, text) + start
                        for a in axis[:case["axes"]]]).int()


def _slopes(H):
    h = torch.arange(1, H + 1, dtype=torch.float64)
    return torch.exp2(-8.0 * h / H).float()


def _ints(lo, hi, n, seed):
    g = torch.Generator().manual_seed(seed * 11 + 3)
    return torch.randint(lo, hi + 1, (n,), generator=g).int()


def _trees(B, T, seed):
    """Bits [B, T, T] of random trees: each draft hangs on an earlier one,
    draft 0 is the root."""
    g = torch.Generator().manual_seed(seed * 13 + 1)
    u = torch.rand(B, T, generator=g)
    t = torch.arange(T)
    parent = (t - 1 - (u * u * (t - 1).clamp(min=0)).floor()).long()
    bits = torch.zeros(B, T, T, dtype=torch.bool)
    for i in range(T):
        if i:
            bits[:, i] = bits.gather(
                1, parent[:, i].view(B, 1, 1).expand(B, 1, T))[:, 0]
        bits[:, i, i] = True
    return bits


def _pack(bits):
    """[B, T, T] truth values -> int32 words [B, T, ceil(T / 32)]."""
    B, T, n = bits.shape
    words = (n + 31) // 32
    full = torch.zeros(B, T, words * 32, dtype=torch.int64)
    full[..., :n] = bits.long()
    v = (full.view(B, T, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(v >= 2 ** 31, v - 2 ** 32, v).int()


def _weight(case, g, dev):
    w = 1.0 + 0.2 * torch.randn(case["D"], generator=g, device=dev)
    return w if case.get("wide") else w.bfloat16()


def _prepare_rotation(case, seed, g, dev):
    B, H, Hkv, S, D = (case[n] for n in ("B", "H", "Hkv", "S", "D"))
    # heads as they lie in one projection's output, of unequal magnitudes
    x = torch.randn(B, S, H + 2 * Hkv, D, generator=g, device=dev)
    x = x * (torch.rand(B, S, H + 2 * Hkv, 1, generator=g, device=dev) * 3
             + 0.2)
    x = x.bfloat16()
    st = dict(case=case, q=x[:, :, :H].transpose(1, 2),
              k=x[:, :, H:H + Hkv].transpose(1, 2),
              positions=_positions(case, seed).to(dev))
    st["q_weight"] = _weight(case, g, dev) if case["norm"] else None
    st["k_weight"] = _weight(case, g, dev) if case["norm"] else None
    if case["op"] == "training":  # gradients as attention's backward has them
        st["gq"] = torch.randn(B, H, S, D, generator=g, device=dev).bfloat16()
        st["gk"] = torch.randn(B, Hkv, S, D, generator=g,
                               device=dev).bfloat16()
    return st


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] in ("rotate", "training"):
        return _prepare_rotation(case, seed, g, dev)
    st = dict(case=case)
    B, Hkv, D, P, T = (case[n] for n in ("B", "Hkv", "D", "page", "T"))
    lens = _ints(case["len_lo"], case["len_hi"], B, seed)
    new = _ints(case["new_lo"], T, B, seed + 1)
    append = case["op"] == "append"
    held = lens + new if append else lens
    pages = (held + P - 1) // P
    width = int((int(case["len_hi"]) + T + P - 1) // P)
    total = B * width if append else int(pages.sum())
    # the sequences' pages lie scattered in the pool, as after some serving
    perm = torch.randperm(total + 3, generator=torch.Generator().manual_seed(
        seed + 17)).int()
    table = torch.full((B, width), -1, dtype=torch.int32)
    first = torch.cumsum(pages, 0) - pages
    slot = torch.arange(width).expand(B, width)
    used = slot < pages[:, None]
    table[used] = perm[(first[:, None] + slot)[used].long()]
    st["table"], st["lens"], st["n_new"] = (
        table.to(dev), lens.to(dev), new.to(dev))
    shape = (total + 3, Hkv, P, D)
    for n in ("k", "v"):
        codes = torch.randn(shape, generator=g, device=dev) * 110.0
        st[n + "_pages"] = codes.clamp_(-448, 448).to(torch.float8_e4m3fn)
        st[n + "_scale"] = torch.exp2(torch.randint(
            -8, -5, shape[:2], generator=g, device=dev).float())
        del codes
    if append:
        for n in ("k_new", "v_new"):  # as a projection leaves them
            x = torch.randn(B, T, Hkv, D, generator=g, device=dev)
            st[n] = x.bfloat16().transpose(1, 2)
        if case["drafts"]:
            depth = _trees(B, T, seed).sum(-1) - 1
            st["positions"] = (lens[:, None] + depth).int().to(dev)
        else:
            at = (lens[:, None] + torch.arange(T)).int()
            st["positions"] = (at.to(dev) if case["axes"] == 1 else
                               at.expand(case["axes"], B, T).to(dev))
        st["k_weight"] = _weight(case, g, dev) if case["norm"] else None
        return st
    H = case["H"]
    q = torch.randn(B, T, H, D, generator=g, device=dev) * 1.5
    st["q"] = q.bfloat16().transpose(1, 2)
    st["tree"] = _pack(_trees(B, T, seed)).to(dev)
    st["slopes"] = _slopes(H).to(dev) if case["alibi"] else None
    return st


# --------------------------------------------------------------- plain form


def _angles(positions, case):
    """cos and sin, [B, 1, S, rot / 2]; the angles in 64 bits."""
    rot, axes = case["rot"], case["axes"]
    i = torch.arange(rot // 2, device=positions.device, dtype=torch.float64)
    freq = case["base"] ** (-2.0 * i / rot)
    pos = positions if axes > 1 else positions[None]
    axis = torch.tensor(_axis_of(rot, axes), device=positions.device)
    a = pos.permute(1, 2, 0)[..., axis].double() * freq
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _turn(y, cos, sin, case):
    """The rows' first `rot` elements turned by the angles."""
    rot = case["rot"]
    head, rest = y[..., :rot], y[..., rot:]
    if case["inter"]:
        a, b = head[..., 0::2], head[..., 1::2]
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
    c, d = a * cos - b * sin, b * cos + a * sin
    head = (torch.stack((c, d), -1).flatten(-2) if case["inter"]
            else torch.cat((c, d), -1))
    return torch.cat((head, rest), -1)


def _normed(x, w, case):
    """(normalised row, 1 / root mean square) of f32 rows."""
    if not case["norm"]:
        return x, None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r * w.float(), r


def _grad(g, x, w, cos, sin, case):
    """(dx, dw) for the gradient g of the turned rows."""
    h = _turn(g.float(), cos, -sin, case)
    if not case["norm"]:
        return h.bfloat16(), None
    x = x.float()
    _, r = _normed(x, w, case)
    n = x * r
    dw = (h * n).sum((0, 1, 2))
    h = h * w.float()
    return (r * (h - n * (h * n).mean(-1, keepdim=True))).bfloat16(), dw


def _plain_rotate(st):
    case = st["case"]
    cos, sin = _angles(st["positions"], case)
    res = {}
    for n in ("q", "k"):
        y, _ = _normed(st[n].float(), st[n + "_weight"], case)
        res[n] = _turn(y, cos, sin, case).bfloat16()
    if case["op"] == "training":
        for n in ("q", "k"):
            res["d" + n], dw = _grad(st["g" + n], st[n], st[n + "_weight"],
                                     cos, sin, case)
            if dw is not None:
                res["d" + n + "_weight"] = dw
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
    P, T = case["page"], case["T"]
    table, lens, n_new = st["table"], st["lens"].long(), st["n_new"].long()
    slots = (T + P - 2) // P + 1  # pages that T tokens can touch
    page = lens[:, None] // P + torch.arange(slots, device=lens.device)
    tok = page[:, :, None] * P + torch.arange(P, device=lens.device)
    old = tok < lens[:, None, None]
    new = ~old & (tok < (lens + n_new)[:, None, None])
    live = new.any(-1)  # [B, slots]
    pid = table.gather(1, page.clamp(max=table.shape[1] - 1))[live].long()
    at = (tok - lens[:, None, None]).clamp(0, T - 1).view(
        case["B"], 1, -1, 1)
    cos, sin = _angles(st["positions"], case)
    k, _ = _normed(st["k_new"].float(), st["k_weight"], case)
    k = _turn(k, cos, sin, case)
    _put(st["k_pages"].view(torch.uint8), st["k_scale"], k, pid, live, at,
         old, new)
    _put(st["v_pages"].view(torch.uint8), st["v_scale"], st["v_new"], pid,
         live, at, old, new)
    return _cache_state(st)


def _cache_state(st):
    return {n: st[n] for n in ("k_pages", "k_scale", "v_pages", "v_scale")}


def _plain_tree(st):
    case = st["case"]
    B, H, Hkv, D, P, T = (case[n] for n in ("B", "H", "Hkv", "D", "page", "T"))
    G, scale = H // Hkv, 1.0 / math.sqrt(D)
    idx = st["table"].clamp(min=0).long()
    dev = idx.device

    def tokens(name):
        x = st[name + "_pages"].view(torch.uint8)[idx].view(
            torch.float8_e4m3fn).float()
        x = x * st[name + "_scale"][idx][:, :, :, None, None]
        return x.transpose(1, 2).reshape(B, Hkv, -1, D)

    k, v = tokens("k"), tokens("v")
    n = st["n_new"].long()[:, None]
    base = st["lens"].long()[:, None] - n  # [B, 1]
    t = torch.arange(T, device=dev)
    bits = (st["tree"][..., t // 32] >> (t % 32)) & 1  # [B, T, T]
    bits = (bits == 1) & (t < n)[:, None, :] & (t < n)[:, :, None]
    depth = bits.sum(-1) - 1
    there = depth >= 0  # [B, T]
    key = torch.arange(k.shape[2], device=dev)[None]
    draft = (key - base).clamp(0, T - 1)  # [B, L]
    own_bits = bits.gather(2, draft[:, None].expand(B, T, -1))
    vis = torch.where((key < base)[:, None], there[:, :, None],
                      own_bits & (key < base + n)[:, None])
    kpos = torch.where(key < base, key, base + depth.gather(1, draft))
    gap = (base + depth)[:, :, None] - kpos[:, None]  # [B, T, L]
    if case["window"] > 0:
        vis = vis & (gap < case["window"])
    # what no draft sees is never read
    seen = vis.any(1)[:, None, :, None]
    k, v = k.masked_fill(~seen, 0.0), v.masked_fill(~seen, 0.0)
    q = st["q"].float().reshape(B, Hkv, G * T, D)
    x = (q @ k.transpose(2, 3) * scale).view(B, Hkv, G, T, -1)
    if case["softcap"] > 0:
        x = torch.tanh(x / case["softcap"]) * case["softcap"]
    if st["slopes"] is not None:
        x = x - st["slopes"].view(1, Hkv, G, 1, 1) * gap[
            :, None, None].abs().float()
    x = x.masked_fill(~vis[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    out = (p.view(B, Hkv, G * T, -1) @ v).view(B, H, T, D)
    return dict(out=out.bfloat16(), lse=lse.reshape(B, H, T))


# ------------------------------------------------------ the framework's calls


@functools.lru_cache(maxsize=None)
def _rope(rot, base, axes, inter):
    """The rotation that a model keeps."""
    import block_sparse_masked_build_gb300 as bsm
    return bsm.Rope(rot, base, axes=_axis_of(rot, axes) if axes > 1 else None,
                    interleaved=inter)


def _turn_args(st, *weights):
    case = st["case"]
    return dict(rope=_rope(case["rot"], case["base"], case["axes"],
                           case["inter"]),
                positions=st["positions"],
                eps=EPS if case["norm"] else None,
                **{w: st[w] for w in weights})


def _own_rotate(st):
    import block_sparse_masked_build_gb300 as bsm
    case = st["case"]
    args = _turn_args(st, "q_weight", "k_weight")
    q, k = bsm.norm_rope(st["q"], st["k"], **args)
    res = dict(q=q, k=k)
    if case["op"] == "training":
        dq, dk, dqw, dkw = bsm.norm_rope_bwd(st["gq"], st["gk"], st["q"],
                                             st["k"], **args)
        res.update(dq=dq, dk=dk)
        if case["norm"]:
            res.update(dq_weight=dqw, dk_weight=dkw)
    return res


def _own_cache(st):
    import block_sparse_masked_build_gb300 as bsm
    if "cache" not in st:  # a program keeps its cache's handle
        st["cache"] = bsm.KVCache(st["k_pages"], st["v_pages"], st["k_scale"],
                                  st["v_scale"])
    return st["cache"]


def _own_append(st):
    import block_sparse_masked_build_gb300 as bsm
    bsm.kv_append(_own_cache(st), st["table"], st["lens"], st["k_new"],
                  st["v_new"], n_new=st["n_new"], **_turn_args(st, "k_weight"))
    return _cache_state(st)


def _own_tree(st):
    import block_sparse_masked_build_gb300 as bsm
    case = st["case"]
    out, lse = bsm.paged_attention(
        st["q"], _own_cache(st), st["table"], st["lens"], tree=st["tree"],
        n_new=st["n_new"], window=case["window"], softcap=case["softcap"],
        alibi_slopes=st["slopes"])
    return dict(out=out, lse=lse)


def run(state):
    op = state["case"]["op"]
    if op == "append":
        return _own_append(state) if own else _plain_append(state)
    if op == "tree":
        return _own_tree(state) if own else _plain_tree(state)
    return _own_rotate(state) if own else _plain_rotate(state)


# -------------------------------------------------------------------- work


def work(case):
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] in ("rotate", "training"):
        tokens = case["B"] * case["S"]
        n = tokens * (case["H"] + Hkv) * D
        nbytes, flops = 4 * n + 4 * tokens * case["axes"], 7 * n
        if case["op"] == "training":  # gradient and row read, gradient written
            nbytes += 6 * n if case["norm"] else 4 * n
            flops += 12 * n
        return dict(bytes=nbytes, flops=flops)
    B, P, T = case["B"], case["page"], case["T"]
    new = B * (case["new_lo"] + T) / 2  # tokens, at their mean
    if case["op"] == "append":
        return dict(bytes=new * Hkv * D * 2 * 3 + 8 * Hkv * (new / P + B)
                    + 4 * new * case["axes"], flops=new * Hkv * D * 11)
    H = case["H"]
    mean = (case["len_lo"] + case["len_hi"]) / 2
    seen = min(mean, case["window"] + T) if case["window"] else mean
    nbytes = (B * seen * Hkv * D * 2 + B * seen / P * (8 * Hkv + 4)
              + B * H * T * (4 * D + 4) + B * T * 4 * ((T + 31) // 32))
    return dict(bytes=nbytes, flops=4 * D * H * new * seen)


# ---------------------------------------------------- definition in 64 bits


def _exact_rows(x, w, positions, case):
    """x [B, h, S, D] in 64 bits, normalised and turned: pairs as complex
    numbers times e^(i angle)."""
    if case["norm"]:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["D"]
                           + EPS) * w.double()
    rot, half = case["rot"], case["rot"] // 2
    pos = positions.double()
    pos = pos[None] if case["axes"] == 1 else pos
    axis = _axis_of(rot, case["axes"])
    angle = torch.stack([pos[axis[i]] / case["base"] ** (2 * i / rot)
                         for i in range(half)], -1)[:, None]
    unit = torch.polar(torch.ones_like(angle), angle)
    if case["inter"]:
        z = torch.view_as_complex(
            x[..., :rot].unflatten(-1, (half, 2)).contiguous()) * unit
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :half], x[..., half:rot]) * unit
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, x[..., rot:]], -1)


def _exact_rotate(case, st):
    res = {}
    for n in ("q", "k"):
        train = case["op"] == "training"
        x = st[n].double().requires_grad_(train)
        w = st[n + "_weight"]
        w = None if w is None else w.double().requires_grad_(train)
        y = _exact_rows(x, w, st["positions"], case)
        res[n] = y.detach()
        if train:
            of = [x] if w is None else [x, w]
            grads = torch.autograd.grad(y, of, st["g" + n].double())
            res["d" + n] = grads[0]
            if w is not None:
                res["d" + n + "_weight"] = grads[1]
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
    rows = dict(k=_exact_rows(st["k_new"].double(), st["k_weight"],
                              st["positions"], case),
                v=st["v_new"].double())
    res = {}
    for name in ("k", "v"):
        pages = st[name + "_pages"].double()
        scales = st[name + "_scale"].double()
        for b in range(case["B"]):
            at, end = lens[b], lens[b] + new[b]
            while at < end:
                pid, lo = table[b][at // P], at % P
                hi = min(P, lo + end - at)
                x = rows[name][b, :, at - lens[b]:at - lens[b] + hi - lo]
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


def _exact_tree(case, st):
    B, H, Hkv, D, P, T = (case[n] for n in ("B", "H", "Hkv", "D", "page", "T"))
    dev = st["q"].device
    out = torch.zeros(B, H, T, D, dtype=torch.float64, device=dev)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device=dev)
    words = (st["tree"].long() & 0xffffffff).tolist()
    for b, (n, new) in enumerate(zip(st["lens"].tolist(),
                                     st["n_new"].tolist())):
        base = n - new
        rows = [sum(w << (32 * i) for i, w in enumerate(r)) & ((1 << new) - 1)
                for r in words[b][:new]]
        depth = [bin(r).count("1") - 1 for r in rows]
        vis = torch.ones(new, n, dtype=torch.bool)
        vis[:, base:] = torch.tensor([[r >> j & 1 == 1 for j in range(new)]
                                      for r in rows])
        vis = vis.to(dev)
        qpos = torch.tensor(depth, dtype=torch.float64, device=dev) + base
        kpos = torch.arange(n, device=dev, dtype=torch.float64)
        kpos[base:] = qpos
        gap = qpos[:, None] - kpos[None]
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
            x = st["q"][b, h, :new].double() @ kv[0][j].T * D ** -0.5
            if case["softcap"] > 0:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            if case["alibi"]:
                x = x - float(st["slopes"][h]) * gap.abs()
            x = x.masked_fill(~vis, -math.inf)
            lse[b, h, :new] = torch.logsumexp(x, -1)
            out[b, h, :new] = torch.softmax(x, -1) @ kv[1][j]
    return dict(out=out, lse=lse)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "tree":
        return _exact_tree(case, st)
    return _exact_rotate(case, st)
