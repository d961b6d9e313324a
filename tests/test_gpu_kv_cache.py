"""The paged 8-bit cache on the GPU: append bit for bit, attention against
fp64.

Tolerances of the attention.  p becomes f16 (half a step, 2^-11 relative) and
the output bf16 (2^-8); e4m3 codes are exact in f16, and q keeps its bf16
bits.  The logits are f32, for which another 2^-11 of sum p |v| is allowed.
So |error| <= 2^-8 |out| (1 + 2^-7) + 2^-10 sum p |v|.  The logsumexp has the
f32 errors alone: 1e-4 of max(1, |lse|).
"""

import math

import numpy as np
import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import kv_cache_ref as ref

pytestmark = pytest.mark.gpu


def status():
    torch.cuda.synchronize()
    return bsm.bsm_device_status()


def same_codes(got, want):
    """float8 codes against fp64 values, bit for bit but for -0 and NaN."""
    g = ref.decode(got.cpu())
    np.testing.assert_array_equal(g, want)


def check(out, lse, want):
    o, l, spread = want
    out, lse = out.double().cpu(), lse.double().cpu()
    assert torch.isfinite(out).all()
    tol = 2.0 ** -8 * o.abs() * (1 + 2.0 ** -7) + 2.0 ** -10 * spread
    err = (out - o).abs()
    assert (err <= tol + 1e-30).all(), float((err - tol).max())
    dead = torch.isinf(l)
    assert torch.equal(torch.isneginf(lse), dead)
    assert (out[dead] == 0).all()
    rel = (lse - l).abs()[~dead] / l.abs()[~dead].clamp(min=1.0)
    assert rel.numel() == 0 or float(rel.max()) <= 1e-4, float(rel.max())


# ------------------------------------------------------------------ append

APPEND = [
    # page, D, H_kv, T, lens, n_new
    (64, 128, 2, 1, [0, 1, 63, 64, 100], [1, 1, 1, 1, 1]),
    (16, 64, 3, 5, [0, 13, 16, 30], [5, 5, 0, 3]),
    (32, 128, 1, 200, [0, 31, 7], [200, 33, 1]),
    (128, 128, 2, 300, [5, 0], [300, 129]),
    (128, 64, 1, 17, [120], [17]),
]


def _append_case(page, D, Hkv, T, lens, n_new, seed, sigma=1.0):
    B = len(lens)
    width = max((a + n + page - 1) // page for a, n in zip(lens, n_new)) + 1
    total = sum((a + n + page - 1) // page for a, n in zip(lens, n_new)) + 2
    k, v, ks, vs = ref.random_cache(total, Hkv, page, D, seed)
    table = ref.random_table([a + n for a, n in zip(lens, n_new)], page,
                             width, total, seed)
    g = torch.Generator().manual_seed(seed + 1)
    new = [(torch.randn(B, Hkv, T, D, generator=g) * sigma).bfloat16()
           for _ in range(2)]
    return (k, v, ks, vs), table, new


def _append(host, table, lens, n_new, new, strided=False):
    cache = bsm.KVCache(*[t.cuda() for t in host])
    dev = [t.cuda() for t in new]
    if strided:  # as projections leave them, inside a wider buffer
        B, Hkv, T, D = new[0].shape
        wide = torch.zeros(B, T, 2, Hkv, D, dtype=torch.bfloat16).cuda()
        for i in range(2):
            wide[:, :, i] = dev[i].transpose(1, 2)
        dev = [wide[:, :, i].transpose(1, 2) for i in range(2)]
    li = torch.tensor(lens, dtype=torch.int32).cuda()
    ni = None if n_new is None else torch.tensor(n_new,
                                                 dtype=torch.int32).cuda()
    bsm.kv_append(cache, table.cuda(), li, *dev, n_new=ni)
    return cache


def _same(cache, host, table, lens, n_new, new):
    k, v, ks, vs = host
    for pages, scales, x, gp, gs in ((k, ks, new[0], cache.k_pages,
                                      cache.k_scale),
                                     (v, vs, new[1], cache.v_pages,
                                      cache.v_scale)):
        wp, ws = ref.append(pages, scales, table, lens, x, n_new)
        same_codes(gp, wp)
        np.testing.assert_array_equal(gs.cpu().double().numpy(), ws)


@pytest.mark.parametrize("sigma", [1.0, 1e-3, 300.0])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case, sigma):
    # small, equal and larger magnitudes than the pages' old scales: kept,
    # and grown with the old codes rounded again
    page, D, Hkv, T, lens, n_new = APPEND[case]
    host, table, new = _append_case(page, D, Hkv, T, lens, n_new, 10 + case,
                                    sigma)
    cache = _append(host, table, lens, n_new, new, strided=case % 2 == 1)
    assert status()[0] == 0
    _same(cache, host, table, lens, n_new, new)


def test_append_all_new_by_default():
    host, table, new = _append_case(16, 64, 2, 3, [4, 15], [3, 3], 31)
    cache = _append(host, table, [4, 15], None, new)
    _same(cache, host, table, [4, 15], [3, 3], new)


def test_append_special_values():
    page, D, lens, n_new = 16, 64, [0, 3, 0, 5, 0], [4, 4, 4, 4, 4]
    host, table, new = _append_case(page, D, 1, 4, lens, n_new, 32)
    for x in new:
        x[0] = 0.0
        x[1, 0, 1, :8] = torch.tensor([math.inf, -math.inf, math.nan, 0.0,
                                       -0.0, 1e-30, 3e38, 448.0]).bfloat16()
        x[2] = math.nan
        x[3, 0, 2, :4] = torch.tensor([1e30, -1e30, 1e-38, 2e-39]).bfloat16()
        # ties of the rounding: halfway between neighbouring codes
        x[4, 0, 0, :8] = torch.tensor([448.0, 17.0, 19.0, 21.0, 2.0 ** -10,
                                       3 * 2.0 ** -10, 240.0, 232.0]
                                      ).bfloat16()
    cache = _append(host, table, lens, n_new, new)
    assert status()[0] == 0
    _same(cache, host, table, lens, n_new, new)


def test_append_reports_and_skips_bad_indices():
    page, D, T = 16, 64, 4
    lens, n_new = [0, 14, 2, 20], [4, 4, 4, 4]
    host, table, new = _append_case(page, D, 2, T, lens, n_new, 33)
    total = host[0].shape[0]
    good = table.clone()
    table[0, 0] = total          # sequence 0: page past the pool
    table[1, 1] = -5             # sequence 1: its second page
    bad_lens = [0, 14, -3, 20]   # sequence 2: negative length
    cache = _append(host, table, bad_lens, [4, 4, 4, 9], new)  # 3: 9 > T
    st, detail = status()
    assert st == -1 and detail[0] == 2
    # only sequence 1's first page was written
    only = [0, 2, 0, 0]
    _same(cache, host, good, lens, only, new)
    assert status()[0] == 0  # read and cleared


# --------------------------------------------------------------- attention


def _attend(lens, page, D, Hkv, G, T, seed, window=0, softcap=0.0, biased=False,
            spread=2, q_sigma=1.0, host=None, table=None, scale=None):
    B, H = len(lens), Hkv * G
    width = max(1, max((n + page - 1) // page for n in lens)) + 1
    total = sum((n + page - 1) // page for n in lens) + 2
    if host is None:
        host = ref.random_cache(total, Hkv, page, D, seed, spread)
    if table is None:
        table = ref.random_table(lens, page, width, total, seed)
    g = torch.Generator().manual_seed(seed + 2)
    q = (torch.randn(B, T, H, D, generator=g) * q_sigma).bfloat16().transpose(
        1, 2)
    slopes = torch.exp2(-8.0 * torch.arange(1, H + 1) / H) if biased else None
    scale = 1 / math.sqrt(D) if scale is None else scale
    li = torch.tensor(lens, dtype=torch.int32)
    out, lse = bsm.paged_attention(
        q.cuda(), bsm.KVCache(*[t.cuda() for t in host]), table.cuda(),
        li.cuda(), window=window, softcap=softcap, scale=scale,
        alibi_slopes=None if slopes is None else slopes.cuda())
    want = ref.attention(q, *host, table, lens, scale, window, softcap, slopes)
    return out, lse, want


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("T", [1, 3])
def test_attention_lengths(page, D, T):
    out, lse, want = _attend(EDGES, page, D, 2, 2, T, page + D + T,
                             softcap=6.0)
    assert status()[0] == 0
    check(out, lse, want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,T", [(1, 1), (5, 1), (8, 1), (9, 1), (16, 1),
                                 (20, 1), (1, 7), (3, 5), (8, 4), (2, 40)])
def test_attention_rows(G, T, D):
    # query rows of a head: less than a tile of 8, a whole one, two, more
    out, lse, want = _attend([300, 41, 8], 32, D, 2, G, T, G * T + D,
                             biased=True)
    assert status()[0] == 0
    check(out, lse, want)


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("window", [1, 16, 33, 1000])
def test_attention_window(window, T):
    out, lse, want = _attend([0, 1, 30, 48, 700], 16, 128, 1, 4, T,
                             window + T, window=window, softcap=8.0,
                             biased=True)
    check(out, lse, want)


@pytest.mark.parametrize("softcap,biased", [(0.0, False), (5.0, False),
                                            (0.0, True), (5.0, True)])
def test_attention_long(softcap, biased):
    out, lse, want = _attend([9000, 5, 4097], 64, 128, 2, 4, 1, 77,
                             softcap=softcap, biased=biased, q_sigma=2.0)
    check(out, lse, want)


@pytest.mark.parametrize("cap", [0.3, 250.0, 5e4])
def test_attention_caps(cap):
    # scores far beyond the cap, and caps that hardly bend them
    out, lse, want = _attend([300, 77], 16, 64, 2, 3, 2, 79, softcap=cap,
                             q_sigma=9.0)
    check(out, lse, want)


def test_attention_widest_window():
    out, lse, want = _attend([100, 3], 16, 64, 1, 2, 3, 80,
                             window=2 ** 31 - 1)
    check(out, lse, want)


def test_attention_many_sequences():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 400, (200,), generator=g).tolist()
    out, lse, want = _attend(lens, 16, 64, 1, 2, 1, 78)
    assert status()[0] == 0
    check(out, lse, want)


def test_attention_scales_far_apart():
    # value scales from 2^-40 to 2^40, key scales kept small: o changes its
    # unit back and forth, and pages of tiny values add nothing, not garbage
    lens, page, D = [700, 64], 16, 128
    k, v, ks, vs = ref.random_cache(50, 2, page, D, 81, spread=1)
    e = torch.randint(-40, 41, vs.shape,
                      generator=torch.Generator().manual_seed(4)).float()
    for n in range(vs.shape[0] // 2):
        vs[n] = torch.exp2(e[n])
    table = ref.random_table(lens, page, 45, 50, 82)
    out, lse, want = _attend(lens, page, D, 2, 3, 1, 83, host=(k, v, ks, vs),
                             table=table)
    check(out, lse, want)


def test_attention_extreme_queries():
    # query rows of zeros, tiny and huge magnitudes
    for sigma, scale in ((0.0, 0.1), (1e-30, 1e29), (1e30, 1e-31)):
        out, lse, want = _attend([100, 17], 16, 64, 2, 3, 2, 84,
                                 q_sigma=sigma, scale=scale)
        check(out, lse, want)


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("window", [0, 20])
def test_nan_where_nobody_looks(T, window):
    # NaN codes behind the last token and before the window change nothing;
    # NaN in a key or value reaches exactly the rows that see it
    lens, page, D, Hkv, G = [45, 77, 16], 16, 128, 1, 2
    k, v, ks, vs = ref.random_cache(20, Hkv, page, D, 85)
    table = ref.random_table(lens, page, 6, 20, 86)
    kb, vb = k.view(torch.uint8), v.view(torch.uint8)
    used = torch.zeros(20, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(max(0, n - T - window + 1) if window else 0, n):
            used[table[b, j // page].item(), j % page] = True
    for x in (kb, vb):
        x.permute(0, 2, 1, 3)[~used] = 0x7f
    out, lse, want = _attend(lens, page, D, Hkv, G, T, 87, window=window,
                             host=(k, v, ks, vs), table=table)
    check(out, lse, want)
    if T == 1:
        return
    # the newest token's value: seen by the last query alone
    n = lens[1]
    vb[table[1, (n - 1) // page].item(), 0, (n - 1) % page, 7] = 0xff
    out, lse, want = _attend(lens, page, D, Hkv, G, T, 87, window=window,
                             host=(k, v, ks, vs), table=table)
    nan = torch.isnan(out.float()).cpu()
    assert torch.equal(nan, torch.isnan(want[0]))
    assert int(nan.sum()) == G  # one dim of the last query of each head
    # the newest token's key: every dim of the last query
    kb[table[0, (lens[0] - 1) // page].item(), 0, (lens[0] - 1) % page, 3] = \
        0x7f
    out, lse, want = _attend(lens, page, D, Hkv, G, T, 87, window=window,
                             host=(k, v, ks, vs), table=table)
    assert torch.equal(torch.isnan(out.float()).cpu(), torch.isnan(want[0]))
    assert torch.equal(torch.isnan(lse).cpu(), torch.isnan(want[1]))


def test_attention_reports_and_masks_bad_indices():
    lens, page, D = [40, 64, 30], 16, 64
    host = ref.random_cache(20, 2, page, D, 88)
    table = ref.random_table(lens, page, 4, 20, 89)
    q = torch.randn(3, 4, 1, D, generator=torch.Generator().manual_seed(
        5)).bfloat16()
    cache = bsm.KVCache(*[t.cuda() for t in host])
    want = ref.attention(q, *host, table, lens, 0.125)
    bad = table.clone()
    bad[0, 2] = 20       # its last 8 tokens
    bad[1, 1] = -1       # a page in the middle
    over = torch.tensor([40, 64, 30000], dtype=torch.int32).cuda()
    out, lse = bsm.paged_attention(q.cuda(), cache, bad.cuda(), over,
                                   scale=0.125)
    st, detail = status()
    assert st == -1 and detail[0] == 2
    assert torch.isfinite(out).all()
    # sequence 0 without its last page is a sequence of 32 tokens
    short = ref.attention(q, *host, table, [32, 64, 30], 0.125)
    check(out[:1], lse[:1], [x[:1] for x in short])
    good = torch.tensor(lens, dtype=torch.int32).cuda()
    out, lse = bsm.paged_attention(q.cuda(), cache, table.cuda(), good,
                                   scale=0.125)
    assert status()[0] == 0
    check(out, lse, want)


def test_attention_outputs_in_place_and_padding_left_alone():
    lens, page, D, H, T = [33, 50], 16, 64, 4, 2
    host = ref.random_cache(12, 2, page, D, 90)
    table = ref.random_table(lens, page, 5, 12, 91)
    q = torch.randn(2, H, T, D, generator=torch.Generator().manual_seed(
        6)).bfloat16()
    wide = torch.full((3, T + 1, H, 2 * D), 7.0, dtype=torch.bfloat16).cuda()
    out = wide[:2, :T, :, :D].transpose(1, 2)
    got, lse = bsm.paged_attention(
        q.cuda(), bsm.KVCache(*[t.cuda() for t in host]), table.cuda(),
        torch.tensor(lens, dtype=torch.int32).cuda(), out=out,
        return_lse=False)
    assert got is out and lse is None
    want = ref.attention(q, *host, table, lens, 1 / math.sqrt(D))
    check(out, want[1], want)
    wide[:2, :T, :, :D] = 7.0
    assert (wide == 7.0).all()


def test_empty_calls():
    k, v, ks, vs = (t.cuda() for t in ref.random_cache(2, 2, 16, 64, 92))
    cache = bsm.KVCache(k, v, ks, vs)
    none = torch.zeros(0, dtype=torch.int32).cuda()
    out, lse = bsm.paged_attention(
        torch.zeros(0, 4, 1, 64, dtype=torch.bfloat16).cuda(), cache,
        torch.zeros(0, 3, dtype=torch.int32).cuda(), none)
    assert out.shape == (0, 4, 1, 64)
    # no page at all: every row sees nothing
    out, lse = bsm.paged_attention(
        torch.ones(2, 4, 1, 64, dtype=torch.bfloat16).cuda(), cache,
        torch.zeros(2, 0, dtype=torch.int32).cuda(),
        torch.zeros(2, dtype=torch.int32).cuda())
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert status()[0] == 0


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("D,page,G", [(128, 64, 4), (64, 16, 2)])
def test_prompt_then_tokens(D, page, G):
    """A prompt's forward, its keys and values into the cache, then tokens
    one by one: each step's cache bit for bit, its attention against fp64."""
    B, Hkv, steps, cap = 2, 2, 5, 6.0
    H = Hkv * G
    prompt = [page + 5, 2 * page - 2]
    S = max(prompt)
    g = torch.Generator().manual_seed(D)
    sl = torch.exp2(-8.0 * torch.arange(1, H + 1) / H)
    mk = lambda h, n: torch.randn(B, h, n, D, generator=g).bfloat16()  # noqa
    q, k, v = mk(H, S), mk(Hkv, S), mk(Hkv, S)
    out, lse = bsm.splash_attention(q.cuda(), k.cuda(), v.cuda(), softcap=cap,
                                    alibi_slopes=sl.cuda())
    total = 12
    table = ref.random_table([n + steps for n in prompt], page, 4, total, 7)
    cache = bsm.KVCache.empty(total, Hkv, page, D)
    for t in (cache.k_pages, cache.v_pages):
        t.view(torch.uint8).fill_(0x7f)  # what a recycled page may hold
    host = [t.cpu().clone() for t in (cache.k_pages, cache.v_pages,
                                      cache.k_scale, cache.v_scale)]
    td = table.cuda()
    lens = torch.zeros(B, dtype=torch.int32).cuda()
    n_new = torch.tensor(prompt, dtype=torch.int32).cuda()
    bsm.kv_append(cache, td, lens, k.cuda(), v.cuda(), n_new=n_new)
    _same(cache, host, table, [0, 0], prompt, (k, v))
    lens += n_new
    have = list(prompt)
    for i in range(steps):
        before = [t.cpu().clone() for t in (cache.k_pages, cache.v_pages,
                                            cache.k_scale, cache.v_scale)]
        q1, k1, v1 = mk(H, 1), mk(Hkv, 1) * (i + 1), mk(Hkv, 1)
        bsm.kv_append(cache, td, lens, k1.cuda(), v1.cuda())
        lens += 1
        out, lse = bsm.paged_attention(q1.cuda(), cache, td, lens,
                                       softcap=cap, alibi_slopes=sl.cuda())
        _same(cache, before, table, have, [1, 1], (k1, v1))
        have = [n + 1 for n in have]
        now = [t.cpu() for t in (cache.k_pages, cache.v_pages, cache.k_scale,
                                 cache.v_scale)]
        check(out, lse, ref.attention(q1, *now, table, have,
                                      1 / math.sqrt(D), 0, cap, sl))
    assert status()[0] == 0


def test_captured_step_and_side_stream():
    """A captured step of append and attention replayed with other tokens and
    lengths, on another stream, gives what eager calls give."""
    B, Hkv, G, D, page = 3, 2, 4, 128, 32
    H = Hkv * G
    lens0 = [40, 700, 31]
    host = ref.random_cache(60, Hkv, page, D, 95)
    table = ref.random_table([n + 4 for n in lens0], page, 30, 60, 96).cuda()
    g = torch.Generator().manual_seed(9)
    toks = [[(torch.randn(B, h, 1, D, generator=g)).bfloat16().cuda()
             for h in (H, Hkv, Hkv)] for _ in range(3)]

    def fresh():
        return bsm.KVCache(*[t.cuda().clone() for t in host])

    def step(cache, lens, q, k, v):
        bsm.kv_append(cache, table, lens, k, v)
        lens.add_(1)
        return bsm.paged_attention(q, cache, table, lens, softcap=9.0)

    eager, cache = [], fresh()
    lens = torch.tensor(lens0, dtype=torch.int32).cuda()
    for x in toks:
        eager.append([t.clone() for t in step(cache, lens, *x)])
    cache = fresh()
    lens = torch.tensor(lens0, dtype=torch.int32).cuda()
    buf = [t.clone() for t in toks[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(cache, lens, *buf)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x, want in zip(toks, eager):
            for d, s in zip(buf, x):
                d.copy_(s)
            graph.replay()
            side.synchronize()
            assert torch.equal(res[0], want[0])
            assert torch.equal(res[1], want[1])
    assert status()[0] == 0


def test_two_calls_at_once():
    # the same inputs on two streams at once and alone: equal bits
    lens, page, D = [3000, 100, 2500], 64, 128
    host = ref.random_cache(100, 2, page, D, 97)
    table = ref.random_table(lens, page, 50, 100, 98).cuda()
    cache = bsm.KVCache(*[t.cuda() for t in host])
    li = torch.tensor(lens, dtype=torch.int32).cuda()
    qs = [torch.randn(3, 8, 1, D, generator=torch.Generator().manual_seed(
        i)).bfloat16().cuda() for i in range(2)]
    alone = [bsm.paged_attention(q, cache, table, li) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        both = []
        for q, s in zip(qs, streams):
            with torch.cuda.stream(s):
                both.append(bsm.paged_attention(q, cache, table, li))
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
