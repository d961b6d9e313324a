"""Attention of drafted tokens over the paged 8-bit cache on the GPU, against
fp64.

Tolerances, as for the cache's attention of single tokens: p becomes f16 (half
a step, 2^-11 relative), the output bf16 (2^-8); e4m3 codes are exact in f16
and q keeps its bf16 bits; the f32 logits and the f16 value of a code times a
scale that is no power of two of its neighbours' may cost another 2^-11 of sum
p |v|.  So |error| <= 2^-8 |out| (1 + 2^-7) + 2^-10 sum p |v|; the logsumexp
has the f32 errors alone, 1e-4 of max(1, |lse|).
"""

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import kv_cache_ref as cref
import tree_ref as ref
from test_gpu_binding import both  # noqa: F401  (a fixture)
from test_gpu_kv_cache import check, status

pytestmark = pytest.mark.gpu

# page, D, H, Hkv, T, lens, n_new (None: all T), window, softcap, bias, tree
CASES = [
    (64, 128, 2, 2, 1, [1, 100, 64], None, 0, 0.0, False, True),
    (64, 128, 8, 2, 5, [5, 6, 70, 133, 300], [5, 0, 3, 5, 1], 0, 0.0, False,
     True),
    (16, 64, 4, 4, 9, [9, 40, 0, 25], [9, 4, 0, 9], 0, 0.0, False, True),
    (32, 128, 16, 2, 16, [300, 16, 129], [16, 9, 16], 0, 0.0, False, True),
    (64, 128, 32, 8, 8, [2000], None, 0, 0.0, False, True),
    (128, 128, 8, 2, 25, [700, 153, 280], [25, 25, 20], 0, 50.0, False, True),
    (16, 64, 6, 2, 33, [400, 33, 257], [33, 33, 1], 0, 0.0, True, True),
    (64, 128, 8, 1, 32, [500, 160], [32, 32], 70, 0.0, False, True),
    (32, 64, 4, 1, 40, [290, 200], [40, 39], 7, 20.0, True, True),
    (64, 128, 12, 4, 64, [1000, 64, 200], [64, 64, 40], 0, 0.0, False, True),
    (128, 64, 8, 2, 64, [900, 100], [64, 3], 0, 30.0, True, True),
    (64, 128, 6, 2, 100, [350, 128], [100, 77], 40, 0.0, True, True),
    (64, 128, 4, 2, 130, [700, 130], [130, 100], 0, 0.0, False, True),
    (16, 128, 3, 1, 257, [600], [257], 0, 0.0, False, True),
    (64, 128, 8, 2, 6, [6, 40, 300], [6, 2, 6], 0, 0.0, False, False),
    (64, 64, 8, 2, 70, [70, 400, 128], [70, 11, 70], 0, 0.0, True, False),
    (32, 128, 8, 2, 48, [500, 10], [48, 0], 60, 50.0, False, False),
    (64, 128, 5, 5, 3, [3000, 3], None, 0, 0.0, False, True),
]


def _case(page, D, H, Hkv, T, lens, n_new, window, softcap, bias, tree,
          seed=0, spread=3, empty=0.1):
    B = len(lens)
    n_new = [min(T, n) for n in lens] if n_new is None else n_new
    width = max((n + page - 1) // page for n in lens) + 1
    total = sum((n + page - 1) // page for n in lens) + 2
    host = cref.random_cache(total, Hkv, page, D, seed, spread=spread)
    table = cref.random_table(lens, page, width, total, seed)
    g = torch.Generator().manual_seed(seed + 5)
    q = (torch.randn(B, H, T, D, generator=g) * 1.5).bfloat16()
    slopes = torch.exp2(-torch.arange(1, H + 1) * 6.0 / H) if bias else None
    bits = ref.random_tree(B, T, seed + 9, empty) if tree else None
    return dict(host=host, table=table, q=q, slopes=slopes, bits=bits,
                n_new=n_new, lens=lens, window=window, softcap=softcap)


def _want(d, scale=None):
    D = d["q"].shape[3]
    return ref.attention(d["q"], *d["host"], d["table"], d["lens"], d["n_new"],
                         d["bits"], D ** -0.5 if scale is None else scale,
                         d["window"], d["softcap"], d["slopes"])


def _ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _run(d, given=True, q=None, scale=None, **kw):
    cache = bsm.KVCache(*[t.cuda() for t in d["host"]])
    return bsm.paged_attention(
        d["q"].cuda() if q is None else q, cache, d["table"].cuda(),
        _ints(d["lens"]), window=d["window"], softcap=d["softcap"],
        alibi_slopes=None if d["slopes"] is None else d["slopes"].cuda(),
        tree=None if d["bits"] is None else ref.pack(d["bits"]).cuda(),
        n_new=_ints(d["n_new"]) if given else None, scale=scale, **kw)


@pytest.mark.parametrize("case", CASES)
def test_against_the_definition(both, case):  # noqa: F811
    d = _case(*case)
    want = _want(d)
    for out, lse in both(lambda: _run(d, given=case[6] is not None)):
        check(out, lse, want)
    assert status()[0] == 0


@pytest.mark.parametrize("case", [CASES[3], CASES[9], CASES[13]])
def test_a_full_lower_triangle_is_a_chain(case):
    """The tree of one guess, and no tree, and (as a chain's rows are a
    sequence's last tokens) the attention without drafts."""
    d = _case(*case)
    T = d["q"].shape[2]
    d["lens"] = [max(n, T) for n in d["lens"]]
    d = _case(*case[:5], d["lens"], [T] * len(d["lens"]), *case[7:])
    d["bits"] = torch.ones(len(d["lens"]), T, T, dtype=torch.bool).tril()
    a = _run(d)
    d["bits"] = None
    b = _run(d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    cache = bsm.KVCache(*[t.cuda() for t in d["host"]])
    out, lse = bsm.paged_attention(d["q"].cuda(), cache, d["table"].cuda(),
                                   _ints(d["lens"]))
    want = _want(d)
    check(out, lse, want)
    check(*a, want)


def test_one_tree_for_all_and_wider_rows():
    d = _case(64, 128, 8, 2, 40, [200, 300], [40, 40], 0, 0.0, False, True)
    d["bits"][1] = d["bits"][0]
    want = _run(d)
    words = ref.pack(d["bits"][0]).cuda()
    wide = torch.full((40, 5), -1, dtype=torch.int32).cuda()
    wide[:, :2] = words
    cache = bsm.KVCache(*[t.cuda() for t in d["host"]])
    args = (d["q"].cuda(), cache, d["table"].cuda(), _ints(d["lens"]))
    for tree in (words, wide[:, :2], wide, words[None].expand(2, 40, 2),
                 words.view(torch.uint32)):
        got = bsm.paged_attention(*args, tree=tree, n_new=_ints([40, 40]))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_bits_behind_the_drafts_are_not_looked_at():
    d = _case(64, 128, 8, 2, 40, [200, 300], [33, 20], 30, 0.0, True, True)
    want = _run(d)
    for b, n in enumerate(d["n_new"]):
        d["bits"][b, :, n:] = True
        d["bits"][b, n:] = True
    got = _run(d)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_strides_and_given_outputs(both):  # noqa: F811
    d = _case(*CASES[9])
    want = _want(d)
    B, H, T, D = d["q"].shape
    base = torch.zeros(B, T, H + 3, D, dtype=torch.bfloat16).cuda()
    q = base[:, :, 1:H + 1].transpose(1, 2)
    q.copy_(d["q"])

    def run():
        wide = torch.full((B, T, H + 2, D), 7.0, dtype=torch.bfloat16).cuda()
        out = wide[:, :, 1:-1].transpose(1, 2)
        lse = torch.zeros(B, H, T).cuda()
        got = _run(d, q=q, out=out, lse=lse)
        assert got[0] is out and got[1] is lse
        assert (wide[:, :, 0] == 7).all() and (wide[:, :, -1] == 7).all()
        return got

    for out, lse in both(run):
        check(out, lse, want)
    out, none = _run(d, return_lse=False)
    assert none is None
    check(out, lse, want)


@pytest.mark.parametrize("T,H,Hkv", [(8, 8, 2), (40, 8, 2), (70, 4, 1)])
def test_scales_far_apart(T, H, Hkv):
    """Pages whose scales lie at the ends of the range, in one tile."""
    d = _case(16, 128, H, Hkv, T, [600, 333], [T, T - 3], 0, 0.0, False, True,
              spread=0)
    k, v, ks, vs = d["host"]
    g = torch.Generator().manual_seed(4)
    vs = torch.exp2(torch.randint(-40, 41, vs.shape, generator=g).float())
    ks = ks * torch.exp2(torch.randint(-20, 1, ks.shape, generator=g).float())
    d["host"] = (k, v, ks, vs)
    check(*_run(d), _want(d))
    # and scales that are no powers of two
    vs = torch.rand(vs.shape, generator=g) * 0.01 + 0.003
    ks = torch.rand(ks.shape, generator=g) * 0.01 + 0.001
    d["host"] = (k, v, ks, vs)
    check(*_run(d), _want(d))


@pytest.mark.parametrize("T,H,Hkv", [(8, 8, 2), (40, 8, 2), (70, 4, 1)])
def test_long_tail_beside_a_dominant_key(T, H, Hkv):
    """Many keys of little weight each, which together weigh as much as one."""
    n = 20000
    d = _case(128, 64, H, Hkv, T, [n], [T], 0, 0.0, False, True, spread=0)
    k, v, ks, vs = d["host"]
    k = torch.zeros(k.shape)
    first = int(d["table"][0, 3])
    k[first, :, 5, 0] = 256.0
    q = torch.zeros(d["q"].shape)
    q[..., 0] = 1.0
    ks = torch.ones_like(ks)
    d["host"] = (k.to(torch.float8_e4m3fn), v, ks, vs)
    d["q"] = q.bfloat16()
    import math
    scale = math.log(n) / 256.0
    check(*_run(d, scale=scale), _want(d, scale))


@pytest.mark.parametrize("T,H,Hkv", [(4, 8, 2), (20, 8, 2), (70, 4, 1)])
def test_nan_of_unseen_tokens(T, H, Hkv):
    """NaN codes of a draft reach the rows that see it and no other; those
    behind a sequence's last token reach none."""
    lens, n_new = [150, 200], [T, T - 2]
    d = _case(64, 128, H, Hkv, T, lens, n_new, 0, 0.0, False, True, empty=0.0)
    k, v, ks, vs = d["host"]
    kb, vb = k.view(torch.uint8), v.view(torch.uint8)
    clean = _run(d)
    for b, n in enumerate(lens):  # behind the last token
        if n % 64:
            pid = int(d["table"][b, n // 64])
            kb[pid, :, n % 64:] = 0x7f
            vb[pid, :, n % 64:] = 0xff
    got = _run(d)
    assert all(torch.equal(a, b) for a, b in zip(got, clean))
    bad = 1  # a draft: its value in some dims, then its key
    for b, (n, m) in enumerate(zip(lens, n_new)):
        at = n - m + bad
        vb[int(d["table"][b, at // 64]), :, at % 64, 5:9] = 0x7f
    out, lse = (t.cpu() for t in _run(d))
    G = H // Hkv
    for b, m in enumerate(n_new):
        sees = d["bits"][b, :m, bad]
        o, c = out[b, :, :m], clean[0].cpu()[b, :, :m]
        assert o[:, sees][..., 5:9].isnan().all()
        assert torch.equal(o[:, ~sees], c[:, ~sees])
        assert torch.equal(o[:, sees][..., 9:], c[:, sees][..., 9:])
        assert torch.equal(lse[b], clean[1].cpu()[b])
    assert G * Hkv == H
    for b, (n, m) in enumerate(zip(lens, n_new)):
        at = n - m + bad
        kb[int(d["table"][b, at // 64]), :, at % 64, 3] = 0xff
    out, lse = (t.cpu() for t in _run(d))
    for b, m in enumerate(n_new):
        sees = d["bits"][b, :m, bad]
        assert out[b, :, :m][:, sees].isnan().all()
        assert lse[b, :, :m][:, sees].isnan().all()
        assert torch.equal(out[b, :, :m][:, ~sees],
                           clean[0].cpu()[b, :, :m][:, ~sees])
    assert status()[0] == 0


def test_window_and_nan_before_it():
    """A NaN value that only some rows' windows still reach."""
    T = 24
    d = _case(32, 128, 4, 1, T, [300], [T], 100, 0.0, False, True, empty=0.0)
    clean = _run(d)
    base = 300 - T
    depth = d["bits"][0].sum(-1) - 1
    at = base - 100 + 3  # seen by the rows of depth 0 .. 2
    vb = d["host"][1].view(torch.uint8)
    vb[int(d["table"][0, at // 32]), :, at % 32] = 0x7f
    out = _run(d)[0].cpu()[0]
    sees = depth + base - at < 100
    assert sees.any() and not sees.all()
    assert out[:, sees].isnan().all()
    assert torch.equal(out[:, ~sees], clean[0].cpu()[0][:, ~sees])


@pytest.mark.parametrize("T", [4, 40])
def test_bad_lengths_and_pages_are_reported(T):
    d = _case(64, 128, 8, 2, T, [300, 200, 100], [T, T, T], 0, 0.0, False,
              True)
    clean = _run(d)
    assert status()[0] == 0
    cache = bsm.KVCache(*[t.cuda() for t in d["host"]])

    def run(table=None, lens=None, n_new=None):
        out = bsm.paged_attention(
            d["q"].cuda(), cache,
            (d["table"] if table is None else table).cuda(),
            _ints(lens or d["lens"]), tree=ref.pack(d["bits"]).cuda(),
            n_new=_ints(n_new or d["n_new"]))
        st, detail = status()
        assert status()[0] == 0  # read once
        return out, st, detail

    invalid = bsm._lib.BSM_ERR_INVALID_ARG
    for n_new in ([T, T + 1, T], [T, -1, T]):
        out, st, detail = run(n_new=n_new)
        assert st == invalid and detail[1:3] == [1, -1]
        assert torch.equal(out[0][0], clean[0][0])
        assert torch.equal(out[0][2], clean[0][2])
        if n_new[1] < 0:
            assert (out[0][1] == 0).all() and (out[1][1] == -torch.inf).all()
    out, st, detail = run(lens=[300, -5, 100])
    assert st == invalid and detail[1:3] == [1, -1]
    assert (out[0][1] == 0).all() and torch.equal(out[0][2], clean[0][2])
    table = d["table"].clone()
    table[1, 0] = 10 ** 6  # its tokens count as masked
    out, st, detail = run(table=table)
    assert st == invalid and detail[1:3] == [1, 0]
    assert torch.equal(out[0][0], clean[0][0])
    assert out[0][1].isfinite().all()


@pytest.mark.parametrize("case", [CASES[1], CASES[9]])
def test_streams_and_graphs(case):
    d = _case(*case)
    want = _run(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _run(d, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    cache = bsm.KVCache(*[t.cuda() for t in d["host"]])
    t = dict(q=d["q"].cuda(), table=d["table"].cuda(), lens=_ints(d["lens"]),
             n=_ints(d["n_new"]), tree=ref.pack(d["bits"]).cuda())

    def call():
        return bsm.paged_attention(t["q"], cache, t["table"], t["lens"],
                                   tree=t["tree"], n_new=t["n"])

    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = call()
        graphs.append((graph, res))
    d["bits"] = ref.random_tree(len(d["lens"]), d["q"].shape[2], 77)
    t["tree"].copy_(ref.pack(d["bits"]))
    d["lens"] = [max(m, n - 5) for n, m in zip(d["lens"], d["n_new"])]
    t["lens"].copy_(_ints(d["lens"]))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for (graph, _), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    want = _want(d)
    for _, res in graphs:
        check(*res, want)


def test_many_sequences():
    """More sequences than a warp has lanes, more items than SMs."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 400, (90,), generator=g).tolist()
    T = 17
    n_new = [min(n, int(torch.randint(0, T + 1, (1,), generator=g)))
             for n in lens]
    d = _case(32, 64, 4, 2, T, lens, n_new, 0, 0.0, False, True)
    check(*_run(d), _want(d))


def test_a_step_of_drafts():
    """As a server uses it: prompts into the cache, drafts normalised, rotated
    by depth and appended, their attention, and the accepted ones appended in
    their place."""
    B, H, Hkv, D, T, P = 2, 8, 2, 64, 12, 32
    g = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    rope, w = bsm.Rope(64, 1e4), (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    cache = bsm.KVCache.empty(20, Hkv, P, D)
    table = torch.randperm(20, generator=g).int().view(B, 10).cuda()
    lens = torch.zeros(B, dtype=torch.int32).cuda()
    kp, vp, n0 = r(B, Hkv, 150, D), r(B, Hkv, 150, D), _ints([150, 77])
    args = dict(rope=rope, k_weight=w, eps=1e-6)
    bsm.kv_append(cache, table, lens, kp, vp, n_new=n0, **args)
    lens += n0
    bits = ref.random_tree(B, T, 5)
    pos = (lens.cpu()[:, None] + bits.sum(-1) - 1).int().cuda()
    q, k, v = r(B, H, T, D), r(B, Hkv, T, D), r(B, Hkv, T, D)
    q1, _ = bsm.norm_rope(q, rope=rope, positions=pos, q_weight=w, eps=1e-6)
    n = _ints([T, T - 4])
    bsm.kv_append(cache, table, lens, k, v, n_new=n, positions=pos, **args)
    out, lse = bsm.paged_attention(q1, cache, table, lens + n,
                                   tree=ref.pack(bits).cuda(), n_new=n)
    want = ref.attention(q1.cpu(), *[t.cpu() for t in cache._tensors],
                         table.cpu(), (lens + n).tolist(), n.tolist(), bits,
                         D ** -0.5)
    check(out, lse, want)
    # the path to the last draft is accepted: its tokens stand in a row
    path = [bits[b, m - 1].nonzero().flatten() for b, m in
            enumerate(n.tolist())]
    m = max(len(x) for x in path)
    rows = torch.zeros(B, m, dtype=torch.int64)
    for b, x in enumerate(path):
        rows[b, :len(x)] = x
    at = rows.cuda()[:, None, :, None].expand(B, Hkv, m, D)
    took = _ints([len(x) for x in path])
    bsm.kv_append(cache, table, lens, k.gather(2, at), v.gather(2, at),
                  n_new=took, **args)
    one, _ = bsm.paged_attention(
        q1.gather(2, (n - 1).long().view(B, 1, 1, 1).expand(B, H, 1, D)),
        cache, table, lens + took)
    # the same keys at the same positions, by another way through the cache:
    # a page's scale may have grown, so codes differ by their rounding
    tip = torch.stack([out[b, :, k - 1] for b, k in enumerate(n.tolist())])
    err = (one[:, :, 0] - tip).float().abs().max()
    assert float(err) <= 2.0 ** -3 * float(tip.float().abs().max())
    assert status()[0] == 0
