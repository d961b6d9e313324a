"""The two ways from Python into the library -- the module that calls it
straight from tensors, and ctypes -- give the same bits and the same errors."""

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import kv_cache_ref as ref
from block_sparse_masked_build_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture
def both(monkeypatch):
    def run(f):
        assert bsm.api._fast()
        a = f()
        with monkeypatch.context() as m:
            m.setattr(bsm.api, "_fast", lambda: False)
            b = f()
        torch.cuda.synchronize()
        return a, b
    return run


def same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        if x is None or y is None:
            assert x is None and y is None
        else:
            assert x.dtype == y.dtype and x.shape == y.shape
            assert x.stride() == y.stride()
            assert torch.equal(x, y)


@pytest.mark.parametrize("kind", ["causal", "segments", "dense", "pointwise"])
def test_splash(both, kind):
    B, H, Hkv, S, D = 2, 4, 2, 300, 64
    g = torch.Generator().manual_seed(1)
    mk = lambda h: torch.randn(B, S, h, D, generator=g).bfloat16().cuda()  # noqa
    q, k, v, do = (mk(h).transpose(1, 2) for h in (H, Hkv, Hkv, H))
    seg = torch.from_numpy(wl.random_segment_ids(B, S, 20, 90, 3)).cuda()
    sl = torch.full((H,), 0.1).cuda()
    kw = dict(scale=0.1)
    if kind == "segments":
        kw.update(mask_flags=bsm.MASK_CAUSAL | bsm.MASK_SEGMENT,
                  q_segment_ids=seg, kv_segment_ids=seg, softcap=5.0)
    elif kind == "dense":
        dm = torch.from_numpy(wl.random_dense_mask(S, S, 0.4, 64, 5)).cuda()
        kw.update(mask_flags=bsm.MASK_DENSE, dense_mask=dm, alibi_slopes=sl)
    elif kind == "pointwise":
        kw.update(score=bsm.SCORE_POINTWISE)
    a, b = both(lambda: bsm.splash_attention(q, k, v, **kw))
    same(a, b)
    ga, gb = both(lambda: bsm.splash_attention_bwd(q, k, v, *a, do, **kw))
    same(ga, gb)
    out = torch.empty_like(q)
    lse = torch.empty(B, H, S).cuda()
    for got, l in both(lambda: bsm.splash_attention(q, k, v, out=out, lse=lse,
                                                    **kw)):
        assert got is out and torch.equal(out, a[0])
        assert l is (None if kind == "pointwise" else lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for r in both(lambda: bsm.splash_attention(q, k, v, stream=s, **kw)):
        s.synchronize()
        same(r, a)


@pytest.mark.parametrize("handle", [False, True])
def test_side_stream_beside_a_busy_one(both, handle):
    """Scratch and mask infos of calls on another stream are not given out
    again on the caller's before that stream has run the calls."""
    B, H, S, D = 1, 4, 700, 64
    g = torch.Generator().manual_seed(6)
    q, k, v, do = (torch.randn(B, H, S, D, generator=g).bfloat16().cuda()
                   for _ in range(4))
    kw = dict(mask_flags=bsm.MASK_CAUSAL, softcap=9.0)
    out, lse = bsm.splash_attention(q, k, v, **kw)
    want = (out, lse) + tuple(
        bsm.splash_attention_bwd(q, k, v, out, lse, do, **kw))
    sizes = {B * H * S * 4, B * H * S * 64, 1 << 12, 1 << 14, 1 << 16}

    def run():
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        s = side.cuda_stream if handle else side
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        got = []
        for _ in range(10):
            o, l = bsm.splash_attention(q, k, v, stream=s, **kw)
            got.append((o, l) + tuple(bsm.splash_attention_bwd(
                q, k, v, o, l, do, stream=s, **kw)))
            for n in sizes:  # would take memory freed too early, and spoil it
                for _ in range(4):
                    torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        side.synchronize()
        return [t for r in got for t in r]

    for r in both(run):
        same(r, list(want) * 10)


def test_host_tensors_on_a_side_stream(both):
    B, H, S, D = 1, 2, 200, 64
    g = torch.Generator().manual_seed(7)
    q, k, v = (torch.randn(B, H, S, D, generator=g).bfloat16()
               for _ in range(3))
    want = bsm.splash_attention(q.cuda(), k.cuda(), v.cuda(), softcap=9.0)
    side = torch.cuda.Stream()
    for r in both(lambda: bsm.splash_attention(q, k, v, softcap=9.0,
                                               stream=side)):
        same([t.cuda() for t in r], want)


def test_mask_info(both):
    a, b = both(lambda: bsm.build_mask_info(
        bsm.MASK_CAUSAL | bsm.MASK_LOCAL, 1, 700, 500, 64, 128, window=90))
    assert torch.equal(a.block_mask, b.block_mask)
    assert torch.equal(a.data_next, b.data_next)
    assert torch.equal(a.super_order, b.super_order)
    for bad in (dict(block_q=48), dict(window=0)):
        kw = dict(flags=bsm.MASK_LOCAL, B=1, Sq=64, Skv=64, window=3)
        kw.update(bad)
        text = []

        def call():
            with pytest.raises(bsm.BsmError) as e:
                bsm.build_mask_info(**kw)
            text.append(str(e.value))

        both(call)
        assert text[0] == text[1]


def test_cache(both):
    lens, page, D, Hkv, H = [30, 64], 16, 64, 2, 6
    host = ref.random_cache(14, Hkv, page, D, 3)
    table = ref.random_table([n + 3 for n in lens], page, 6, 14, 4).cuda()
    g = torch.Generator().manual_seed(2)
    new = [torch.randn(2, Hkv, 3, D, generator=g).bfloat16().cuda()
           for _ in range(2)]
    q = torch.randn(2, H, 3, D, generator=g).bfloat16().cuda()
    li = torch.tensor(lens, dtype=torch.int32).cuda()

    def run():
        c = bsm.KVCache(*[t.cuda() for t in host])
        bsm.kv_append(c, table, li, *new)
        r = bsm.paged_attention(q, c, table, li + 3, window=40, softcap=7.0)
        return r + (c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8),
                    c.k_scale, c.v_scale)

    same(*both(run))


def test_errors_are_the_same(both):
    q = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16).cuda()
    info = bsm.build_mask_info(bsm.MASK_CAUSAL, 1, 64, 64)
    wide = torch.zeros(1, 2, 64, 128, dtype=torch.bfloat16).cuda()
    calls = [
        lambda: bsm.splash_attention(q, q, q, softcap=-1.0),
        lambda: bsm.splash_attention(q, q, q, alibi_slopes=torch.zeros(2)),
        lambda: bsm.splash_attention(q, q, q, softcap=3.0,
                                     score=bsm.SCORE_POINTWISE),
        lambda: bsm.splash_attention(*[q[..., :32]] * 3),
        lambda: bsm.splash_attention(*[wide[..., ::2]] * 3, mask_info=info),
        lambda: bsm.splash_attention_bwd(q, q, q, q, None, q),
    ]
    for f in calls:
        seen = []

        def call():
            with pytest.raises((bsm.BsmError, ValueError)) as e:
                f()
            seen.append((type(e.value), str(e.value)))

        both(call)
        assert seen[0] == seen[1]
