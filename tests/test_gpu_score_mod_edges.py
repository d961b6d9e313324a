"""Modified softmax scores at their edges.  Tolerances as in
test_gpu_score_mod."""

import math

import numpy as np
import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import score_mod_ref as ref
from gpu_helpers import dense_device_bits
from test_gpu_score_mod import (BD, C, DN, HALF, L, MODS, SG, check_out,
                                inputs, run, slopes_of)

pytestmark = pytest.mark.gpu


def _masks(S):
    """name -> (flags, window, segment ids, dense mask, keys for NaN: next to
    one that a row sees without them)"""
    i = np.arange(S)
    mixed = (i % 2)[None].astype(np.int32)  # neighbours never see each other
    return {
        "causal": (C, 0, None, None, [79]),
        "local": (C | L, 40, None, None, [79, 200]),
        "band": (L | BD, 40, None, None, [79, 200]),
        "mixed_ids": (SG, 0, mixed, None, [133, 201]),
        "dense": (DN, 0, None,
                  (i[None, :] <= i[:, None]) & (i[None, :] % 5 != 1)
                  | (i[None, :] == i[:, None]), [79]),
    }


@pytest.mark.parametrize("cap,mod", [  # cap: times the modification's
    (c, m) for m in MODS for c in ((1.0, 500.0) if m[1] else (1.0,))],
    ids=lambda x: x[0] if isinstance(x, tuple) else str(x))
@pytest.mark.parametrize("kind", list(_masks(1)))
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_in_keys_that_a_row_does_not_see(D, many, kind, cap, mod):
    """Keys of NaN leave the rows that do not see them as they are, the
    neighbouring columns' among them; those that do become NaN."""
    S = 300
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    H = sms // 2 + 4 if many else 2  # two 256-row units per head
    flags, window, seg, dense, bad = _masks(S)[kind]
    q, k, v, _ = inputs(f"nan{D}{kind}{mod[0]}", 1, H, H, S, S, D, 9.0)
    slopes = slopes_of(H, mod[2]) if mod[2] else None
    vis = ref.visible(flags, window, S, S, 1, seg, seg, dense)
    hit = vis[0][:, bad].any(1)
    assert bool(hit.any()) and not bool(hit.all())
    softcap, scale = mod[1] * cap, 1 / math.sqrt(D)
    want = ref.forward(q, k, v, vis, scale, softcap, slopes)
    k[:, :, bad] = float("nan")
    ids = None if seg is None else torch.from_numpy(seg).cuda()
    bits = None if dense is None else dense_device_bits(dense)
    info = bsm.build_mask_info(flags, 1, S, S, 128, 128, window, ids, ids,
                               dense_bits=bits)
    out, lse = bsm.splash_attention(
        q.cuda(), k.cuda(), v.cuda(), mask_info=info, q_segment_ids=ids,
        kv_segment_ids=ids, softcap=softcap,
        alibi_slopes=None if slopes is None else slopes.cuda())
    assert bsm.bsm_device_status()[0] == 0
    out, lse = out.cpu(), lse.cpu()
    check_out(out[:, :, ~hit], lse[:, :, ~hit],
              [x[:, :, ~hit] for x in want])
    assert bool(torch.isnan(out[:, :, hit].float()).all())


@pytest.mark.parametrize("mod", MODS, ids=[m[0] for m in MODS])
@pytest.mark.parametrize("kind", ["causal", "dense"])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_with_nan_have_a_nan_logsumexp(D, kind, mod):
    # (-inf would say that the row sees nothing)
    S, H = 300, 3
    flags, window, _, dense, _ = _masks(S)[kind]
    q, k, v, _ = inputs(f"nanlse{D}{kind}{mod[0]}", 1, H, 1, S, S, D, 3.0)
    q[:, :, 140] = float("nan")
    bits = None if dense is None else dense_device_bits(dense)
    info = bsm.build_mask_info(flags, 1, S, S, dense_bits=bits)
    out, lse = bsm.splash_attention(
        q.cuda(), k.cuda(), v.cuda(), mask_info=info, softcap=mod[1],
        alibi_slopes=slopes_of(H).cuda() if mod[2] else None)
    want = torch.zeros(S, dtype=torch.bool)
    want[140] = True
    assert torch.equal(torch.isnan(out.float()).any(-1).cpu(),
                       want.expand(1, H, S))
    assert torch.equal(torch.isnan(lse).cpu(), want.expand(1, H, S))


@pytest.mark.parametrize("mod", MODS + [("none", 0.0, 0.0)],
                         ids=[m[0] for m in MODS] + ["none"])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_in_queries_that_a_key_does_not_serve(D, H, Hkv, mod):
    """A query of NaN leaves dV of the keys that it does not see as it is:
    there its weight is 0 and its gradient finite."""
    S, window = 300, 41
    q, k, v, do = inputs(f"nanq{D}{H}{mod[0]}", 1, H, Hkv, S, S, D, 9.0)
    bad = torch.tensor([77, 200, 255])
    slopes = slopes_of(H, mod[2]) if mod[2] else None
    vis = ref.visible(C | L, window, S, S, 1)
    hit = vis[0][bad].any(0)
    scale = 1 / math.sqrt(D)
    want, tol = ref.backward(q, k, v, do, vis, scale, mod[1], slopes,
                             bounds=True)
    q[:, :, bad] = float("nan")
    kw = dict(mask_info=bsm.build_mask_info(C | L, 1, S, S, window=window),
              softcap=mod[1],
              alibi_slopes=None if slopes is None else slopes.cuda())
    dev = [t.cuda() for t in (q, k, v)]
    out, lse = bsm.splash_attention(*dev, **kw)
    _, _, dv = bsm.splash_attention_bwd(*dev, out, lse, do.cuda(), **kw)
    assert bsm.bsm_device_status()[0] == 0
    err = (dv.double().cpu() - want[2]).abs()[:, :, ~hit]
    assert (err <= tol[2][:, :, ~hit] + 1e-30).all()  # (false for NaN)


@pytest.mark.parametrize("mod", [m for m in MODS if m[1]],
                         ids=[m[0] for m in MODS if m[1]])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_gradients_of_scores_beyond_f32_exponentials(D, H, Hkv, mod):
    # |x| / cap in the hundreds: e^(-2 |x| / cap) underflows, tanh is +-1 and
    # its derivative 0, so dQ and dK nearly vanish and dV does not
    q, k, v, do = inputs(f"hugebwd{D}{H}{mod[0]}", 1, H, Hkv, 130, 130, D,
                         200.0)
    _, _, grads = run(q, k, v, do, C, softcap=1.0,
                      slopes=slopes_of(H, 1.0) if mod[2] else None)
    assert len(grads) == 3 and bool((grads[2] != 0).any())


@pytest.mark.parametrize("D", [64, 128])
def test_one_key_that_outweighs_all_under_an_arbitrary_mask(D):
    """Logits of 42 to 47 at a row's own key and 17 or more below that
    elsewhere: the row is its own key's value to the last bit, as with a
    running maximum its p is 1 and not rounded, wherever v is not so small
    that the others show in it (`far` is the exact result's distance from v).
    A p rounded to bf16 under a sum that is not moves many elements by a
    step."""
    S, H = 100, 4
    g = torch.Generator().manual_seed(D)
    sign = torch.randint(0, 2, (1, H, S, D), generator=g) * 2.0 - 1.0
    q = (sign * torch.linspace(5.0, 6.0, S).view(1, 1, S, 1)
         * math.sqrt(128 / D)).bfloat16()
    k, v = sign.bfloat16(), torch.randn(1, H, S, D, generator=g).bfloat16()
    i = np.arange(S)
    dense = (i[None, :] * 7 + i[:, None] * 3) % 4 != 0
    dense |= i[None, :] == i[:, None]
    vis = ref.visible(DN, 0, S, S, 1, dense=dense)
    scale = 1 / math.sqrt(D)
    want = ref.forward(q, k, v, vis, scale, 55.0)
    far = float((want[0] - v.double()).abs().max())
    assert far < 1e-4
    info = bsm.build_mask_info(DN, 1, S, S,
                               dense_bits=dense_device_bits(dense))
    out, lse = bsm.splash_attention(q.cuda(), k.cuda(), v.cuda(),
                                    mask_info=info, softcap=55.0)
    check_out(out, lse, want)
    # where v is not so small that the others show in its last bit
    clear = v.float().abs() > 4 * far / HALF
    assert bool(clear.float().mean() > 0.9)
    assert torch.equal(out.cpu()[clear], v[clear])


@pytest.mark.parametrize("slope", [0.02, -0.002])
@pytest.mark.parametrize("flags", [SG, C | SG])
@pytest.mark.parametrize("rows", ["none", "third", "few"])
def test_references_with_absent_segments(rows, flags, slope):
    """Unsorted ids over many key tiles, rows whose id no key has: all of
    them, every third, those of one warp."""
    S, H = 1500, 2
    q, k, v, _ = inputs(f"absent{rows}{flags}{slope}", 1, H, H, S, S, 64, 4.0)
    rng = np.random.default_rng(11)
    ids = rng.integers(0, 40, (1, S)).astype(np.int32)
    want = ids.copy()
    if rows == "none":
        want[:] = 77
    elif rows == "third":
        want[:, ::3] = 77
    else:
        want[:, 700:720] = 77
    run(q, k, v, v, flags, 0, want, ids, softcap=30.0, bwd=False,
        slopes=slope * torch.tensor([1.0, 8.0]))


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("slope", [4.0, 0.05, -0.05])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_whose_keys_lie_in_one_far_tile(D, slope, many):
    """Unsorted ids; a row's keys all in one KV tile far from it, which one of
    two pipelines sharing the query tile has, while the other sees none of
    them and all around the row are keys of another segment."""
    S = 512
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    H = sms // 2 + 4 if many else 2
    q, k, v, _ = inputs(f"far{D}{slope}", 1, H, H, S, S, D, 4.0)
    ids = (np.arange(S, dtype=np.int32) % 2)[None].copy()
    rows = ids.copy()
    for j, tile in enumerate((0, 1, 2, 3)):
        ids[0, 128 * tile + 5:128 * tile + 40:3] = 10 + j
    rows[0, 3::5] = 10
    rows[0, 4::5] = 11
    rows[0, 7::10] = 12
    rows[0, 9::10] = 13
    run(q, k, v, v, SG, 0, rows, ids, softcap=30.0, bwd=False,
        slopes=torch.full((H,), slope))


@pytest.mark.parametrize("share", [0.5, 1.0])
def test_absent_segments_cost_no_walk_over_the_keys(share):
    """Rows whose id no key has: a bias beside the cap needs the distance of
    each row's nearest key, which is looked for in the unit's tiles alone.
    (A walk over all keys took 5 to 80 times the cap's own time.)"""
    S, H, D = 16384, 4, 64
    q, k, v, _ = (t.cuda() for t in inputs("walk", 1, H, H, S, S, D))
    g = torch.Generator().manual_seed(3)
    ids = torch.randint(0, 4, (1, S), generator=g).int()
    rows = torch.where(torch.rand(1, S, generator=g) < share, 9, ids).int()
    ids, rows = ids.cuda(), rows.cuda()
    info = bsm.build_mask_info(C | SG, 1, S, S, q_segment_ids=rows,
                               kv_segment_ids=ids)
    kw = dict(mask_info=info, q_segment_ids=rows, kv_segment_ids=ids,
              softcap=30.0)

    def time(**more):
        best = math.inf
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            bsm.splash_attention(q, k, v, **kw, **more)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    alone = time()
    both = time(alibi_slopes=torch.full((H,), 0.02).cuda())
    assert both <= 4 * alone + 0.1, (alone, both)
