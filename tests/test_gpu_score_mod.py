"""Forward and backward with modified softmax scores (tanh cap, distance
bias) against fp64, under every mask kind and through every kernel
instance.

Tolerances.  The forward rounds each p to bf16 (half a step, 2^-8 relative)
and the output to bf16 (2^-8), so |error| <= 2^-8 (sum_k p |v| + |out|); the
logits and sums are f32 (cap and exponentials to a few 2^-22, the dot
product of D terms to D 2^-24 of sum |q k| scale), for which 2^-11 more of
sum p |v| is allowed.  The logsumexp has the f32 errors alone: 1e-4 relative
to max(1, |lse|).  Gradients: the element-wise bounds of the roundings that
score_mod_ref.backward derives.  (The gates of the unmodified backward's
tests, relative to the mean gradient, are derived there for smooth softmax
rows; in the peaked rows here dP - D_q cancels, and the rounding of the
output that D_q is taken from weighs more.)
"""

import math
import zlib

import numpy as np
import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import score_mod_ref as ref
from block_sparse_masked_build_gb300 import workloads as wl
from gpu_helpers import dense_device_bits

pytestmark = pytest.mark.gpu

C, L, SG, BD, DN = (bsm.MASK_CAUSAL, bsm.MASK_LOCAL, bsm.MASK_SEGMENT,
                     bsm.MASK_BAND, bsm.MASK_DENSE)
HALF = 2.0 ** -8  # bf16: half a step


def check_out(out, lse, want, lse_slack=0.0):
    o, l, spread = want
    out, lse = out.double().cpu(), lse.double().cpu()
    err = (out - o).abs()
    tol = HALF * (o.abs() + spread) * (1 + 2.0 ** -7) + 2.0 ** -11 * spread
    assert torch.isfinite(out).all()
    assert (err <= tol + 1e-30).all(), float((err - tol).max())
    dead = torch.isinf(l)
    assert torch.equal(torch.isneginf(lse), dead)
    off = (lse - l).abs()[~dead] - lse_slack
    rel = off / l.abs()[~dead].clamp(min=1.0)
    assert rel.numel() == 0 or float(rel.max()) <= 1e-4, float(rel.max())
    assert (out[dead] == 0).all()


def inputs(name, B, H, Hkv, Sq, Skv, D, sigma=1.0):
    g = torch.Generator().manual_seed(zlib.crc32(name.encode()) % 100000)
    mk = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return ((mk(B, H, Sq, D) * sigma).bfloat16(), mk(B, Hkv, Skv, D).bfloat16(),
            mk(B, Hkv, Skv, D).bfloat16(), mk(B, H, Sq, D).bfloat16())


def slopes_of(H, sign=1.0):
    return sign * torch.exp2(-8.0 * torch.arange(1, H + 1) / H)


def run(q, k, v, do, flags, window=0, seg_q=None, seg_kv=None, scale=None,
        softcap=0.0, slopes=None, dense=None, blk=128, bwd=True,
        lse_slack=0.0):
    dev = torch.device("cuda")
    scale = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    qd, kd, vd, dod = (t.to(dev) for t in (q, k, v, do))
    sq = None if seg_q is None else torch.from_numpy(seg_q).to(dev)
    sk = None if seg_kv is None else torch.from_numpy(seg_kv).to(dev)
    sl = None if slopes is None else slopes.to(dev)
    db = None if dense is None else dense_device_bits(dense)
    info = bsm.build_mask_info(flags, q.shape[0], q.shape[2], k.shape[2], blk,
                               blk, window, sq, sk, device=dev, dense_bits=db)
    kw = dict(mask_info=info, q_segment_ids=sq, kv_segment_ids=sk,
              scale=scale, softcap=softcap, alibi_slopes=sl)
    out, lse = bsm.splash_attention(qd, kd, vd, **kw)
    grads = ()
    if bwd:
        grads = bsm.splash_attention_bwd(qd, kd, vd, out, lse, dod, **kw)
    torch.cuda.synchronize()
    st, detail = bsm.bsm_device_status()
    assert st == 0, f"device status {st} {detail}"
    vis = ref.visible(flags, window, q.shape[2], k.shape[2], q.shape[0], seg_q,
                      seg_kv, dense)
    check_out(out, lse, ref.forward(q, k, v, vis, scale, softcap, slopes),
              lse_slack)
    if bwd:
        want, tol = ref.backward(q, k, v, do, vis, scale, softcap, slopes,
                                 bounds=True)
        for n, g, r, b in zip(("dq", "dk", "dv"), grads, want, tol):
            err = (g.double().cpu() - r).abs()
            assert torch.isfinite(g).all(), n
            assert (err <= b + 1e-30).all(), (n, float((err - b).max()))
    return out, lse, grads


MODS = [("cap", 8.0, 0.0), ("bias", 0.0, 1.0), ("both", 8.0, 1.0)]

CASES = [
    # name, B, H, Hkv, Sq, Skv, D, flags, window
    ("causal", 1, 2, 2, 384, 384, 128, C, 0),
    ("causal_tail_d64", 2, 1, 1, 300, 300, 64, C, 0),
    ("full_cross", 1, 2, 2, 200, 333, 128, 0, 0),
    ("full_cross_d64", 1, 2, 1, 333, 130, 64, 0, 0),
    ("local", 1, 2, 2, 700, 700, 128, C | L, 200),
    ("band", 1, 1, 1, 600, 600, 128, L | BD, 100),
    ("gqa", 1, 6, 2, 320, 320, 128, C, 0),
    ("one", 1, 2, 1, 1, 1, 128, C, 0),
    ("one_query", 2, 2, 2, 1, 77, 64, 0, 0),
]


@pytest.mark.parametrize("mod", MODS, ids=[m[0] for m in MODS])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_small(case, mod):
    name, B, H, Hkv, Sq, Skv, D, flags, window = case
    q, k, v, do = inputs(name + mod[0], B, H, Hkv, Sq, Skv, D, 4.0)
    if Skv == 1:  # dS of a lone key is a rounding error: only P and dV count
        do = torch.zeros_like(do)
    run(q, k, v, do, flags, window, softcap=mod[1],
        slopes=slopes_of(H, mod[2]) if mod[2] else None)


@pytest.mark.parametrize("mod", MODS, ids=[m[0] for m in MODS])
@pytest.mark.parametrize("kind", ["sorted", "unsorted"])
@pytest.mark.parametrize("D", [64, 128])
def test_segments(kind, D, mod):
    B, H, S = 2, 2, 520
    q, k, v, do = inputs(f"seg{kind}{D}{mod[0]}", B, H, H, S, S, D, 3.0)
    if kind == "sorted":
        seg = wl.random_segment_ids(B, S, 30, 250, 41)
    else:
        seg = np.random.default_rng(42).integers(0, 3, size=(B, S)).astype(
            np.int32)
    run(q, k, v, do, C | SG, 0, seg, seg, softcap=mod[1], blk=64,
        slopes=slopes_of(H, mod[2]) if mod[2] else None)


@pytest.mark.parametrize("mod", MODS, ids=[m[0] for m in MODS])
@pytest.mark.parametrize("per_sm", [0.3, 0.8, 1.7])
@pytest.mark.parametrize("D", [64, 128])
def test_query_tiles_per_sm(D, per_sm, mod):
    """Few 256-row units share a CTA's pipelines, more take one pipeline
    each, and above one per SM they are drawn from a counter."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    S = 400
    H = int(per_sm * sms / 2)  # two units per head
    q, k, v, do = inputs(f"units{D}{per_sm}{mod[0]}", 1, H, H, S, S, D, 3.0)
    run(q, k, v, do, C, softcap=mod[1],
        slopes=slopes_of(H, mod[2]) if mod[2] else None, bwd=False)


@pytest.mark.parametrize("mod", MODS, ids=[m[0] for m in MODS])
@pytest.mark.parametrize("per_sm", [0.1, 1.3])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing(D, per_sm, mod):
    """A band over fewer keys than queries leaves rows, and whole query
    tiles, empty; segment ids that no key has leave rows empty inside tiles
    that are not, in the one or the other half of the keys' tiles."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Sq, Skv = 640, 300
    H = max(1, int(per_sm * sms / 3))
    q, k, v, do = inputs(f"dead{D}{per_sm}{mod[0]}", 1, H, H, Sq, Skv, D, 3.0)
    sl = slopes_of(H, mod[2]) if mod[2] else None
    _, lse, _ = run(q, k, v, do, L | BD, 100, softcap=mod[1], slopes=sl,
                    bwd=False)
    assert bool(torch.isneginf(lse[..., 400:]).all())
    rng = np.random.default_rng(77)
    sq = rng.integers(0, 4, size=(1, Sq)).astype(np.int32)
    skv = np.repeat(np.array([[0, 1, 2]], np.int32), 128, axis=1)[:, :Skv]
    # unsorted: element by element
    skv_mixed = np.array([2, 0, 1], np.int32)[skv]
    for ids in (skv, skv_mixed):
        _, lse, _ = run(q, k, v, do, SG, 0, sq, np.ascontiguousarray(ids),
                        softcap=mod[1], slopes=sl, bwd=False)
        dead = torch.from_numpy(sq[0] == 3).to(lse.device)
        assert bool(torch.isneginf(lse[..., dead]).all())


@pytest.mark.parametrize("mod", MODS, ids=[m[0] for m in MODS])
def test_arbitrary_mask_with_empty_rows(mod):
    S, H = 500, 2
    q, k, v, do = inputs("dense" + mod[0], 1, H, H, S, S, 128, 3.0)
    dm = wl.random_dense_mask(S, S, 0.4, 64, 51)
    dm[40:90] = False
    out, lse, (dq, _, _) = run(
        q, k, v, do, DN, 0, dense=dm, softcap=mod[1],
        slopes=slopes_of(H, mod[2]) if mod[2] else None)
    assert (dq[:, :, 40:90] == 0).all()


@pytest.mark.parametrize("mod", MODS, ids=[m[0] for m in MODS])
def test_long_rows(mod):
    # from 4096 keys on the score warps of the two query tiles take turns
    q, k, v, do = inputs("long" + mod[0], 1, 2, 1, 4200, 4200, 128, 2.0)
    run(q, k, v, do, C, softcap=mod[1],
        slopes=slopes_of(2, mod[2]) if mod[2] else None)


@pytest.mark.parametrize("cap", [0.5, 5.0, 70.0, 1000.0, 2e4])
def test_saturated_and_loose_caps(cap):
    # scores far beyond the cap (most rows at +-cap, where dS vanishes) and
    # a cap that hardly bends them
    q, k, v, do = inputs(f"sat{cap}", 1, 2, 2, 260, 260, 128, 12.0)
    run(q, k, v, do, C, softcap=cap)


def test_scores_beyond_f32_exponentials():
    # |x| / cap in the hundreds: e^(2 x / cap) overflows to infinity, or
    # underflows to zero, and tanh is exactly +-1
    q, k, v, do = inputs("huge", 1, 1, 1, 130, 130, 64, 200.0)
    out, lse, grads = run(q, k, v, do, C, softcap=1.0, bwd=False)
    for g in grads:
        assert torch.isfinite(g).all()


@pytest.mark.parametrize("cap", [0.5, 20.0, 51.0, 53.0, 61.0, 200.0])
@pytest.mark.parametrize("kind", ["causal", "full", "far", "band"])
def test_references_of_cap_and_bias(kind, cap):
    """Small caps take the row's largest bias for the softmax's reference,
    larger ones a running maximum: saturated scores, slopes of both signs,
    rows whose nearest key is far away or that see none."""
    Sq, Skv = (700, 200) if kind == "far" else (330, 330)
    flags = {"causal": C, "band": L | BD}.get(kind, 0)
    H = 6
    q, k, v, do = inputs(f"ref{kind}{cap}", 1, H, H, Sq, Skv, 64, 6.0)
    sl = torch.tensor([0.004, 0.3, 2.0, -0.004, -0.02, 0.0])
    run(q, k, v, do, flags, 90 if kind == "band" else 0, softcap=cap,
        slopes=sl, scale=1.0 if cap < 1 else None, bwd=False)


@pytest.mark.parametrize("sign", [1.0, -0.02])
@pytest.mark.parametrize("flags", [SG, C | SG])
def test_references_with_unsorted_segments(flags, sign):
    """Rows whose nearest (farthest) key of their segment is not the nearest
    (farthest) of the mask's interval, and rows whose id no key has."""
    S, H = 400, 3
    q, k, v, do = inputs(f"refseg{flags}{sign}", 2, H, H, S, S, 64, 4.0)
    ids = np.zeros((2, S), np.int32)
    ids[:, 300:] = 1      # far from the rows that look for 0
    ids[1] = np.random.default_rng(5).integers(0, 4, S)
    ids[1, :40] = 9
    rows = ids.copy()
    rows[:, 350:] = 0
    rows[:, 380:] = 7     # no key has it
    run(q, k, v, do, flags, 0, rows, ids, softcap=30.0,
        slopes=sign * torch.tensor([0.01, 1.0, 4.0]), bwd=False)


@pytest.mark.parametrize("scale", [-0.09, 0.0, 2.0 ** -22, 2.0 ** -19, 3.0])
@pytest.mark.parametrize("D", [64, 128])
def test_bias_with_unusual_scales(D, scale):
    """A bias alone is added inside the product as slope / scale, but for
    scales that are negative or next to nothing."""
    q, k, v, do = inputs(f"scales{D}{scale}", 1, 3, 1, 300, 333, D, 0.5)
    for flags in (C, 0):
        run(q, k, v, do, flags, scale=scale, slopes=slopes_of(3))


def test_bias_of_many_heads_and_signs():
    """Every unit brings its own head's slope: far more units than SMs, steep
    and flat, rising and falling slopes next to one another."""
    H = 120
    q, k, v, do = inputs("heads", 2, H, H, 300, 300, 64, 2.0)
    sl = slopes_of(H) * torch.where(torch.arange(H) % 3 == 0, -0.1, 3.0)
    for flags in (C, 0):
        run(q, k, v, do, flags, slopes=sl, bwd=False)


@pytest.mark.parametrize("cap", [0.0, 20.0, 60.0])
@pytest.mark.parametrize("S", [200, 700])
@pytest.mark.parametrize("flags", [C, 0])
def test_one_key_that_outweighs_all(flags, S, cap):
    """With slopes this steep every other key weighs less than e^-30, so each
    row is its own key's value to the last bit: its p is not rounded.  (To
    1e-9, as the other keys' share, at most e^-30 700 |v| with |v| < 6, shows
    where a value is 0.)

    A bias alone is added to S as up to 64 slope / scale, whose sum with q.k
    the tensor core may truncate (2^-23 of it: 2^-23 64 slope in the logit);
    the rest, up to 128 slope in the row's own tile, is rounded to f32 (half
    a step: 2^-24 128 slope).  Both together are 2^-22 64 slope; at a slope of
    60 that is 9e-4, more than the 1e-4 that gentler slopes stay within."""
    H = 40
    q, k, v, _ = inputs(f"one{flags}{S}{cap}", 1, H, H, S, S, 64)
    sl = torch.full((H,), 60.0)
    out, _, _ = run(q, k, v, v, flags, softcap=cap, slopes=sl, bwd=False,
                    lse_slack=2.0 ** -22 * 64 * 60.0)
    assert bool(((out.cpu().float() - v.float()).abs() <= 1e-9).all())


def test_negative_and_zero_slopes():
    q, k, v, do = inputs("neg", 1, 2, 2, 300, 300, 128)
    run(q, k, v, do, C, slopes=torch.tensor([-0.02, 0.0]))
    run(q, k, v, do, 0, slopes=torch.tensor([-0.02, 0.0]))


def test_rising_bias_past_the_last_query():
    # a bias that grows with the distance, no mask, a ragged end: queries past
    # the last one, whose bias alone would overflow, must not reach dK and dV
    q, k, v, do = inputs("rise", 1, 1, 1, 200, 333, 128)
    run(q, k, v, do, 0, slopes=torch.tensor([-2.0]))
    q, k, v, do = inputs("rise2", 1, 1, 1, 20, 2000, 128)
    run(q, k, v, do, 0, slopes=torch.tensor([-1.0]))


@pytest.mark.parametrize("kind", ["causal", "segments", "full"])
@pytest.mark.parametrize("D", [64, 128])
def test_cut_key_walks(kind, D):
    # few keys and K/V heads under many query heads: dK and dV are summed in
    # parts, here with walks that do not divide evenly, and with part of the
    # walks empty; without the larger workspace they are summed in one
    B, H, Hkv, Sq, Skv = 1, 10, 1, 460, 300
    assert bsm.bsm_splash_bwd_mod_workspace_bytes(B, H, Hkv, Sq, Skv, D) > \
        bsm.bsm_splash_bwd_workspace_bytes(B, H, Sq, 0)
    q, k, v, do = inputs(f"cut{kind}{D}", B, H, Hkv, Sq, Skv, D, 3.0)
    sq = sk = None
    flags = 0 if kind == "full" else C
    if kind == "segments":
        flags = C | SG
        sq = wl.random_segment_ids(B, Sq, 30, 90, 5)
        sk = sq[:, :Skv].copy()
        sk[:, 128:256] = 99  # a key tile that no query sees
    _, _, grads = run(q, k, v, do, flags, 0, sq, sk, softcap=6.0,
                      slopes=slopes_of(H))
    if kind == "segments":
        assert (grads[1][:, :, 128:256] == 0).all()
        assert (grads[2][:, :, 128:256] == 0).all()


def test_cut_and_whole_walks_agree():
    B, H, Hkv, S, D = 1, 8, 1, 300, 128
    q, k, v, do = (t.cuda() for t in inputs("whole", B, H, Hkv, S, S, D, 2.0))
    info = bsm.build_mask_info(C, B, S, S)
    out, lse = bsm.splash_attention(q, k, v, mask_info=info, softcap=9.0)
    res = []
    for n in (bsm.bsm_splash_bwd_workspace_bytes(B, H, S, 0),
              bsm.bsm_splash_bwd_mod_workspace_bytes(B, H, Hkv, S, S, D)):
        ws = torch.full((n,), 0xff, dtype=torch.uint8).cuda()  # NaN leftovers
        g = [torch.full_like(t, float("nan")) for t in (q, k, v)]
        bsm.bsm_splash_bwd(q, k, v, out, lse, do, info, None, None,
                           1 / math.sqrt(D), 0, *g, workspace=ws, softcap=9.0)
        res.append(g)
    assert torch.equal(res[0][0], res[1][0])
    for a, b in zip(res[0][1:], res[1][1:]):
        # equal f32 sums up to their order, then one rounding to bf16 each
        a, b = a.double(), b.double()
        assert ((a - b).abs() <= HALF * 2.1 * a.abs() + 1e-5 *
                a.abs().amax()).all()


def test_no_modification_is_the_unmodified_call():
    q, k, v, do = (t.cuda() for t in inputs("none", 1, 2, 2, 300, 300, 128))
    a = bsm.splash_attention(q, k, v)
    b = bsm.splash_attention(q, k, v, softcap=0.0, alibi_slopes=None)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = bsm.splash_attention_bwd(q, k, v, *a, do)
    gb = bsm.splash_attention_bwd(q, k, v, *a, do, softcap=0.0)
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))


def test_operands_are_checked():
    q = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16).cuda()
    info = bsm.build_mask_info(C, 1, 64, 64)
    lse = torch.zeros(1, 2, 64).cuda()
    seg = torch.zeros(1, 64, dtype=torch.int32).cuda()
    for bad in ((q.half(), q, q), (q, q.cpu(), q), (q, q, q.float()),
                (q, q, q[:, :, :32]), (q, q[..., :32], q[..., :32])):
        with pytest.raises(ValueError):
            bsm.splash_attention(*bad, mask_info=info, softcap=5.0)
        with pytest.raises(ValueError):
            bsm.splash_attention_bwd(*bad, q, lse, q, mask_info=info,
                                     softcap=5.0)
    for kw in (dict(out=q.float()), dict(out=q[:, :1]), dict(lse=lse.double()),
               dict(lse=lse[:, :, ::2])):
        with pytest.raises(ValueError):
            bsm.splash_attention(q, q, q, mask_info=info, **kw)
    for ids in (seg.long(), seg.cpu(), seg[:, :32]):
        with pytest.raises((ValueError, bsm.BsmError)):
            bsm.splash_attention(q, q, q, q_segment_ids=ids,
                                 kv_segment_ids=ids, mask_info=info)
    with pytest.raises(ValueError):
        bsm.splash_attention_bwd(q, q, q, q, lse, q.cpu(), mask_info=info)


def test_strided_and_host_tensors():
    B, H, S, D = 2, 2, 200, 64
    q, k, v, do = inputs("strided", B, H, H, S, S, D, 3.0)
    sl = slopes_of(H)
    kw = dict(softcap=6.0)
    dev = [t.cuda() for t in (q, k, v)]
    want, wlse = bsm.splash_attention(*dev, alibi_slopes=sl.cuda(), **kw)
    bshd = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in dev]
    out, lse = bsm.splash_attention(*bshd, alibi_slopes=sl.cuda(), **kw)
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    # host tensors: copied in, computed on the device, copied back
    out, lse = bsm.splash_attention(q, k, v, alibi_slopes=sl, **kw)
    assert out.device.type == "cpu"
    assert torch.equal(out, want.cpu()) and torch.equal(lse, wlse.cpu())
    with pytest.raises(ValueError, match="alibi_slopes"):
        bsm.splash_attention(*dev, alibi_slopes=sl, **kw)


def test_nan_scores_reach_their_rows_only():
    q, k, v, _ = inputs("nan", 1, 1, 1, 256, 256, 128)
    q[0, 0, 17, 3] = float("nan")
    out, _ = bsm.splash_attention(q.cuda(), k.cuda(), v.cuda(), softcap=5.0)
    bad = torch.isnan(out.float()).any(-1)[0, 0].cpu()
    assert bad[17] and int(bad.sum()) == 1


def test_graph_replay_and_side_stream():
    B, H, S, D = 1, 2, 700, 128
    a = [t.cuda() for t in inputs("graph_a", B, H, H, S, S, D, 3.0)]
    b = [t.cuda() for t in inputs("graph_b", B, H, H, S, S, D, 3.0)]
    sl = slopes_of(H).cuda()
    info = bsm.build_mask_info(C, B, S, S)
    kw = dict(mask_info=info, softcap=6.0, alibi_slopes=sl)

    def step(q, k, v, do):
        out, lse = bsm.splash_attention(q, k, v, **kw)
        return (out, lse) + tuple(bsm.splash_attention_bwd(q, k, v, out, lse,
                                                           do, **kw))

    want = [[t.clone() for t in step(*x)] for x in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(*a)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want[0]))
    buf = [t.clone() for t in a]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(*buf)
    for x, w in ((b, want[1]), (a, want[0]), (b, want[1])):
        for t, s in zip(buf, x):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, y) for g, y in zip(res, w))


def test_gradients_against_differences():
    # central differences of the fp64 forward along the reference gradient
    # (unit length): the kernel's component there is off by at most the sum
    # of the element bounds weighted with the direction
    B, H, Hkv, S, D = 1, 4, 2, 90, 64
    q, k, v, do = inputs("diff", B, H, Hkv, S, S, D, 3.0)
    sl, cap, scale = slopes_of(H), 4.0, 1 / 8
    _, _, grads = run(q, k, v, do, C, softcap=cap, slopes=sl, scale=scale)
    vis = ref.visible(C, 0, S, S, B)
    want, tol = ref.backward(q, k, v, do, vis, scale, cap, sl, bounds=True)
    for n in range(3):
        u = want[n] / want[n].norm()
        f = []
        for h in (1e-4, -1e-4):
            x = [q.double(), k.double(), v.double()]
            x[n] = x[n] + h * u
            f.append((ref.forward(*x, vis, scale, cap, sl)[0]
                      * do.double()).sum())
        diff = float(f[0] - f[1]) / 2e-4
        got = float((grads[n].double().cpu() * u).sum())
        room = float((tol[n] * u.abs()).sum()) + 1e-6 * abs(diff)
        # (worst-case bounds add up over the elements, to 7.5 % of the
        # derivative for dq and 12.3 % for dk from the reference's values
        # alone; a wrong factor of a quarter or more cannot pass)
        assert abs(got - diff) <= room < 0.25 * abs(diff)
