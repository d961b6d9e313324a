"""The cache's append with keys normalised and rotated on the way, against
fp64.

A code is the rotated key rounded to e4m3 once: half a step (2^-4 of a normal
value, 2^-10 of the scale below that) from the exact key, plus what f32 costs
before it, 2^-16 of the element's size (see test_gpu_norm_rope).  A scale is
exact, as no case's largest magnitude is within 2^-14 of a border.  Values are
as the plain append leaves them.
"""

import numpy as np
import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import kv_cache_ref as cref
import rope_ref as ref
from test_gpu_binding import both  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

EPS = 1e-5

# page, D, Hkv, T, lens, n_new, dim, interleaved, axes, norm, weight
CASES = [
    (64, 128, 2, 1, [0, 1, 63, 64, 100], [1, 1, 1, 1, 0], 128, False, 1, True,
     torch.bfloat16),
    (16, 64, 3, 5, [0, 13, 16, 30], [5, 5, 0, 3], 32, True, 1, True,
     torch.float32),
    (32, 128, 1, 200, [0, 31, 7], [200, 33, 1], 112, False, 3, False, None),
    (128, 128, 2, 300, [5, 0], [300, 129], 64, True, 2, True, None),
    (128, 64, 1, 17, [120], [17], 48, False, 1, True, torch.float32),
    (16, 128, 2, 40, [3, 90], [40, 37], 0, False, 1, True, torch.bfloat16),
    (32, 64, 5, 33, [0, 2], [33, 30], 64, False, 1, False, None),
    (64, 64, 2, 64, [0, 64], [64, 1], 64, True, 1, False, None),
]


def _case(page, D, Hkv, T, lens, n_new, dim, inter, axes, norm, wtype, seed=0,
          given=True):
    B = len(lens)
    g = torch.Generator().manual_seed(seed + 50)
    width = max((a + n + page - 1) // page for a, n in zip(lens, n_new)) + 1
    total = sum((a + n + page - 1) // page for a, n in zip(lens, n_new)) + 2
    host = cref.random_cache(total, Hkv, page, D, seed)
    table = cref.random_table([a + n for a, n in zip(lens, n_new)], page,
                              width, total, seed)
    new = [torch.randn(B, Hkv, T, D, generator=g).bfloat16() for _ in range(2)]
    rope, pos, angle = None, None, None
    if dim:
        axis = [i % axes for i in range(dim // 2)]
        rope = bsm.Rope(dim, 1e4, axes=axis if axes > 1 else None,
                        interleaved=inter)
        at = torch.tensor(lens)[:, None] + torch.arange(T)
        pos = torch.randint(0, 30000, (axes, B, T), generator=g) if given \
            else at.expand(axes, B, T)
        angle = ref.angles(pos, ref.frequencies(dim, 1e4), axis)
        pos = pos.int().cuda() if given else None
    w = None if wtype is None else \
        (1 + 0.2 * torch.randn(D, generator=g)).to(wtype)
    k, size = ref.forward(new[0], w, EPS if norm else None, angle, inter)
    args = dict(rope=rope, positions=pos, eps=EPS if norm else None,
                k_weight=None if w is None else w.cuda())
    return host, table, new, k, size, args


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_append(both, case, given):  # noqa: F811
    page, D, Hkv, T, lens, n_new = case[:6]
    host, table, new, k, size, args = _case(*case, given=given)
    ints = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731

    def run():
        cache = bsm.KVCache(*[t.cuda() for t in host])
        bsm.kv_append(cache, table.cuda(), ints(lens), new[0].cuda(),
                      new[1].cuda(), n_new=ints(n_new), **args)
        assert bsm.bsm_device_status()[0] == 0
        return cache

    want_v, want_vs = cref.append(host[1], host[3], table, lens, new[1], n_new)
    want_k, want_ks = cref.append(host[0], host[2], table, lens, k, n_new)
    for cache in both(run):
        np.testing.assert_array_equal(cref.decode(cache.v_pages.cpu()), want_v)
        np.testing.assert_array_equal(cache.v_scale.double().cpu().numpy(),
                                      want_vs)
        ks = cache.k_scale.double().cpu()
        np.testing.assert_array_equal(ks.numpy(), want_ks)
        got = torch.from_numpy(cref.decode(cache.k_pages.cpu()))
        fresh = torch.zeros(got.shape[0], page, dtype=torch.bool)
        for b, (a, n) in enumerate(zip(lens, n_new)):
            for t in range(n):
                pid, at = int(table[b, (a + t) // page]), (a + t) % page
                fresh[pid, at] = True
                x, s = k[b, :, t], ks[pid][:, None]
                err = (got[pid, :, at] * s - x).abs()
                tol = torch.maximum(x.abs() * 2.0 ** -4, s * 2.0 ** -10) \
                    * (1 + 2.0 ** -10) + 2.0 ** -16 * size[b, :, t]
                assert bool((err <= tol).all()), (b, t)
        # tokens that were there: rounded again where a scale grew, exactly
        old = ~fresh[:, None, :, None].expand(got.shape)
        np.testing.assert_array_equal(got[old].numpy(),
                                      torch.from_numpy(want_k)[old].numpy())


def test_rotation_alone_matches_rotated_keys_in_scale():
    """Appending keys that norm_rope has turned (and rounded to bf16) gives
    codes at most one step away."""
    host, table, new, _, _, args = _case(*CASES[3])
    lens = torch.tensor(CASES[3][4], dtype=torch.int32).cuda()
    n = torch.tensor(CASES[3][5], dtype=torch.int32).cuda()
    a = bsm.KVCache(*[t.cuda() for t in host])
    b = bsm.KVCache(*[t.cuda() for t in host])
    bsm.kv_append(a, table.cuda(), lens, new[0].cuda(), new[1].cuda(),
                  n_new=n, **args)
    q = torch.empty(2, 0, 300, 128, dtype=torch.bfloat16, device="cuda")
    _, k = bsm.norm_rope(q, new[0].cuda(), **args)
    bsm.kv_append(b, table.cuda(), lens, k, new[1].cuda(), n_new=n)
    assert torch.equal(a.k_scale, b.k_scale)
    x, y = (c.k_pages.float() * c.k_scale[:, :, None, None] for c in (a, b))
    step = torch.maximum(x.abs() * 2.0 ** -3, a.k_scale[:, :, None, None]
                         * 2.0 ** -9)
    assert bool(((x - y).abs() <= step * 1.001).all())
    assert float((x != y).float().mean()) < 0.1


def test_nothing_else_is_written_and_bad_sequences_are_skipped():
    page, D, Hkv = 32, 64, 2
    host = cref.random_cache(8, Hkv, page, D, 3)
    cache = bsm.KVCache(*[t.cuda() for t in host])
    table = torch.tensor([[0, 1], [2, 99], [3, 4], [5, 6]],
                         dtype=torch.int32).cuda()
    lens = torch.tensor([10, 20, -1, 60], dtype=torch.int32).cuda()
    n_new = torch.tensor([5, 20, 3, 20], dtype=torch.int32).cuda()
    k, v = (torch.randn(4, Hkv, 20, D).bfloat16().cuda() for _ in range(2))
    bsm.kv_append(cache, table, lens, k, v, n_new=n_new, rope=bsm.Rope(64),
                  eps=EPS)
    st, detail = bsm.bsm_device_status()
    assert st == bsm._lib.BSM_ERR_INVALID_ARG and detail[1] in (1, 2, 3)
    assert bsm.bsm_device_status()[0] == 0
    got = cache.k_pages.view(torch.uint8).cpu()
    was = host[0].view(torch.uint8)
    changed = (got != was).any(-1).any(1)  # [page, token]
    want = torch.zeros_like(changed)
    want[0, 10:15] = True
    want[2, 20:] = True
    # (tokens of a page whose scale grew are rounded again)
    want[0, :10] |= changed[0, :10]
    want[2, :20] |= changed[2, :20]
    assert torch.equal(changed, want)


def test_captured():
    host, table, new, k, size, args = _case(*CASES[1])
    page, D, Hkv, T, lens, n_new = CASES[1][:6]
    cache = bsm.KVCache(*[t.cuda() for t in host])
    dev = dict(table=table.cuda(), k=new[0].cuda(), v=new[1].cuda(),
               n=torch.zeros(len(lens), dtype=torch.int32).cuda(),
               lens=torch.tensor(lens, dtype=torch.int32).cuda())

    def call(c):
        bsm.kv_append(c, dev["table"], dev["lens"], dev["k"], dev["v"],
                      n_new=dev["n"], **args)

    call(cache)  # nothing new: nothing written
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(cache)
    assert torch.equal(cache.k_pages.view(torch.uint8).cpu(),
                       host[0].view(torch.uint8))
    dev["n"].copy_(torch.tensor(n_new))
    graph.replay()
    other = bsm.KVCache(*[t.cuda() for t in host])
    call(other)
    for a, b in zip(cache._tensors, other._tensors):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
