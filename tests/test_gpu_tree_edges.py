"""Attention of drafted tokens on the GPU where warps and tiles are not full
and their lanes have different things to do, against fp64 (tolerances as in
test_gpu_tree.py)."""

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
from test_gpu_kv_cache import check, status
from test_gpu_tree import _case, _run, _want

pytestmark = pytest.mark.gpu

# D, H, Hkv, T, lens, n_new, window, softcap, bias: 17, 33, 100 and 77 rows (one
# tile), 129, 150 and 290 (two), 9 and 15 (the kernel of few rows); whole items
# and ones cut across CTAs
ODD = [
    (128, 1, 1, 17, [300, 17], [17, 11], 0, 0.0, False),
    (64, 3, 1, 11, [131, 500], [11, 10], 40, 0.0, True),
    (128, 4, 1, 25, [700, 300, 25], [25, 7, 25], 100, 0.0, False),
    (128, 7, 1, 11, [5000], [11], 0, 30.0, True),
    (64, 3, 1, 43, [400, 43], [43, 42], 0, 50.0, False),
    (128, 3, 1, 50, [3000, 77], [50, 31], 60, 0.0, True),
    (64, 10, 2, 58, [350, 160], [58, 3], 0, 0.0, False),
    (128, 3, 1, 3, [400, 50], [3, 2], 20, 0.0, True),
    (64, 10, 2, 3, [300, 9], [3, 1], 0, 20.0, False),
]


def _same(got, want):
    """check(), NaN where the reference has NaN and nowhere else."""
    out, lse = (t.cpu() for t in got)
    nan, nan_lse = want[0].isnan(), want[1].isnan()
    assert torch.equal(out.isnan(), nan) and torch.equal(lse.isnan(), nan_lse)
    assert not nan.all()
    check(out.masked_fill(nan, 0), lse.masked_fill(nan_lse, 0),
          (want[0].masked_fill(nan, 0), want[1].masked_fill(nan_lse, 0),
           want[2].masked_fill(nan, 0)))


@pytest.mark.parametrize("scale", [None, -0.07])
@pytest.mark.parametrize("case", ODD)
def test_rows_that_fill_no_warp(case, scale):
    """NaN values that some rows see, in a draft and ahead of the drafts, beside
    rows that are empty or not there; the same bits from each call."""
    D, H, Hkv, T, lens, n_new, *mod = case
    d = _case(32, D, H, Hkv, T, lens, n_new, *mod, True, empty=0.2)
    first = _run(d, scale=scale)
    _same(first, _want(d, scale))
    assert all(torch.equal(a, b) for a, b in zip(first, _run(d, scale=scale)))
    vb = d["host"][1].view(torch.uint8)
    for b, (n, m) in enumerate(zip(lens, n_new)):
        places = [(n - m + m // 2, 3)]  # a draft's, in one dim
        if d["window"] and n - m > d["window"]:
            # the farthest that the rows of the least depths see
            places.append((n - m + 2 - d["window"], 40))
        for at, dim in places:
            vb[int(d["table"][b, at // 32]), :, at % 32, dim] = 0x7f
    _same(_run(d, scale=scale), _want(d, scale))
    assert status()[0] == 0


@pytest.mark.parametrize("H,T", [(8, 2), (8, 40), (8, 70)])
def test_any_bits(H, T):
    """Bits that are no tree's: drafts that see later ones and not themselves,
    with a bias by the distance of their depths."""
    d = _case(64, 128, H, 2, T, [300, 90], [T, T - 1], 0, 0.0, True, True)
    g = torch.Generator().manual_seed(T)
    d["bits"] = torch.rand(2, T, T, generator=g) < 0.3
    _same(_run(d), _want(d))


@pytest.mark.parametrize("window", [1, 3])
@pytest.mark.parametrize("H,T", [(8, 2), (8, 40), (8, 70)])
def test_any_bits_and_a_window(H, T, window):
    """A later position than the row's is within every window."""
    d = _case(64, 128, H, 2, T, [300, 90], [T, T - 1], window, 0.0, True, True)
    g = torch.Generator().manual_seed(T)
    d["bits"] = torch.rand(2, T, T, generator=g) < 0.3
    depth = d["bits"].sum(-1) - 1
    later = d["bits"] & (depth[:, None, :] - depth[:, :, None] >= window)
    assert T == 2 or bool(later.any())
    _same(_run(d), _want(d))


@pytest.mark.parametrize("drafts", [False, True])
@pytest.mark.parametrize("D,G", [(64, 8), (128, 40), (128, 200)])
def test_weights_far_below_the_largest(D, G, drafts):
    """A row's first key weighs 1 and has values of 0, its second 2^-w with
    values of 1 (in units whose scale is 1/64 to 4 of the first's): what is left
    of 2^-w is within 2^-28, beside f16's 2^-11 and bf16's 2^-8 of itself."""
    page = 16
    w = torch.arange(G).double() * 40 / G
    q = torch.zeros(1, G, 1, D)
    q[0, :, 0, 0] = w * 0.6931471805599453
    q = q.bfloat16()
    k = torch.zeros(2, 1, page, D)
    k[0, :, 0, 0] = 1.0
    v = torch.zeros(2, 1, page, D)
    v[1, :, 0] = 1.0
    ones = torch.ones(2, 1)
    table = torch.tensor([[0, 1]], dtype=torch.int32)
    lens = torch.tensor([page + 1], dtype=torch.int32)
    k[0, :, 1:, 0] = -448.0  # the keys between the two: next to no weight
    more = dict(tree=torch.ones(1, 1, dtype=torch.int32).cuda()) if drafts \
        else {}
    for unit in (2.0 ** -6, 1.0, 4.0):
        vs = ones.clone()
        vs[1] = unit
        cache = bsm.KVCache(*[t.cuda() for t in (
            k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), ones, vs)])
        out, lse = bsm.paged_attention(q.cuda(), cache, table.cuda(),
                                       lens.cuda(), scale=1.0, **more)
        x = q[0, :, 0, 0].double()
        total = 1 + torch.exp(-x) + 15 * torch.exp(-449 * x)
        want = (torch.exp(-x) / total * unit)[:, None]
        err = (out[0, :, 0].double().cpu() - want).abs()
        tol = want * (2.0 ** -8 * (1 + 2.0 ** -7) + 2.0 ** -10) \
            + 2.0 ** -28 * unit
        assert bool((err <= tol).all()), float((err - tol).max())
        rel = (lse[0, :, 0].double().cpu() - x - torch.log(total)).abs()
        assert float(rel.max()) <= 1e-4
