"""Norm and rotation of query and key rows on the GPU, forward and backward,
against fp64.

Tolerances.  The result is rounded to bf16 once (half a step, 2^-8 relative).
Before that everything is f32: cosines and sines are off by at most 2^-20 of the pair's
length, the norm's factor, the weight and the products by a few 2^-24, the sum
of up to 128 squares or products by at most 128 * 2^-24 of the sum of
magnitudes: together less than 2^-16 of the element's size as the reference
gives it.  A weight's gradient is a sum of N products in f32 whose terms carry
those 2^-16; its own additions, in chains of at most 1024 per lane and two more
levels, stay below 2^-13 of the sum of magnitudes.
"""

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import rope_ref as ref
from test_gpu_binding import both  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

EPS = 1e-6


def near(got, want, size, what):
    got = got.double().cpu()
    tol = 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8) + 2.0 ** -16 * size + 1e-38
    err = (got - want).abs()
    assert bool((err <= tol).all()), (what, float((err - tol).max()))


# B, H, Hkv, S, D, dim, interleaved, axes, norm, weights, far
CASES = [
    (1, 1, 0, 1, 64, 64, False, 1, True, torch.float32, 0),
    (1, 1, 1, 1, 128, 128, False, 1, True, torch.bfloat16, 5),
    (2, 5, 1, 37, 128, 128, False, 1, True, torch.bfloat16, 1000),
    (2, 4, 2, 33, 64, 32, True, 1, True, torch.float32, 0),
    (1, 12, 4, 300, 128, 112, False, 1, True, None, 250000),
    (1, 3, 3, 129, 64, 48, False, 3, False, None, 100),
    (3, 8, 8, 65, 128, 64, True, 2, True, torch.float32, 2 ** 30),
    (1, 7, 1, 200, 128, 16, True, 1, False, None, 77),
    (2, 6, 2, 50, 128, 0, False, 1, True, torch.bfloat16, 0),
    (2, 6, 0, 50, 64, 0, False, 1, True, None, 0),
    (1, 40, 8, 1500, 128, 128, False, 4, True, torch.bfloat16, 3000000),
]


def _case(B, H, Hkv, S, D, dim, inter, axes, norm, wtype, far, seed=0,
          strided=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, S, H + Hkv + 1, D, generator=g)
    x = (x * torch.exp2(torch.randint(-6, 7, (B, S, H + Hkv + 1, 1),
                                      generator=g).float())).bfloat16()
    q, k = (x[:, :, a:a + n].transpose(1, 2) for a, n in ((0, H), (H, Hkv)))
    d = dict(q=q, k=k if Hkv else None, rope=None, positions=None, angle=None,
             inter=inter, eps=EPS if norm else None, qw=None, kw=None)
    if wtype is not None and norm:
        d["qw"], d["kw"] = ((1 + 0.3 * torch.randn(D, generator=g)).to(wtype)
                            for _ in range(2))
        if not Hkv:
            d["kw"] = None
    if dim:
        axis = [i * axes // (dim // 2) for i in range(dim // 2)]
        base = 1e4 if D == 64 else 1e6
        d["rope"] = bsm.Rope(dim, base, axes=axis if axes > 1 else None,
                             interleaved=inter)
        pos = torch.randint(0, 5000, (axes, B, S), generator=g) + far
        d["positions"] = pos.int()
        d["angle"] = ref.angles(pos, ref.frequencies(dim, base), axis)
    return d


def _args(d):
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    return dict(rope=d["rope"], positions=c(d["positions"]),
                q_weight=c(d["qw"]), k_weight=c(d["kw"]), eps=d["eps"])


def _wide(d, name):
    """The tensor on the GPU as a view into a wider buffer, as a projection
    leaves it."""
    t = d[name]
    if t is None:
        return None
    base = torch.zeros(t.shape[0], t.shape[2], t.shape[1] + 2, t.shape[3],
                       dtype=t.dtype, device="cuda")
    view = base[:, :, 1:-1].transpose(1, 2)
    view.copy_(t)
    return view


@pytest.mark.parametrize("case", CASES)
def test_forward(both, case):  # noqa: F811
    d = _case(*case)
    for got in both(lambda: bsm.norm_rope(_wide(d, "q"), _wide(d, "k"),
                                          **_args(d))):
        for t, x, w, n in ((got[0], "q", "qw", "out"),
                           (got[1], "k", "kw", "k_out")):
            if d[x] is None:
                assert t is None
                continue
            near(t, *ref.forward(d[x], d[w], d["eps"], d["angle"],
                                 d["inter"]), n)


@pytest.mark.parametrize("case", CASES)
def test_backward(both, case):  # noqa: F811
    d = _case(*case)
    g = torch.Generator().manual_seed(9)
    d["gq"] = torch.randn(d["q"].shape, generator=g).bfloat16()
    d["gk"] = None if d["k"] is None else torch.randn(
        d["k"].shape, generator=g).bfloat16()
    x = (_wide(d, "q"), _wide(d, "k")) if d["eps"] is not None else ()
    for got in both(lambda: bsm.norm_rope_bwd(_wide(d, "gq"), _wide(d, "gk"),
                                              *x, **_args(d))):
        for i, n in ((0, "q"), (1, "k")):
            if d[n] is None:
                assert got[i] is None and got[2 + i] is None
                continue
            dx, size, dw, dsize = ref.backward(d["g" + n], d[n], d[n + "w"],
                                               d["eps"], d["angle"],
                                               d["inter"])
            near(got[i], dx, size, "d" + n)
            if d[n + "w"] is None:
                assert got[2 + i] is None
                continue
            err = (got[2 + i].double().cpu() - dw).abs()
            assert bool((err <= 2.0 ** -13 * dsize).all()), n


def test_backward_against_differences():
    """The gradient of sum(g y) against differences of the definition itself
    (fp64), so that formula and kernel cannot share a mistake."""
    d = _case(2, 2, 1, 5, 64, 32, True, 2, True, torch.float32, 10)
    g = {n: torch.randn(d[n].shape, generator=torch.Generator().manual_seed(i))
         .bfloat16() for i, n in ((1, "q"), (2, "k"))}
    got = bsm.norm_rope_bwd(g["q"].cuda(), g["k"].cuda(), d["q"].cuda(),
                            d["k"].cuda(), **_args(d))

    def loss(n, x, w):
        y, _ = ref.forward(x, w, EPS, d["angle"], True)
        return float((y * g[n].double()).sum())

    for i, n in ((0, "q"), (1, "k")):
        x, w = d[n].double(), d[n + "w"].double()
        for at in ((0, 0, 0, 3), (1, 0, 4, 33), (0, x.shape[1] - 1, 2, 63)):
            h = 1e-4 * max(1e-3, float(x[at].abs()))
            hi, lo = x.clone(), x.clone()
            hi[at] += h
            lo[at] -= h
            want = (loss(n, hi, w) - loss(n, lo, w)) / (2 * h)
            have = float(got[i][at])
            assert abs(have - want) <= 2.0 ** -7 * abs(want) + 1e-3, (n, at)
        for at in (0, 17, 63):
            hi, lo = w.clone(), w.clone()
            hi[at] += 1e-4
            lo[at] -= 1e-4
            want = (loss(n, x, hi) - loss(n, x, lo)) / 2e-4
            assert abs(float(got[2 + i][at]) - want) <= 1e-3 * (1 + abs(want))


def test_in_place_and_default_positions(both):  # noqa: F811
    d = _case(2, 4, 2, 70, 128, 128, False, 1, True, torch.bfloat16, 0)
    args = _args(d)
    at = torch.arange(70, dtype=torch.int32, device="cuda").expand(2, 70)
    args["positions"] = at  # a row that repeats: stride 0
    want = bsm.norm_rope(d["q"].cuda(), d["k"].cuda(), **args)
    args["positions"] = None

    def run():
        q, k = _wide(d, "q"), _wide(d, "k")
        got = bsm.norm_rope(q, k, out=q, k_out=k, **args)
        assert got[0] is q and got[1] is k
        return got

    for got in both(run):
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_far_positions_are_exact():
    """A position and the same one some whole turns on agree: frequencies of a
    whole fraction of a turn."""
    import math
    freq = [2 * math.pi / 2 ** (i % 8 + 2) for i in range(32)]
    rope = bsm.Rope(64, inv_freq=freq)
    q = torch.randn(1, 2, 9, 64).bfloat16()
    at = torch.arange(9, dtype=torch.int32)[None]
    far = (at + 2 ** 30).cuda()
    want = ref.angles(at[None], torch.tensor(freq, dtype=torch.float64),
                      [0] * 32)
    out, _ = bsm.norm_rope(q.cuda(), rope=rope, positions=far)
    # (inv_freq / 2 pi as a double: 2^30 positions of 2^-54 turns each)
    near(out, *ref.forward(q, None, None, want, False), "far")
    back, _ = bsm.norm_rope(out, rope=rope, positions=-far)
    # there and back: two roundings, each 2^-8 of a pair's length at most
    size = ref.sizes(q.double(), 32, False)
    assert bool(((back.double().cpu() - q.double()).abs()
                 <= 2.0 ** -6.9 * size).all())


def test_edge_values():
    """A zero row stays zero; rows with NaN or infinity keep to themselves; an
    infinity in a pair does not reach elements that do not turn."""
    rope = bsm.Rope(64)
    q = torch.randn(1, 4, 6, 128).bfloat16()
    q[0, 0, 1] = 0
    q[0, 1, 2, 5] = float("nan")
    q[0, 2, 3, 7] = float("inf")
    out, _ = bsm.norm_rope(q.cuda(), rope=rope, eps=EPS)
    out = out.cpu()
    assert (out[0, 0, 1] == 0).all()
    assert out[0, 1, 2].isnan().all()
    rows = torch.ones(4, 6, dtype=torch.bool)
    rows[1, 2] = rows[2, 3] = False
    assert out[0][rows].isfinite().all()
    plain, _ = bsm.norm_rope(q.cuda(), rope=rope)
    assert torch.equal(plain[0, 2, 3, 64:].cpu(), q[0, 2, 3, 64:])
    big = torch.full((1, 1, 1, 64), 2.0 ** 59).bfloat16().cuda()
    y, _ = bsm.norm_rope(big, eps=0.0)
    assert torch.equal(y, torch.ones_like(y))


def test_no_rows():
    rope = bsm.Rope(64)
    w = torch.ones(64).cuda()
    for shape in ((0, 2, 5, 64), (1, 2, 0, 64), (1, 0, 5, 64)):
        q = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        out, none = bsm.norm_rope(q, rope=rope, eps=EPS, q_weight=w)
        assert out.shape == q.shape and none is None
        r = bsm.norm_rope_bwd(q, None, q, rope=rope, eps=EPS, q_weight=w)
        assert r[0].shape == q.shape and (r[2] == 0).all()


def test_streams_and_graphs():
    """On a given stream, and captured: a graph replays on new contents."""
    d = _case(2, 8, 2, 120, 128, 128, False, 1, True, torch.float32, 3)
    args = _args(d)
    q, k = d["q"].cuda(), d["k"].cuda()
    g = torch.randn_like(q), torch.randn_like(k)
    want = bsm.norm_rope(q, k, **args) + bsm.norm_rope_bwd(*g, q, k, **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bsm.norm_rope(q, k, stream=side, **args) + bsm.norm_rope_bwd(
        *g, q, k, stream=side, **args)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):  # two graphs of one stream, with memory of their own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = bsm.norm_rope(q, k, **args) + bsm.norm_rope_bwd(*g, q, k,
                                                                  **args)
        graphs.append((graph, res))
    q.mul_(1.5)
    args["positions"].add_(7)
    want = bsm.norm_rope(q, k, **args) + bsm.norm_rope_bwd(*g, q, k, **args)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for (graph, _), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    for _, res in graphs:
        assert all(torch.equal(a, b) for a, b in zip(res, want))


def test_layer(both):  # noqa: F811
    """As a layer uses it: norm and rotation, attention, and their backwards,
    against autograd of the formulas in fp64."""
    d = _case(1, 4, 2, 150, 64, 64, False, 1, True, torch.float32, 0)
    v = torch.randn(1, 2, 150, 64).bfloat16()
    do = torch.randn(1, 4, 150, 64).bfloat16()
    x = [t.double().requires_grad_() for t in (d["q"], d["k"], d["qw"],
                                               d["kw"])]

    def rows(t, w):
        n = t / torch.sqrt(t.square().mean(-1, keepdim=True) + EPS) * w
        return ref.turn(n, d["angle"], False)

    q, k = rows(x[0], x[2]), rows(x[1], x[3]).repeat_interleave(2, 1)
    z = (q @ k.transpose(2, 3) / 8).masked_fill(
        ~torch.ones(150, 150, dtype=torch.bool).tril(), float("-inf"))
    y = torch.softmax(z, -1) @ v.double().repeat_interleave(2, 1)
    want = torch.autograd.grad(y, x, do.double())

    def run():
        args = _args(d)
        a = (d["q"].cuda(), d["k"].cuda())
        q, k = bsm.norm_rope(*a, **args)
        out, lse = bsm.splash_attention(q, k, v.cuda())
        dq, dk, _ = bsm.splash_attention_bwd(q, k, v.cuda(), out, lse,
                                             do.cuda())
        return (out, *bsm.norm_rope_bwd(dq, dk, *a, **args))

    # the attention's own gates: 2e-2 of the largest element
    for got in both(run):
        for t, w in zip(got, (y.detach(), *want)):
            err = (t.double().cpu() - w).abs().max()
            assert float(err) <= 2e-2 * float(w.abs().max())


@pytest.mark.parametrize("case", [
    (1, 13, 3, 5003, 64, 64, False, 1, True, torch.bfloat16, 9),
    (2, 5, 2, 3001, 128, 64, True, 2, True, torch.float32, 0),
    (1, 9, 1, 8195, 64, 32, False, 1, False, None, 70000)])
def test_many_rows(case):
    """Several heads of a token for a group of lanes, unevenly, and several
    tokens one after another in the backward; the forward also in place."""
    d = _case(*case)
    g = torch.Generator().manual_seed(4)
    gq, gk = (torch.randn(d[n].shape, generator=g).bfloat16() for n in "qk")
    args = _args(d)
    q, k = d["q"].cuda(), d["k"].cuda()
    x = (q, k) if d["eps"] is not None else ()
    got = bsm.norm_rope_bwd(gq.cuda(), gk.cuda(), *x, **args)
    res = bsm.norm_rope(q, k, **args)
    for i, n in ((0, "q"), (1, "k")):
        w = d[n + "w"]
        near(res[i], *ref.forward(d[n], w, d["eps"], d["angle"], d["inter"]),
             n)
        dx, size, dw, dsize = ref.backward((gq, gk)[i], d[n], w, d["eps"],
                                           d["angle"], d["inter"])
        near(got[i], dx, size, "d" + n)
        if w is not None:
            err = (got[2 + i].double().cpu() - dw).abs()
            assert bool((err <= 2.0 ** -13 * dsize).all()), n
    bsm.norm_rope(q, k, out=q, k_out=k, **args)
    assert torch.equal(q, res[0]) and torch.equal(k, res[1])
    assert bsm.bsm_device_status()[0] == 0
