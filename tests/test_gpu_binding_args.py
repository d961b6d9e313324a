"""What splash_attention and its backward take beside the plain shapes, and
what they refuse, on both ways into the library."""

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
from test_gpu_binding import both, same  # noqa: F401  (both: a fixture)

pytestmark = pytest.mark.gpu

SEG = bsm.MASK_CAUSAL | bsm.MASK_SEGMENT


def _tensors(B=1, H=2, S=200, D=64, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, H, S, D, generator=g).bfloat16().cuda()
            for _ in range(4)]


@pytest.mark.parametrize("dtype", [torch.int16, torch.uint16])
def test_bf16_bits_under_an_integer_type(both, dtype):  # noqa: F811
    q, k, v, do = _tensors()
    want = bsm.splash_attention(q, k, v)
    grads = bsm.splash_attention_bwd(q, k, v, *want, do)
    b = [t.view(dtype) for t in (q, k, v, do)]
    out = torch.empty_like(b[0])
    for got in both(lambda: bsm.splash_attention(*b[:3])):
        same(got, want)
    for got, lse in both(lambda: bsm.splash_attention(*b[:3], out=out)):
        assert got is out
        same([got.view(torch.bfloat16), lse], want)
    for got in both(lambda: bsm.splash_attention_bwd(
            *b[:3], want[0].view(dtype), want[1], b[3])):
        same([t.view(torch.bfloat16) for t in got], grads)


@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_flat_ids_and_logsumexp(both, softcap):  # noqa: F811
    """Segment ids of one row as [S], a logsumexp buffer of another shape."""
    q, k, v, do = _tensors()
    S = q.shape[2]
    ids = (torch.arange(S) // 70).int().cuda()
    kw = dict(mask_flags=SEG, softcap=softcap)
    two = dict(q_segment_ids=ids[None], kv_segment_ids=ids[None], **kw)
    one = dict(q_segment_ids=ids, kv_segment_ids=ids, **kw)
    want = bsm.splash_attention(q, k, v, **two)
    grads = bsm.splash_attention_bwd(q, k, v, *want, do, **two)
    lse = torch.empty(2 * S).cuda()
    for got, l in both(lambda: bsm.splash_attention(q, k, v, lse=lse, **one)):
        assert l is lse
        same([got, l.view(1, 2, S)], want)
    for got in both(lambda: bsm.splash_attention_bwd(q, k, v, want[0], lse,
                                                     do, **one)):
        same(got, grads)


def test_larger_buffers(both):  # noqa: F811
    """A larger out, or k and v of more batch rows, or v longer than k."""
    q, k, v, _ = _tensors(B=2)
    want = bsm.splash_attention(q[:1], k[:1], v[:1])
    wide = torch.full((2, 3, 300, 64), 7.0, dtype=torch.bfloat16).cuda()
    longer = torch.cat([v, v], 2)[:1]
    for got, lse in both(lambda: bsm.splash_attention(q[:1], k, longer,
                                                      out=wide)):
        assert got is wide
        same([got[:1, :2, :200].contiguous(), lse], want)
        assert (got[1:] == 7.0).all() and (got[:, 2:] == 7.0).all()
        assert (got[:, :, 200:] == 7.0).all()


def test_refusals_are_the_same(both):  # noqa: F811
    """Wrong types, devices and shapes: the same error on both ways."""
    q = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16).cuda()
    info = bsm.build_mask_info(bsm.MASK_CAUSAL, 1, 64, 64)
    lse = torch.zeros(1, 2, 64).cuda()
    seg = torch.zeros(1, 64, dtype=torch.int32).cuda()
    bad = [(q.half(), q, q), (q, q.cpu(), q), (q, q, q.float()),
           (q, q, q[:, :, :32]), (q, q[..., :32], q[..., :32]),
           (q, q[:, :, :, ::2], q)]
    calls = [lambda b=b: bsm.splash_attention(*b, mask_info=info, scale=1.0)
             for b in bad]
    calls += [lambda b=b: bsm.splash_attention_bwd(*b, q, lse, q, scale=1.0,
                                                   mask_info=info)
              for b in bad]
    calls += [lambda kw=kw: bsm.splash_attention(q, q, q, mask_info=info, **kw)
              for kw in (dict(out=q.float()), dict(out=q[:, :1]),
                         dict(out=q.cpu()), dict(lse=lse.double()),
                         dict(lse=lse[:, :, ::2]), dict(lse=lse.cpu()))]
    calls += [lambda i=i: bsm.splash_attention(
        q, q, q, mask_info=info, q_segment_ids=i, kv_segment_ids=i)
        for i in (seg.long(), seg.cpu(), seg[:, :32])]
    calls += [lambda: bsm.splash_attention_bwd(q, q, q, q, lse, q.cpu(),
                                               mask_info=info),
              lambda: bsm.splash_attention_bwd(q, q, q, q.half(), lse, q,
                                               mask_info=info),
              lambda: bsm.splash_attention_bwd(q, q, q, q, lse[:, :1], q,
                                               mask_info=info),
              lambda: bsm.splash_attention_bwd(q.cpu(), q, q, q, lse, q,
                                               mask_info=info)]
    for f in calls:
        seen = []

        def call():
            with pytest.raises((bsm.BsmError, ValueError)) as e:
                f()
            seen.append((type(e.value), str(e.value)))

        both(call)
        assert seen[0] == seen[1]


def test_host_tensors_with_the_current_stream_by_handle(both):  # noqa: F811
    q, k, v, _ = (t.cpu() for t in _tensors())
    want = bsm.splash_attention(q, k, v, softcap=9.0)
    for handle in (0, torch.cuda.current_stream().cuda_stream):
        for r in both(lambda: bsm.splash_attention(q, k, v, softcap=9.0,
                                                   stream=handle)):
            same(r, want)
