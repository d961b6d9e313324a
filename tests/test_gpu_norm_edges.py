"""The norm at the ends of the magnitudes that its f32 sums hold, on the GPU."""

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import rope_ref as ref
from test_gpu_norm_rope import near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("top", [-59, 0, 59])
def test_magnitudes_without_eps(D, top):
    """Rows whose largest element is 2^top: alone, beside others up to it, and
    equal to all of them; a row of zeros is NaN and no other one."""
    g = torch.Generator().manual_seed(D + top)
    x = torch.randn(1, 3, 40, D, generator=g)
    x = (x / x.abs().amax(-1, keepdim=True)).double() * 2.0 ** top
    x[0, 0, :5] = 0
    x[0, 0, :5, 3] = 2.0 ** top
    x[0, 0, 5] = -2.0 ** top
    x = x.bfloat16()
    w = (1 + 0.3 * torch.randn(D, generator=g)).float()
    gr = torch.randn(1, 3, 40, D, generator=g).bfloat16()
    args = dict(q_weight=w.cuda(), eps=0.0)
    out, _ = bsm.norm_rope(x.cuda(), **args)
    near(out, *ref.forward(x, w, 0.0, None, False), "out")
    dx, _, dw, _ = bsm.norm_rope_bwd(gr.cuda(), None, x.cuda(), **args)
    want, size, want_dw, size_dw = ref.backward(gr, x, w, 0.0, None, False)
    # (in units of 1 / 2^top, as the least number of the tolerance is absolute)
    near(dx.double() * 2.0 ** top, want * 2.0 ** top, size * 2.0 ** top, "dx")
    assert bool(((dw.double().cpu() - want_dw).abs()
                 <= 2.0 ** -13 * size_dw).all())
    x[0, 1, 7] = 0
    out, _ = bsm.norm_rope(x.cuda(), eps=0.0)
    rows = out.cpu()[0].isnan().any(-1)
    assert bool(out.cpu()[0, 1, 7].isnan().all()) and int(rows.sum()) == 1
