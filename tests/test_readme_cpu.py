"""The README's examples of drafted tokens, run with the checks of their
arguments in place of the kernels."""

import os
import re
import types

import torch

import block_sparse_masked_build_gb300 as bsm
from block_sparse_masked_build_gb300 import api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_drafted_tokens():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    code = [b for b in blocks if "tree=tree" in b]
    assert len(code) == 1
    B, T, H, Hkv, D = 2, 5, 4, 2, 64
    cpu, calls = torch.device("cpu"), []

    def kv_append(cache, table, lens, k, v, *, n_new, rope, positions,
                  k_weight, eps):
        calls.append(("append", lens.clone(), positions))
        api._check_table(cpu, table, B, lens, n_new)
        api._turn(rope, positions, None, k_weight, eps, B, T, D, cpu)

    def norm_rope(q, *, rope, positions, q_weight, eps):
        calls.append(("rotate", None, positions))
        api._turn(rope, positions, q_weight, None, eps, B, T, D, cpu)
        return q, None

    def paged_attention(q, cache, table, lens, *, tree, n_new):
        calls.append(("attend", lens.clone(), None))
        api._check_table(cpu, table, B, lens, n_new)
        api._check_tree(tree, B, T, cpu)
        return q, None

    bits = torch.ones(B, T, T, dtype=torch.bool).tril()
    lens, n = (torch.tensor(x, dtype=torch.int32) for x in ([7, 30], [5, 4]))
    z = lambda h: torch.zeros(B, h, T, D, dtype=torch.bfloat16)  # noqa: E731
    exec(code[0], dict(
        bsm=types.SimpleNamespace(kv_append=kv_append, norm_rope=norm_rope,
                                  paged_attention=paged_attention),
        cache=None, page_table=torch.zeros(B, 4, dtype=torch.int32),
        rope=bsm.Rope(D), wq=torch.ones(D), wk=torch.ones(D), q=z(H), k=z(Hkv),
        v=z(Hkv), lens=lens, n=n, bits=bits, depth=bits.sum(-1) - 1,
        tree=torch.zeros(B, T, 1, dtype=torch.int32)))
    want = torch.tensor([[7, 8, 9, 10, 11], [30, 31, 32, 33, 34]])
    assert [c[0] for c in calls] == ["append", "rotate", "attend"]
    assert calls[0][1].tolist() == [7, 30] and calls[2][1].tolist() == [12, 34]
    assert all(torch.equal(c[2].long(), want) for c in calls[:2])
