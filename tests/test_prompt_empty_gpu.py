"""Batches without rows in buffers that hold some: every prompt call accepts a host
bound n_max of 0, checks the offsets and writes nothing."""
from __future__ import annotations

import pytest
import torch

from speculative_tree_verify_masked_gb300 import binding as B
from tests.test_prompt_gpu import BF, F32, Front, Gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 256), (BF, 64), (BF, 256)])
@pytest.mark.parametrize("max_len", [5, 3000])
def test_no_rows(dtype, D, max_len):
    Hq, Hkv, n, cap = 4, 2, 11, 4096
    K, V = ([torch.full((Hkv, cap, D), 7.0, device="cuda", dtype=dtype) for _ in range(2)] for _ in range(2))
    layer = B.AttnLayer(K, V, Hq)
    ln = torch.tensor([max_len, 0], dtype=torch.int32, device="cuda")
    q, k = torch.ones(n, Hq, D, device="cuda", dtype=dtype), torch.ones(n, Hkv, D, device="cuda", dtype=dtype)
    out, q2 = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    p = B.Prompt([0, 0], n_total=n)
    assert p.n_max == 0
    ws = torch.zeros(max(16, B.tv_attn_prompt_workspace_bytes(layer, p, max_len)), dtype=torch.uint8, device="cuda")

    def calls():
        B.tv_prompt_check(p, ln, max_len, cap)
        B.tv_attn_prompt_front(layer, p, ln, max_len, None, None, 1e-6, D, 1e4, q, k, k, q2)
        B.tv_attn_prompt(layer, p, ln, max_len, q, None, out, 0.1, ws)
        B.tv_prompt_advance(p, ln)

    calls()
    torch.cuda.synchronize()
    assert p.status_code() == 0 and ln.tolist() == [max_len, 0]
    assert all(bool((t == 7.0).all()) for t in K + V + [out, q2])
    p.row_off.copy_(torch.tensor([0, 1, 1]))  # a row more than the bound
    B.tv_attn_prompt(layer, p, ln, max_len, q, None, out, 0.1, ws)
    torch.cuda.synchronize()
    assert p.status_code() == 12 and bool((out == 7.0).all())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_no_rows_gdn(dtype):
    f = Front([0, 0], 2, 4, 64, 4, dtype, pad=9)
    x = Gdn([0, 0], 2, 4, 64, 64, dtype, pad=9)
    old = [t.clone() for t in f.tails]
    assert f.prompt.n_max == 0 and x.prompt.n_max == 0
    f.run()
    x.run()
    torch.cuda.synchronize()
    assert f.prompt.status_code() == 0 and x.prompt.status_code() == 0
    assert all(bool((t == 7.0).all()) for t in f.outs()) and bool((x.out == 7.0).all())
    assert all(torch.equal(a, b) for a, b in zip(old + x.S0, f.tails + x.S))
