"""Where the prompt calls' buffers may lie: in place, and side by side in one allocation."""
from __future__ import annotations

import pytest
import torch

from speculative_tree_verify_masked_gb300 import binding as B
from tests.test_prompt_gpu import BF, F32, Attn, Front, gen_of, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF])
def test_norm_rope_in_place_and_side_by_side(dtype):
    g, n, Hq, Hkv, D = gen_of(81), 33, 6, 2, 128
    q_raw, k_raw, v = (rnd(g, n, H, D, dtype=dtype) for H in (Hq, Hkv, Hkv))
    w = [1 + 0.2 * rnd(g, D) for _ in range(2)]
    ln = torch.tensor([5], dtype=torch.int32, device="cuda")

    def run(q_raw, k_raw, v, q):
        K, V = ([torch.zeros(Hkv, 64, D, device="cuda", dtype=dtype)] for _ in range(2))
        p = B.Prompt([n])
        B.tv_attn_prompt_front(B.AttnLayer(K, V, Hq), p, ln, 5, w[0], w[1], 1e-6, 64, 1e4, q_raw, k_raw, v, q)
        torch.cuda.synchronize()
        assert p.status_code() == 0
        return q.clone(), K[0], V[0]

    ref = run(q_raw, k_raw, v, torch.empty_like(q_raw))
    pack = torch.cat([torch.zeros_like(q_raw).flatten(), q_raw.flatten(), k_raw.flatten(), v.flatten()])
    nq, nk = q_raw.numel(), k_raw.numel()
    q, qr, kr, vr = pack.split([nq, nq, nk, nk])
    views = qr.view(n, Hq, D), kr.view(n, Hkv, D), vr.view(n, Hkv, D)
    for out in (q.view(n, Hq, D), views[0]):  # ahead of the raw rows, then over them
        for a, b in zip(ref, run(*views, out)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,Hq,Hkv,D", [(F32, 6, 2, 64), (BF, 24, 4, 256), (BF, 16, 2, 128)])
@pytest.mark.parametrize("rows,ctx", [([90, 40], [30, 200]), ([24], [20000])])
def test_attn_prompt_gate_in_place(dtype, Hq, Hkv, D, rows, ctx):
    """The output over its own gates, far ones among them."""
    a, b = (Attn(rows, ctx, Hq, Hkv, D, dtype, gate=True, seed=82) for _ in range(2))
    for x in (a, b):
        x.gate[3, 1, ::9] = -70.0
        x.gate[4, 0, 5] = float("-inf")
    b.out = b.gate
    a.run()
    b.run()
    torch.cuda.synchronize()
    assert a.prompt.status_code() == b.prompt.status_code() == 0
    assert torch.equal(a.out, b.out)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_gdn_prompt_front_gates_in_place(dtype):
    a, b = (Front([70, 5], 2, 4, 64, 4, dtype, seed=83) for _ in range(2))
    b.alpha, b.beta = b.b, b.a  # crossed over, even
    a.run()
    b.run()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.outs(), b.outs()))
