"""Prompts on pooled caches whose committed pages end with the last row that a
sequence holds: nothing behind it is touched, and the bits are those of static
caches.  (A row's place decides where a page ends: head 1 starts 64 rows past a
page, so its pages end 64 rows before a multiple of 128.)"""
from __future__ import annotations

import pytest
import torch

from speculative_tree_verify_masked_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("D,dtype,Hq", [(256, BF, 12), (128, BF, 4), (64, BF, 2), (256, F32, 4)])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_prompt_ends_with_its_pages(D, dtype, Hq, n):
    pool = B.KVPool(0)
    try:
        per = pool.page_bytes // (D * dtype.itemsize)  # rows of a page
        cap, held = per + 64, per - 64
        L = held - n
        g = torch.Generator(device="cuda")
        g.manual_seed(D + n)

        def rnd(*shape):
            return torch.randn(*shape, generator=g, device="cuda").to(dtype)

        prompt, ln = B.Prompt([n]), torch.tensor([L, 0, 0, 0], dtype=torch.int32, device="cuda")
        q, k, v, w = rnd(n, Hq, D), rnd(n, 2, D), rnd(n, 2, D), torch.ones(D, device="cuda")
        old = [rnd(2, L, D) for _ in range(2)]
        outs = []
        for pooled in (False, True):
            kv = []
            for x in old:
                if pooled:
                    t = pool.cache(2, cap, D, dtype)
                    pool.commit_rows(t, held)
                else:
                    t = torch.zeros(2, cap, D, device="cuda", dtype=dtype)
                t[:, :L].copy_(x)
                kv.append(t)
            layer = B.AttnLayer(kv[:1], kv[1:], Hq)
            qr, out = torch.empty_like(q), torch.empty_like(q)
            ws = torch.empty(max(16, B.tv_attn_prompt_workspace_bytes(layer, prompt, L)), dtype=torch.uint8, device="cuda")
            B.tv_attn_prompt_front(layer, prompt, ln, L, w, w, 1e-6, 64, 1e4, q, k, v, qr)
            B.tv_attn_prompt(layer, prompt, ln, L, qr, None, out, D ** -0.5, ws)
            torch.cuda.synchronize()
            assert prompt.status_code() == 0
            outs.append((out, kv[0][:, :held].clone(), kv[1][:, :held].clone()))
        for a, b in zip(*outs):
            assert torch.equal(a, b)
    finally:
        pool.close()
