"""Pools, tables and expected results for the tests of the calls over pages."""
from __future__ import annotations

import random

import numpy as np
import torch

import oracle.paged as O
from speculative_tree_verify_masked_gb300 import binding as B

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def f64(t):
    return t.detach().double().cpu().numpy()


class Pools:
    """Pools and tables for slots of `lens` rows (-1: idle), room for `extra` more each; groups of
    (members, shared rows) share their first pages.  Whatever no slot sees at lens[s] + 1 rows is NaN."""

    def __init__(self, lens, page=64, heads=(24, 4, 256), dtype=torch.bfloat16, seed=0, extra=1, groups=(), max_len=None,
                 spare=3, cols=None, fill=float("nan")):
        rng, gen = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.page, self.dtype = list(lens), page, dtype
        self.Hq, self.Hkv, self.D = heads
        self.max_len = max(max(lens), 0) if max_len is None else max_len
        n = len(lens)
        cols = max(-(-(self.max_len + extra) // page), cols or 0)
        table, used, at = [[-1] * cols for _ in lens], 0, 0
        own_from = [0] * n
        for members, shared in groups:
            for i in range(at, at + members):
                table[i][:shared // page] = range(used, used + shared // page)
                own_from[i] = shared // page
            used, at = used + shared // page, at + members
        for i, L in enumerate(lens):
            if L >= 0:
                for j in range(own_from[i], -(-(L + extra) // page)):
                    table[i][j], used = used, used + 1
        self.n_pages = used + spare
        order = list(range(self.n_pages))
        rng.shuffle(order)
        self.rows = [[order[x] if x >= 0 else -1 for x in r] for r in table]  # host table
        self.table = torch.tensor(self.rows, dtype=torch.int32, device="cuda")
        self.len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        shape = (self.n_pages, self.Hkv, page, self.D)
        self.K, self.V = (torch.randn(shape, generator=gen, device="cuda").to(dtype) for _ in range(2))
        seen = torch.zeros(self.n_pages, page, dtype=torch.bool)
        for i, L in enumerate(lens):
            for j in range(L // page + 1 if L >= 0 else 0):
                seen[self.rows[i][j], :min(page, L + 1 - j * page)] = True
        if fill is not None:
            hide = ~seen.to("cuda")[:, None, :, None].expand(shape)
            self.K[hide] = fill
            self.V[hide] = fill
        self.q = torch.randn((n, self.Hq, self.D), generator=gen, device="cuda").to(dtype)
        self.gate = torch.randn((n, self.Hq, self.D), generator=gen, device="cuda").to(dtype)
        self.out = torch.full((n, self.Hq, self.D), 7.0, dtype=dtype, device="cuda")
        self.scale = self.D ** -0.5
        self.layer = B.PagedLayer(self.K, self.V, self.Hq)
        self.batch = B.PagedBatch(self.table, self.len, self.max_len)
        self.groups = B.PagedGroups([m for m, _ in groups], [x for _, x in groups]) if groups else None

    def space(self, need):
        # workspaces hold whatever was there before
        return torch.full((max(need, 16),), 0xff, dtype=torch.uint8, device="cuda")

    def attn(self, gate=None, groups=None, stream=None):
        ws = self.space(B.tv_paged_attn_workspace_bytes(self.layer, self.batch, groups))
        B.tv_paged_attn(self.layer, self.batch, groups, self.q, gate, self.out, self.scale, ws, stream)
        return self.out

    def selected(self, sel, count, gate=None, stream=None):
        ws = self.space(B.tv_paged_attn_selected_workspace_bytes(self.layer, self.batch, sel.shape[-1]))
        B.tv_paged_attn_selected(self.layer, self.batch, sel, count, self.q, gate, self.out, self.scale, ws, stream)
        return self.out

    def status(self):
        return self.batch.status_code()

    def expect(self, got, gate=None, places=None, slots=None):
        """Every slot's rows against the oracle.  A weight is off by half a step of bf16 where it is rounded
        for the product, by its score's error (D roundings of the products' sum at most, in fp32) and by a few
        fp32 steps of the exponential; the sums add a rounding a row at most; then the output's rounding."""
        got = f64(got)
        K, V = f64(self.K), f64(self.V)
        low = self.dtype == torch.bfloat16
        for i, L in enumerate(self.lens):
            if slots is not None and i not in slots:
                continue
            if L < 0:
                assert (got[i] == 7).all(), f"idle slot {i} written"
                continue
            ref, mag, prod = O.attend(K, V, self.rows[i], L, f64(self.q[i]), self.scale, None if gate is None else f64(gate[i]),
                                      None if places is None else places[i])
            rel = 2.0 ** -24 * (2 * self.D * prod + L + 64) + (HALF[self.dtype] if low else 0.0)
            tol = rel * mag * 1.01 + HALF[self.dtype] * np.abs(ref) * 1.01 + 1e-37
            err = np.abs(got[i] - ref)
            assert np.isfinite(got[i]).all(), f"slot {i}: not finite"
            assert (err <= tol).all(), f"slot {i} (len {L}): {err.max():.3e}, allowed {tol.flat[(err - tol).argmax()]:.3e}"
