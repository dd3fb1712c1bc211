"""Infinities and NaN among a prompt's own rows: rows before them, other
columns where the definition keeps them apart, and other sequences are as if
they were finite, and rows that do see them are not finite there.  Bounds as in
test_prompt_gpu.py."""
from __future__ import annotations

import pytest
import torch

import oracle.prompt as OP
from tests.test_prompt_gpu import BF, F32, NAN, U, Attn, Gdn, within

pytestmark = pytest.mark.gpu

INF = float("inf")


def clean(t):
    return torch.where(torch.isfinite(t), t, torch.zeros_like(t))


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(24, 4, 256, BF), (4, 4, 64, BF), (16, 2, 128, BF), (6, 2, 64, F32)])
@pytest.mark.parametrize("rows,ctx", [([150, 40], [30, 0]), ([24], [20000]), ([3, 70], [126, 5]), ([300], [1000]),
                                      ([1, 128], [128, 128])])
@pytest.mark.parametrize("gate", [False, True])
def test_attn_prompt_values_not_finite(Hq, Hkv, D, dtype, rows, ctx, gate):
    a = Attn(rows, ctx, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, gate=gate, seed=31, pad=3)
    for s, (L, n) in enumerate(zip(ctx, rows)):  # value rows all over the prompt, its last row among them
        for j, (x, c) in enumerate([(NAN, 0), (INF, 1), (-INF, D - 1), (INF, D // 2), (-INF, D // 2)]):
            a.V[s][j % Hkv, L + (n - 1) * (j + 1) // 5, c] = x
    a.run()
    torch.cuda.synchronize()
    assert a.prompt.status_code() == 0
    off = 0
    for s, (L, n) in enumerate(zip(ctx, rows)):
        g = None if a.gate is None else a.gate[off:off + n]
        got, V = a.out[off:off + n], a.V[s]
        ref, reach = OP.attn_prompt(a.K[s], clean(V[:, :L + n]), L, a.q[off:off + n], a.scale, g)
        hit = (~torch.isfinite(V[:, :L + n])).cumsum(1)[:, L:].bool()  # [Hkv, n, D]: seen by row i
        hit = hit.transpose(0, 1).repeat_interleave(Hq // Hkv, 1)
        assert torch.equal(~torch.isfinite(got), hit), f"sequence {s}"
        noise, u = (4e-4, U[BF]) if dtype == BF else (8e-5, U[F32])
        keep = torch.where(hit, torch.zeros_like(ref), ref)
        within(torch.where(hit, torch.zeros_like(got), got), keep, 2 * u * keep.abs() + (u + noise) * reach + 1e-30, f"sequence {s}")
        off += n


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(24, 4, 256, BF), (8, 2, 64, BF), (6, 2, 64, F32)])
@pytest.mark.parametrize("rows,ctx", [([150, 40], [30, 0]), ([24], [20000])])
def test_attn_prompt_keys_and_queries_not_finite(Hq, Hkv, D, dtype, rows, ctx):
    a = Attn(rows, ctx, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=32)
    n0, L0 = rows[0], ctx[0]
    a.K[0][1, L0 + n0 // 2, 3] = NAN   # rows from here on, heads of KV head 1
    a.q[n0 // 3, 0, 5] = NAN           # one row of one head
    a.run()
    torch.cuda.synchronize()
    G = Hq // Hkv
    bad = torch.zeros(sum(rows), Hq, dtype=torch.bool, device="cuda")
    bad[n0 // 2:n0, G:2 * G] = True
    bad[n0 // 3, 0] = True
    assert torch.equal(torch.isfinite(a.out).all(-1), ~bad) and torch.equal(torch.isnan(a.out).all(-1), bad)
    off = 0
    for s, (L, n) in enumerate(zip(ctx, rows)):
        b = bad[off:off + n, :, None]
        ref, reach = OP.attn_prompt(clean(a.K[s][:, :L + n]), a.V[s][:, :L + n], L, clean(a.q[off:off + n]), a.scale)
        noise, u = (4e-4, U[BF]) if dtype == BF else (8e-5, U[F32])
        got = a.out[off:off + n]
        within(torch.where(b, torch.zeros_like(got), got), torch.where(b, torch.zeros_like(ref), ref),
               2 * u * ref.abs() + (u + noise) * reach + 1e-30, f"sequence {s}")
        off += n


def test_attn_prompt_keys_not_finite_over_whole_pieces():
    """A long run of NaN keys in the context: every row of that KV head is NaN, also where the keys are split."""
    a = Attn([5], [30000], Hq=8, Hkv=2, D=128, seed=33)
    a.K[0][0, 1000:25000] = NAN
    a.run()
    torch.cuda.synchronize()
    assert bool(torch.isnan(a.out[:, :4]).all()) and bool(torch.isfinite(a.out[:, 4:]).all())


@pytest.mark.parametrize("Hk,Hv,dk,dv,dtype", [(4, 8, 128, 128, BF), (2, 4, 64, 64, BF), (2, 2, 64, 64, F32), (2, 4, 64, 96, BF)])
@pytest.mark.parametrize("what,x", [("v", NAN), ("v", -INF), ("k", NAN), ("k", INF), ("q", NAN), ("alpha", NAN), ("beta", NAN),
                                    ("beta", INF), ("S", NAN)])
def test_gdn_prompt_not_finite(Hk, Hv, dk, dv, dtype, what, x):
    rows = [200, 30, 64, 129]
    g = Gdn(rows, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype=dtype, seed=34)
    off = [0, 200, 230, 294]
    for s, r in ((0, 70), (2, 63), (3, 0)):
        if what == "S":
            g.S[s][1, 5, 3] = x
            g.S0[s][1, 5, 3] = x
        elif what in ("v", "k", "q"):
            getattr(g, what)[off[s] + r, 1, 5] = x
        else:
            getattr(g, what)[off[s] + r, 1] = x
    g.run()
    torch.cuda.synchronize()
    assert g.prompt.status_code() == 0
    for s, n in enumerate(rows):
        sl = slice(off[s], off[s] + n)
        ref, S = OP.gdn_prompt(g.S0[s], g.q[sl], g.k[sl], g.v[sl], g.alpha[sl], g.beta[sl], g.scale)
        hit, hitS = ~torch.isfinite(ref), ~torch.isfinite(S)
        assert torch.equal(~torch.isfinite(g.out[sl]), hit), f"out {s}"
        assert torch.equal(~torch.isfinite(g.S[s]), hitS), f"state {s}"
        got, ref = torch.where(hit, 0, g.out[sl].double()), torch.where(hit, 0, ref)
        err = float((got - ref).norm() / ref.norm()) if bool((~hit).any()) else 0.0
        assert err <= (5e-3 if dtype == BF else 1e-5), (s, err)
        gotS, S = torch.where(hitS, 0, g.S[s].double()), torch.where(hitS, 0, S)
        err = float((gotS - S).norm() / S.norm()) if bool((~hitS).any()) else 0.0
        assert err <= 2e-5, (s, err)
