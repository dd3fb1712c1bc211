"""Infinities, NaN and far values in a prompt's rows and caches, told apart: what
comes out is NaN, +inf or -inf where the definition gives that, and as if the rest
were alone elsewhere.  Bounds as in test_prompt_gpu.py."""
from __future__ import annotations

import pytest
import torch

import oracle.prompt as OP
from tests.test_prompt_gpu import BF, F32, NAN, U, Attn, Front

pytestmark = pytest.mark.gpu

INF = float("inf")


def same(got, ref, bound, what):
    """NaN and each infinity where ref has it, within the bound elsewhere."""
    got = got.double()
    for name, f in (("nan", torch.isnan), ("+inf", torch.isposinf), ("-inf", torch.isneginf)):
        bad = f(got) != f(ref)
        assert not bool(bad.any()), f"{what}: {name} differs at {bad.nonzero()[0].tolist()} ({int(bad.sum())} places)"
    fin = torch.isfinite(ref)
    over = torch.where(fin, (got - ref).abs() - bound, torch.full_like(ref, -1.0))
    assert float(over.max()) <= 0, f"{what}: {float(over.max()):.3e} over its bound"


def check_attn(a, what=""):
    """The call's outputs against the definition, non-finite places told apart."""
    torch.cuda.synchronize()
    assert a.prompt.status_code() == 0
    off = 0
    for s, (L, n) in enumerate(zip(a.ctx, a.rows)):
        g = None if a.gate is None else a.gate[off:off + n]
        ref, _ = OP.attn_prompt(a.K[s], a.V[s], L, a.q[off:off + n], a.scale, g)
        # a weight of 0 must not meet an unseen value: the definition over each row's own prefix
        V = a.V[s][:, :L + n].double()
        if not bool(torch.isfinite(V).all()):
            fin = torch.where(torch.isfinite(V), V, torch.zeros_like(V))
            ref, _ = OP.attn_prompt(a.K[s], fin, L, a.q[off:off + n], a.scale)
            G = ref.shape[1] // V.shape[0]
            seen = lambda x: (x.cumsum(1) > 0)[:, L:].transpose(0, 1).repeat_interleave(G, 1)
            nan, pos, neg = seen(torch.isnan(V)), seen(torch.isposinf(V)), seen(torch.isneginf(V))
            ref = torch.where(pos, ref + INF, ref)
            ref = torch.where(neg, ref - INF, ref)
            ref = torch.where(nan, ref + NAN, ref)
            if g is not None:
                ref = ref * torch.sigmoid(g.double())
        fin = torch.where(torch.isfinite(V), V, torch.zeros_like(V))
        _, reach = OP.attn_prompt(torch.nan_to_num(a.K[s][:, :L + n]), fin, L, torch.nan_to_num(a.q[off:off + n]), a.scale)
        if g is not None:
            reach = reach * torch.nan_to_num(torch.sigmoid(g.double()))
        noise, u = (4e-4, U[BF]) if a.dtype == BF else (8e-5, U[F32])
        same(a.out[off:off + n], ref, 2 * u * torch.nan_to_num(ref, 0, 0, 0).abs() + (u + noise) * reach + 1e-30,
             f"{what} sequence {s}")
        off += n


LAYOUTS = [(24, 4, 256, BF), (4, 4, 64, BF), (16, 2, 128, BF), (6, 2, 64, F32)]
BATCHES = [([150, 40], [30, 0]), ([24], [20000]), ([3, 70], [126, 5]), ([1], [400])]


@pytest.mark.parametrize("Hq,Hkv,D,dtype", LAYOUTS)
@pytest.mark.parametrize("rows,ctx", BATCHES)
def test_attn_prompt_far_gates(Hq, Hkv, D, dtype, rows, ctx):
    """Whole and split items: gates that are NaN, infinite or far out, each beside finite ones."""
    a = Attn(rows, ctx, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, gate=True, seed=41)
    n = sum(rows)
    for i, x in enumerate([NAN, INF, -INF, -50.0, -100.0, 100.0, -44.0, 3e38, -3e38]):
        for c in (2 * i, D - 1 - 2 * i):  # the pair's other half stays as it was
            a.gate[(7 * i) % n, i % Hq, c] = x
    a.gate[n - 1, Hq - 1, D // 2], a.gate[n - 1, Hq - 1, D // 2 + 1] = -INF, -INF
    a.gate[n - 1, 0, D // 2], a.gate[n - 1, 0, D // 2 + 1] = -60.0, -61.0
    a.run()
    check_attn(a)


@pytest.mark.parametrize("Hq,Hkv,D,dtype", LAYOUTS)
@pytest.mark.parametrize("rows,ctx", [([40], [500]), ([150, 9], [300, 400]), ([24], [20000]), ([1], [129]), ([200], [0]), ([3, 60], [254, 70])])
def test_attn_prompt_infinities_ahead_of_the_last_tile(Hq, Hkv, D, dtype, rows, ctx):
    """Infinities just before the last 128-position boundary, which a last tile that is not
    whole may load again: they come out as they are, not as NaN."""
    a = Attn(rows, ctx, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=43)
    for s, (L, n) in enumerate(zip(ctx, rows)):
        edge = (L + n - 1) // 128 * 128
        for c, back, x in ((0, 1, INF), (1, 1, -INF), (2, 1, NAN), (3, 9, INF), (D - 1, 30, -INF)):
            if edge - back >= 0:
                a.V[s][c % Hkv, edge - back, c] = x
    a.run()
    check_attn(a)


MEET = [([40], [500]), ([150, 9], [300, 400]), ([24], [20000])]


@pytest.mark.parametrize("Hq,Hkv,D,dtype", LAYOUTS)
@pytest.mark.parametrize("rows,ctx", MEET)
@pytest.mark.parametrize("gate", [False, True])
def test_attn_prompt_values_meet(Hq, Hkv, D, dtype, rows, ctx, gate):
    """Infinities of both signs and NaN, some seen by all rows, some by the later ones, in one column."""
    a = Attn(rows, ctx, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, gate=gate, seed=42)
    for s, (L, n) in enumerate(zip(ctx, rows)):
        V = a.V[s]
        for c, early, late in ((0, -INF, INF), (1, NAN, INF), (2, INF, INF), (3, INF, -INF), (D - 1, INF, None), (D - 2, None, -INF)):
            if early is not None:
                V[c % Hkv, 3, c] = early
            if late is not None:
                V[c % Hkv, L + n // 3, c] = late
        V[0, L + n - 1, 5], V[0, L + n // 2, 5] = -INF, INF
    a.q[rows[0] - 1, 0, 7] = NAN  # a row of one head, whatever its values are
    if gate:
        a.gate[:, :, 2] = -INF  # 0 times an infinity
        a.gate[rows[0] // 2:, :, D - 2] = NAN
        a.gate[:, :, 3] = INF
    a.run()
    check_attn(a)


@pytest.mark.parametrize("Hk,Hv,d,dtype", [(4, 8, 128, BF), (2, 2, 64, F32), (3, 6, 64, BF)])
@pytest.mark.parametrize("W", [1, 4, 5])
def test_gdn_prompt_front_far_inputs(Hk, Hv, d, dtype, W):
    """Infinities and far negative inputs beside ordinary ones: SiLU as the formula has it (x / (1 + e^-x),
    NaN from -inf), pairs of channels apart from each other."""
    rows = [37, 9]
    f = Front(rows, Hk, Hv, d, W, dtype, seed=44)
    Hc = 2 * Hk * d  # value channels: SiLU alone
    f.w[Hc:] = 0
    f.w[Hc:, W - 1] = 1.0  # the convolution of a value channel is its own row
    far = [-INF, INF, NAN, -50.0, -60.0, -43.0, -44.0, -80.0, -88.0, -100.0, -1e30, 1e30]
    for i, x in enumerate(far):
        f.x[3 * i, Hc + 2 * i] = x
        f.x[3 * i, Hc + d + 2 * i + 1] = x
    f.x[1, Hc + 8:Hc + 16] = torch.tensor([-50, -60, -70, -44, 1, -45, -46, -80.0]).to(dtype)
    old = [t.clone() for t in f.tails]
    f.run()
    torch.cuda.synchronize()
    assert f.prompt.status_code() == 0
    off = 0
    for s, n in enumerate(rows):
        sl = slice(off, off + n)
        own = f.x[sl, Hc:].double().reshape(n, Hv, d)
        ref = own / (1 + torch.exp(-own))
        if W > 1:  # (0 times an infinity of a row before, in the window)
            z = torch.cat([old[s], f.x[sl]])[:, Hc:].double()
            ref = ref + sum(0.0 * z[j:j + n] for j in range(W - 1)).reshape(n, Hv, d)
        # e^-x as 2^u, u = x log2(e): the product's rounding (2^-24 of u) and the constant's (2^-26, at most 2^-25
        # of u) change 2^u by ln 2 |u| (2^-24 + 2^-25) = 1.5 |x| 2^-24 of itself; exponential, sum, reciprocal and
        # products are within 16 steps
        bound = torch.nan_to_num(ref, 0, 0, 0).abs() * (U[dtype] + 2.0 ** -20 + torch.nan_to_num(own, 0, 0, 0).abs() * 2.0 ** -23)
        same(f.v[sl], ref, bound + 2.0 ** -119, "v")  # (sigmoids below 2^-126 are 0: at most 100 times that)
        off += n


@pytest.mark.parametrize("Hq,Hkv,D,dtype", LAYOUTS)
@pytest.mark.parametrize("rows,ctx,upto", [([40], [500], 33), ([40], [500], 130), ([40], [500], 510), ([70, 5], [0, 60], 40), ([24], [20000], 9000)])
def test_attn_prompt_scores_of_minus_infinity(Hq, Hkv, D, dtype, rows, ctx, upto):
    """Whole tiles and pieces of keys whose scores are -inf: no weight; a row that sees nothing else is NaN."""
    a = Attn(rows, ctx, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=45)
    a.q[:, :, 3] = a.q[:, :, 3].abs() + 0.1
    for s in range(len(rows)):
        a.K[s][0, :min(upto, ctx[s] + rows[s] - 1), 3] = -INF
    a.run()
    check_attn(a)
