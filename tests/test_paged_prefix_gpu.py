"""Prefixes that are read once for all members, where things go wrong or are not finite: entries that name no
page, the word, infinities and NaN among the shared rows, more query heads than an item holds, and captured
calls whose groups change between replays from sharing to not and back."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_tree_verify_masked_gb300 import binding as B
from speculative_tree_verify_masked_gb300.paged import PagedCaches
from tests.paged_helpers import Pools, f64

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ERR_ROWS, ERR_PAGE = 12, 13


def _shared(n=56, rows=2048, page=64, heads=(24, 4, 256), seed=0, first_idle=False):
    """n slots on `rows` shared rows (what they save is well above what sharing has to), some rows of their own each."""
    lens = [rows + 7 * i for i in range(n)]
    if first_idle:
        lens[0] = -1
    p = Pools(lens, page, heads, seed=seed, groups=[(n, rows)])
    assert (n - 2) * rows * 4 * heads[1] * heads[2] >= 1.05 * (200 << 20)
    return p


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("first_idle", [False, True])
def test_entries_that_name_no_page(page, first_idle):
    p = _shared(page=page, first_idle=first_idle)
    want = p.attn(p.gate, p.groups).clone()
    p.expect(want, p.gate, slots=[0, 1, 30, 55])
    assert p.status() == 0
    reads = 1 if first_idle else 0  # the member whose table names the prefix's pages
    for j in (0, 2048 // page // 2, 2048 // page - 1):
        keep = int(p.table[reads, j])
        for entry in (p.n_pages, -1, 1 << 30, -(1 << 31)):
            p.table[reads, j] = entry
            p.out.fill_(7.0)
            out = p.attn(p.gate, p.groups)
            assert p.status() == ERR_PAGE
            # (rows of shared prefixes are written by the join, which does nothing given the word)
            assert (out == 7).all()
            p.batch.status.zero_()
        p.table[reads, j] = keep
    p.out.fill_(7.0)
    assert torch.equal(p.attn(p.gate, p.groups), want) and p.status() == 0
    p.table[2, :2048 // page] = p.n_pages  # another member's entries of the prefix are not read
    assert torch.equal(p.attn(p.gate, p.groups), want) and p.status() == 0
    p.batch.status[0] = ERR_PAGE
    p.out.fill_(7.0)
    p.attn(p.gate, p.groups)
    assert (p.out == 7).all()


@pytest.mark.parametrize("heads,page", [((24, 4, 256), 64), ((16, 8, 128), 16), ((16, 16, 64), 128)])
def test_values_that_are_not_finite(heads, page):
    """Infinities and NaN among the shared rows reach the heads and columns that the formula lets them reach, in every member."""
    inf, nan = float("inf"), float("nan")
    p = _shared(heads=heads, page=page)
    G, D, n = heads[0] // heads[1], heads[2], len(p.lens)
    base = p.attn(None, p.groups).clone()

    def at(t):
        return p.rows[0][t // page], t % page

    pg, r = at(77)
    p.V[pg, 1, r, 5], p.V[pg, 1, r, 9] = inf, nan
    pg, r = at(2047)
    p.K[pg, 2, r, 0] = nan
    pg, r = at(1000)
    p.K[pg, 3, r, :] = inf  # scores of +inf and -inf, or NaN where products of both signs meet
    got = p.attn(None, p.groups)
    assert p.status() == 0
    assert (got[:, G:2 * G, 5] == inf).all() and got[:, G:2 * G, 9].isnan().all()
    assert got[:, 2 * G:3 * G].isnan().all()  # a NaN score
    assert got[:, 3 * G:4 * G].isnan().all()  # inf - inf
    keep = torch.ones(D, dtype=torch.bool, device="cuda")
    keep[[5, 9]] = False
    assert torch.equal(got[:, G:2 * G][:, :, keep], base[:, G:2 * G][:, :, keep])
    others = [h for h in range(heads[0]) if not G <= h < 4 * G]
    assert torch.equal(got[:, others], base[:, others])


@pytest.mark.parametrize("heads,page", [((24, 4, 256), 64), ((16, 8, 128), 32), ((16, 16, 64), 16)])
@pytest.mark.parametrize("first,last", [(0, 2048), (0, 1500), (0, 128), (640, 1920), (2047, 2048)])
def test_scores_of_minus_infinity(heads, page, first, last):
    """Shared keys whose every score is -inf have no weight: whole prefixes, whole pieces, tiles and a single row; an infinite
    value beside one of them is 0 times infinity."""
    p = _shared(heads=heads, page=page)
    p.q.copy_(p.q.abs() + 0.1)
    G = heads[0] // heads[1]
    for t in range(first, last):
        p.K[p.rows[0][t // page], 1, t % page] = -float("inf")
    got = p.attn(None, p.groups).clone()
    assert p.status() == 0 and got.isfinite().all()
    K, V, slots = p.K.clone(), p.V.clone(), (0, 1, 27, 55)
    # the rest of the rows alone, by the formula (the oracle's differences of infinities left out)
    Kh, Vh, q = f64(K[:, 1]), f64(V[:, 1]), f64(p.q)
    for s in slots:
        ids = p.rows[s][:p.lens[s] // page + 1]
        k, v = np.concatenate(Kh[ids])[:p.lens[s] + 1], np.concatenate(Vh[ids])[:p.lens[s] + 1]
        seen = np.ones(len(k), bool)
        seen[first:last] = False
        k, v = k[seen], v[seen]
        for h in range(G, 2 * G):
            w = k @ q[s, h] * p.scale
            prod = (np.abs(k) @ np.abs(q[s, h])).max() * p.scale
            w = np.exp(w - w.max())
            w /= w.sum()
            ref, mag = w @ v, w @ np.abs(v)
            # as Pools.expect: half a step of each weight and of the result, fp32 roundings of scores and sums
            tol = (2.0 ** -8 + 2.0 ** -24 * (2 * p.D * prod + p.lens[s] + 64)) * mag * 1.01 + 2.0 ** -8 * np.abs(ref) * 1.01
            assert (np.abs(f64(got[s, h]) - ref) <= tol).all(), (s, h)
    t = (first + last) // 2
    p.V[p.rows[0][t // page], 1, t % page, 3] = float("inf")
    out = p.attn(None, p.groups)
    assert out[:, G:2 * G, 3].isnan().all()
    out[:, G:2 * G, 3] = got[:, G:2 * G, 3]
    assert torch.equal(out, got) and p.status() == 0


@pytest.mark.parametrize("heads,n,rows,page", [((32, 1, 64), 120, 8192, 64), ((128, 1, 128), 60, 8192, 32), ((64, 2, 256), 30, 4096, 16),
                                               ((128, 1, 256), 30, 8192, 128), ((34, 2, 128), 60, 4096, 64)])
def test_more_query_heads_than_an_item(heads, n, rows, page):
    """Groups of more than sixteen query heads a KV head: several items of each slot joined with one prefix."""
    lens = [rows + (211 * i) % 900 for i in range(n)] + [50, -1, 3000]
    p = Pools(lens, page, heads, seed=n, groups=[(n, rows), (1, 0), (2, 0)])
    assert (n - 1) * rows * 4 * heads[1] * heads[2] >= 1.05 * (200 << 20)
    got = p.attn(p.gate, p.groups).clone()
    p.expect(got, p.gate, slots=[0, n // 2, n - 1, n, n + 1, n + 2])
    for _ in range(3):
        assert torch.equal(got, p.attn(p.gate, p.groups))
    assert p.status() == 0


# of a batch of 60 slots, 2,944 of whose rows are the same pages: groups, each allowed
STEPS = [([60, 0, 0], [2944, 0, 0]), ([60, 0, 0], [64, 0, 0]), ([20, 30, 10], [2944, 1024, 2944]), ([1, 58, 1], [2944, 2048, 0]),
         ([60, 0, 0], [0, 0, 0]), ([3, 54, 3], [1024, 2880, 64]), ([30, 0, 30], [2944, 0, 2944])]


@pytest.mark.parametrize("heads", [(24, 4, 256), (16, 8, 128)])
def test_captured_groups_change(heads):
    """One graph, captured where the groups share nothing, for groups that share much, little and nothing, of other sizes, with
    lengths and active slots that change: the bits of the call that is not captured, and the oracle's rows."""
    n, rows = 60, 2944
    p = Pools([rows + 3 * i for i in range(n)], 64, heads, groups=[(n, rows)], extra=200, max_len=4000, fill=None)
    g = B.PagedGroups([n, 0, 0], [0, 0, 0])
    assert (n - 1) * p.max_len * 4 * heads[1] * heads[2] >= 200 << 20  # (the kernel for prefixes is launched)
    ws, other = (p.space(B.tv_paged_attn_workspace_bytes(p.layer, p.batch, g)) for _ in range(2))
    out, stream = torch.empty_like(p.out), torch.cuda.Stream()
    torch.cuda.synchronize()
    B.tv_paged_attn(p.layer, p.batch, g, p.q, p.gate, out, p.scale, ws, stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        B.tv_paged_attn(p.layer, p.batch, g, p.q, p.gate, out, p.scale, ws, stream)
    for step, (sizes, shared) in enumerate(STEPS + STEPS[::-1]):
        g.set_groups(sizes, shared)
        for s in range(n):
            p.lens[s] = -1 if (s + step) % 17 == 16 else rows + (3 * s + 5 * step) % 190
        p.len.copy_(torch.tensor(p.lens, dtype=torch.int32))
        out.fill_(7.0)
        p.out.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        B.tv_paged_attn(p.layer, p.batch, g, p.q, p.gate, p.out, p.scale, other)
        assert torch.equal(out, p.out) and p.status() == 0, step
        p.expect(out, p.gate, slots=[0, (7 * step) % n, 59])
    # groups that are not allowed, found in a replay
    g.set_groups([60, 0, 0], [3968, 0, 0])
    out.fill_(7.0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert p.status() == ERR_ROWS and (out == 7).all()


def test_caches_share_prefixes_that_pay():
    """PagedCaches: 60 slots admitted on one's 2,048 rows, steps that are run and captured ones, against caches without groups."""
    Hq, Hkv, D, page, n = 24, 4, 256, 64, 60
    gen = torch.Generator(device="cuda").manual_seed(11)
    raw = lambda k, H: torch.randn((k, H, D), generator=gen, device="cuda").to(BF)
    first = [raw(2048, H) for H in (Hq, Hkv, Hkv)]

    def fresh():
        c = PagedCaches(1, 220, page, Hq, Hkv, D, n, 4000, rot_dims=64)
        c.admit(0)
        counts = [2048] + [0] * (n - 1)
        c.grow(counts)
        r = B.PagedRows(counts)
        c.append(0, r, *first, torch.empty_like(first[0]))
        c.advance(r)
        c.advanced(counts)
        for s in range(1, n):
            c.admit(s, like=0, rows=2048)
        return c

    a, b, plain = fresh(), fresh(), fresh()
    assert (n - 1) * 2048 * 4 * Hkv * D >= 1.05 * (200 << 20)
    ga, gb = a.groups([n, 0], [2048, 0]), b.groups([n, 0], [0, 0])
    xs = [{"q": raw(n, Hq), "k": raw(n, Hkv), "v": raw(n, Hkv), "gate": raw(n, Hq)} for _ in range(6)]
    x, y, z = ({**{k: torch.empty_like(t) for k, t in xs[0].items()}, "out": torch.zeros((n, Hq, D), dtype=BF, device="cuda")} for _ in range(3))
    stream, graph = torch.cuda.Stream(), None
    for i, new in enumerate(xs * 12):
        for k in new:
            for w in (x, y, z):
                w[k].copy_(new[k])
        sizes, shared = (([n, 0], [2048, 0]), ([40, 20], [2048, 0]), ([n, 0], [0, 0]), ([10, 50], [2048, 2048]))[i // 9 % 4]
        if i == 20:
            for c in (a, b, plain):
                c.retire(0)  # its pages stay with the others
        for g in (ga, gb):
            g.set_groups(sizes, shared)
        torch.cuda.synchronize()
        a.decode([x], ga)
        plain.decode([z])
        torch.cuda.synchronize()
        b.grow(stream=stream)
        if graph is None:
            with torch.cuda.stream(stream):
                b.layer(0, y, gb, stream)  # (warm; the same rows are written again)
                stream.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=stream):
                    b.layer(0, y, gb, stream)
                    b.advance(stream=stream)
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()
        b.advanced()
        assert torch.equal(x["out"], y["out"]) and a.lens == b.lens == b.len.tolist(), i
        # both sides round each weight and the output (half a step each), over values whose largest is under 6
        assert (x["out"].float() - z["out"].float()).abs().max() <= 4 * 2.0 ** -8 * 6
    assert a.status() == 0 and b.status() == 0 and plain.status() == 0


@pytest.mark.parametrize("sizes,shared", [([1] * 1024, [0] * 1024), ([2, 3, 5, 1, 0, 4] * 68 + [4], [512, 448, 320, 64, 512, 512] * 68 + [512]),
                                          ([700, 0, 324], [512, 64, 512])])
def test_as_many_slots_as_a_call_takes(sizes, shared):
    """1,024 slots in up to as many groups, more of both than a CTA has threads; idle ones among them."""
    n = sum(sizes)
    assert n == 1024
    lens = [512 + (i * 7) % 60 if i % 23 else -1 for i in range(n)]
    p = Pools(lens, 16, (4, 2, 128), groups=list(zip(sizes, shared)))
    saved = sum(max(0, sum(lens[i] >= 0 for i in range(a, a + m)) - 1) * x for a, m, x in
                zip([sum(sizes[:g]) for g in range(len(sizes))], sizes, shared)) * 2 * 128 * 4
    assert saved >= 1.05 * (200 << 20) or max(sizes) == 1
    got = p.attn(p.gate, p.groups).clone()
    p.expect(got, p.gate, slots=sorted({0, 1, 2, 23, 287, 288, 383, 384, 699, 700, 1022, 1023}))
    assert torch.equal(got, p.attn(p.gate, p.groups)) and p.status() == 0
    # all of them, beside the call that shares nothing: each side rounds every weight and the output, over values under 6
    plain = p.attn(p.gate).float()
    assert (got.float() - plain).abs().max() <= 4 * 2.0 ** -8 * 6
