"""Paged calls as they are used together: steps of several layers against contiguous
caches, shared prefixes, captured steps, two streams, errors that the device finds,
values that are not finite."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.paged as O
from speculative_tree_verify_masked_gb300 import binding as B
from speculative_tree_verify_masked_gb300.paged import PagedCaches
from tests.paged_helpers import HALF, Pools, f64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ERR = {"LEN": 10, "ROWS": 12, "PAGE": 13, "CAPACITY": 6}


def _raw(gen, n, H, D, dt=BF):
    return torch.randn((n, H, D), generator=gen, device="cuda").to(dt)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dtype,heads", [(BF, (24, 4, 256)), (BF, (8, 8, 64)), (F32, (4, 2, 128))])
def test_steps_equal_contiguous_caches(dtype, heads, page):
    """Two layers: prompts through the contiguous calls and into pages, then steps on both.  Rows of the caches are the
    same bits; outputs differ by the roundings of either side."""
    Hq, Hkv, D = heads
    gen = torch.Generator(device="cuda").manual_seed(page)
    prompts, n_slots = [70, 5, 129], 4  # slot 2 stays idle
    slots = [0, 1, 3]
    norms = [tuple(1 + 0.1 * torch.randn(D, generator=gen, device="cuda") for _ in range(2)) for _ in range(2)]
    c = PagedCaches(2, 64, page, Hq, Hkv, D, n_slots, 300, dtype, rot_dims=32, theta=1e6, norms=norms)
    for s in slots:
        c.admit(s)
    counts = [prompts[slots.index(s)] if s in slots else 0 for s in range(n_slots)]
    c.grow(counts)
    rows, n = B.PagedRows(counts), sum(counts)
    cap = 320
    flat = [[torch.zeros((Hkv, cap, D), dtype=dtype, device="cuda") for _ in slots] for _ in range(4)]
    layers = [B.AttnLayer(flat[2 * li], flat[2 * li + 1], Hq) for li in range(2)]
    ln = torch.zeros(3, dtype=torch.int32, device="cuda")
    prompt = B.Prompt(prompts)
    for li in range(2):
        q_raw, k_raw, v = _raw(gen, n, Hq, D, dtype), _raw(gen, n, Hkv, D, dtype), _raw(gen, n, Hkv, D, dtype)
        qa, qb = torch.empty_like(q_raw), torch.empty_like(q_raw)
        B.tv_attn_prompt_front(layers[li], prompt, ln, 0, *norms[li], 1e-6, 32, 1e6, q_raw, k_raw, v, qa)
        c.append(li, rows, q_raw, k_raw, v, qb)
        assert torch.equal(qa, qb)
    B.tv_prompt_advance(prompt, ln)
    c.advance(rows)
    c.advanced(counts)
    assert c.len.tolist() == [70, 5, -1, 129] == c.lens
    plan = B.plan(256)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    for step in range(20):  # over pages' ends
        inputs = []
        for li in range(2):
            x = {"q": _raw(gen, n_slots, Hq, D, dtype), "k": _raw(gen, n_slots, Hkv, D, dtype), "v": _raw(gen, n_slots, Hkv, D, dtype),
                 "gate": _raw(gen, n_slots, Hq, D, dtype), "out": torch.full((n_slots, Hq, D), 7.0, dtype=dtype, device="cuda")}
            inputs.append(x)
        want = []
        for li, x in enumerate(inputs):
            at = torch.tensor(slots, device="cuda")
            q, k = x["q"][at].contiguous(), x["k"][at].contiguous()
            B.tv_attn_norm_rope(layers[li], None, 3, ln, 300, *norms[li], 1e-6, 32, 1e6, q, k, q, k, status)
            out = torch.empty_like(q)
            ws = torch.empty(max(16, B.tv_attn_workspace_bytes(plan, layers[li], 3, 1, 300)), dtype=torch.uint8, device="cuda")
            B.tv_attn_decode_gated(plan, layers[li], 3, ln, 300, q, k, x["v"][at].contiguous(), x["gate"][at].contiguous(), out,
                                   D ** -0.5, ws, status)
            want.append(out)
        B.tv_len_advance(ln, None, 1, 3)
        c.decode(inputs)
        for li, x in enumerate(inputs):
            got = x["out"]
            assert (got[2] == 7).all()
            # both sides round weights (unless fp32) and outputs: twice the bound of one, over values of at most 5
            tol = (4 * HALF[dtype] * 5 if dtype == BF else 2e-5)
            assert (got[slots].float() - want[li].float()).abs().max() <= tol
    assert c.status() == 0 and int(status[0]) == 0
    for li in range(2):
        for i, s in enumerate(slots):
            L = prompts[i] + 20
            assert c.lens[s] == L
            for flat_x, pool in ((flat[2 * li][i], c.K[li]), (flat[2 * li + 1][i], c.V[li])):
                rows_ = torch.stack([pool[c.pages[s][t // page], :, t % page] for t in range(L)], 1)
                assert torch.equal(rows_, flat_x[:, :L])


def test_slots_come_and_go_with_shared_prefixes():
    """Slots admitted on another's pages decode as if they had rows of their own; pages come back when the last leaves."""
    Hq, Hkv, D, page = 24, 4, 256, 16
    gen = torch.Generator(device="cuda").manual_seed(3)
    c = PagedCaches(1, 120, page, Hq, Hkv, D, 6, 500)
    c.admit(0)
    counts = [100, 0, 0, 0, 0, 0]
    c.grow(counts)
    q_raw, k_raw, v = (_raw(gen, 100, H, D) for H in (Hq, Hkv, Hkv))
    c.append(0, B.PagedRows(counts), q_raw, k_raw, v, torch.empty_like(q_raw))
    c.advance(B.PagedRows(counts))
    c.advanced(counts)
    for s in (1, 2, 4):
        c.admit(s, like=0, rows=96)
    with pytest.raises(ValueError):
        c.admit(1)
    with pytest.raises(ValueError):
        c.admit(3, like=0, rows=90)
    with pytest.raises(ValueError):
        c.admit(3, like=0, rows=112)
    groups = c.groups([3, 3], [96, 0])
    for step in range(40):
        x = {"q": _raw(gen, 6, Hq, D), "k": _raw(gen, 6, Hkv, D), "v": _raw(gen, 6, Hkv, D),
             "out": torch.empty((6, Hq, D), dtype=BF, device="cuda")}
        c.decode([x], groups)
        if step % 13 == 0:
            K, V = f64(c.K[0]), f64(c.V[0])
            for s in (0, 1, 2, 4) if step < 21 else (1, 2, 4):  # (slot 0 has left)
                ref, mag, prod = O.attend(K, V, c.pages[s], c.lens[s] - 1, f64(c.q[s]), c.scale)
                tol = HALF[BF] * 1.01 * (mag + np.abs(ref)) + 2.0 ** -24 * (2 * D * prod + 600) * mag
                assert (np.abs(f64(x["out"][s]) - ref) <= tol).all()
        if step == 20:
            c.retire(0)  # its first pages stay with the others
    assert c.status() == 0
    used = sum(len(set(c.pages[s])) for s in (1, 2, 4)) - 2 * 6
    assert len(c.free) == 120 - used
    for s in (1, 2, 4):
        c.retire(s)
    assert sorted(c.free) == list(range(120)) and not any(c.users)
    c.admit(5)
    with pytest.raises(ValueError):
        c.grow([0, 0, 0, 0, 0, 502])
    for s in range(5):
        c.admit(s)
    with pytest.raises(MemoryError):
        c.grow([400] * 6)
    assert len(c.free) == 120  # nothing was taken


def test_sparse_steps():
    """Steps that look at a few pages alone: the choice and the outputs against the oracle, with bounds kept step by step."""
    Hq, Hkv, D, page, n_sel = 12, 2, 128, 16, 6
    gen = torch.Generator(device="cuda").manual_seed(9)
    c = PagedCaches(1, 200, page, Hq, Hkv, D, 3, 400, sparse=(n_sel, 1, 2), rot_dims=64)
    counts = [210, 0, 47]
    for s in (0, 2):
        c.admit(s)
    c.grow(counts)
    q_raw, k_raw, v = (_raw(gen, 257, H, D) for H in (Hq, Hkv, Hkv))
    rows = B.PagedRows(counts)
    c.append(0, rows, q_raw, k_raw, v, torch.empty_like(q_raw))
    c.advance(rows)
    c.advanced(counts)
    for step in range(36):
        x = {"q": _raw(gen, 3, Hq, D), "k": _raw(gen, 3, Hkv, D), "v": _raw(gen, 3, Hkv, D), "gate": _raw(gen, 3, Hq, D),
             "out": torch.empty((3, Hq, D), dtype=BF, device="cuda")}
        c.decode([x])
        if step % 5:
            continue
        K, V, q = f64(c.K[0]), f64(c.V[0]), f64(c.q)
        for s in (0, 2):
            L = c.lens[s] - 1
            nb = L // page + 1
            places = []
            for g in range(Hkv):
                ids = c.pages[s][1:nb - 2]
                code, e = zip(*(O.bounds(K[p, g]) for p in ids)) if nb > n_sel else ((), ())
                places.append(O.select(q[s, g * 6:g * 6 + 6], np.array(code), np.array(e), nb, 1, 2, n_sel))
                got = c.sel[s, g, :int(c.count[s, g])].tolist()
                assert got == places[-1], (step, s, g)
            ref, mag, prod = O.attend(K, V, c.pages[s], L, q[s], c.scale, f64(x["gate"][s]), places)
            tol = HALF[BF] * 1.01 * (mag + np.abs(ref)) + 2.0 ** -24 * (2 * D * prod + 600) * mag
            assert (np.abs(f64(x["out"][s]) - ref) <= tol).all()
    assert c.status() == 0


def test_slots_up_to_their_bound():
    """A slot takes max_len rows and no more; a full one beside it troubles no other slot; idle ones get no pages."""
    page, Hq, Hkv, D = 16, 4, 2, 64
    c = PagedCaches(1, 40, page, Hq, Hkv, D, 3, 64, sparse=(3, 1, 1))
    gen = torch.Generator(device="cuda").manual_seed(0)

    def prompt(counts):
        c.grow(counts)
        n = sum(counts)
        r = B.PagedRows(counts)
        q = _raw(gen, n, Hq, D)
        c.append(0, r, q, _raw(gen, n, Hkv, D), _raw(gen, n, Hkv, D), q)
        c.advance(r)
        c.advanced(counts)

    c.admit(0)
    c.admit(1)
    for bad in ([65, 0, 0], [0, 0, 1], [1, 0], [1, -1, 0]):
        with pytest.raises(ValueError):
            c.grow(bad)
    assert len(c.free) == 40
    prompt([64, 3, 0])
    with pytest.raises(ValueError):
        c.grow([1, 0, 0])
    prompt([0, 20, 0])
    assert c.lens == [64, 23, -1] and c.len.tolist() == [64, 23, -1] and c.status() == 0
    with pytest.raises(ValueError):
        c.decode([])  # the full slot would take a row
    c.retire(0)
    out = torch.full((3, Hq, D), 7.0, dtype=BF, device="cuda")
    c.decode([{"q": _raw(gen, 3, Hq, D), "k": _raw(gen, 3, Hkv, D), "v": _raw(gen, 3, Hkv, D), "out": out}])
    assert c.lens == [-1, 24, -1] and c.len.tolist() == [-1, 24, -1] and c.status() == 0
    assert (out[[0, 2]] == 7).all() and out[1].isfinite().all()


def test_groups_after_a_capture():
    """Groups that need a larger workspace leave the one of captured steps where it is."""
    page, Hq, Hkv, D = 64, 24, 4, 256
    c = PagedCaches(1, 20, page, Hq, Hkv, D, 2, 500)
    ws = c.ws
    c.groups([2], [0])
    assert c.ws.numel() > ws.numel() and any(x is ws for x in c.outgrown)


@pytest.mark.parametrize("sparse", [None, (5, 1, 1)])
def test_captured_steps(sparse):
    """One graph serves steps whose lengths, pages, active slots and groups change between replays."""
    Hq, Hkv, D, page, n = 24, 4, 256, 32, 5
    gen = torch.Generator(device="cuda").manual_seed(4)

    def fresh():
        c = PagedCaches(1, 100, page, Hq, Hkv, D, n, 600, sparse=sparse, rot_dims=64)
        for s in (0, 1, 3):
            c.admit(s)
        return c

    xs = [{"q": _raw(gen, n, Hq, D), "k": _raw(gen, n, Hkv, D), "v": _raw(gen, n, Hkv, D)} for _ in range(80)]
    a, b = fresh(), fresh()
    ga, gb = (None, None) if sparse else (a.groups([2, 3], [0, 0]), b.groups([2, 3], [0, 0]))
    x = {k: torch.empty_like(t) for k, t in xs[0].items()}
    x["out"] = torch.zeros((n, Hq, D), dtype=BF, device="cuda")
    y = {**{k: torch.empty_like(t) for k, t in xs[0].items()}, "out": torch.zeros((n, Hq, D), dtype=BF, device="cuda")}
    stream = torch.cuda.Stream()
    graph = None
    for i, new in enumerate(xs):
        for k in new:
            x[k].copy_(new[k])
            y[k].copy_(new[k])
        if i == 30:
            for c in (a, b):
                c.retire(1)
                c.admit(4, like=0, rows=0)
        if i == 40:
            for c in (a, b):
                c.admit(2, like=3, rows=32)
            if ga:
                for g in (ga, gb):
                    g.set_groups([2, 3], [0, 0])
        torch.cuda.synchronize()
        a.decode([x], ga)  # eager
        torch.cuda.synchronize()
        b.grow(stream=stream)
        if graph is None:
            with torch.cuda.stream(stream):
                b.layer(0, y, gb, stream)  # (warm)
                stream.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=stream):
                    b.layer(0, y, gb, stream)
                    b.advance(stream=stream)
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()
        b.advanced()
        assert torch.equal(x["out"], y["out"]) and a.len.tolist() == b.len.tolist() == a.lens, i
    assert a.status() == 0 and b.status() == 0


def test_two_streams_at_once():
    """Calls on two streams with workspaces of their own, many times: the bits of each alone."""
    ps = [Pools([3000 + 700 * i, 64, 900], 64, (24, 4, 256), seed=i) for i in range(2)] + \
         [Pools([1024 + i % 7 for i in range(60)], 32, (24, 4, 256), seed=5, groups=[(60, 1024)])]
    want = [p.attn(p.gate, p.groups).clone() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    spaces = [p.space(B.tv_paged_attn_workspace_bytes(p.layer, p.batch, p.groups)) for p in ps]
    torch.cuda.synchronize()
    for _ in range(100):
        for p, st, ws in zip(ps, streams, spaces):
            B.tv_paged_attn(p.layer, p.batch, p.groups, p.q, p.gate, p.out, p.scale, ws, st)
    torch.cuda.synchronize()
    for p, w in zip(ps, want):
        assert torch.equal(p.out, w) and p.status() == 0


@pytest.mark.parametrize("groups", [False, True])
def test_bad_lengths_and_pages(groups):
    p = Pools([100, 200, 300], 32, (24, 4, 256), max_len=320, groups=[(3, 96)] if groups else ())
    g = p.groups
    for L in (-2, 321, 1 << 30):
        p.len[1] = L
        p.attn(None, g)
        assert p.status() == ERR["LEN"]
        p.out.fill_(7.0)
        p.attn(None, g)  # a call that is given the word does nothing
        assert (p.out == 7).all()
        p.batch.status.zero_()
    p.len[1] = 200
    for bad in (-1, p.n_pages, 1 << 30, -(1 << 31)):
        keep = int(p.table[2, 7])
        p.table[2, 7] = bad
        p.attn(None, g)
        assert p.status() == ERR["PAGE"]
        p.table[2, 7] = keep
        p.batch.status.zero_()
    p.expect(p.attn(None, g))
    assert p.status() == 0
    # entries behind the last page are not read
    p.table[0, 4:] = 1 << 30
    p.expect(p.attn(None, g))
    assert p.status() == 0


@pytest.mark.parametrize("off,shared", [([1, 3], [64]), ([0, 2], [64]), ([0, 4], [64]), ([0, 3], [48]), ([0, 3], [-32]), ([0, 3], [128]),
                                        ([0, 2, 1, 3], [0, 0, 0]), ([0, 2, 3], [64, 320])])
@pytest.mark.parametrize("many", [1, 400])
def test_bad_groups(off, shared, many):
    """Offsets and prefixes that are not allowed, in calls that share and in calls that only check."""
    p = Pools([100, 200, 300], 32, (24, 4, 256), max_len=320 * many, groups=[(3, 96)])
    g = B.PagedGroups([3] + [0] * (len(shared) - 1), [0] * len(shared))
    g.group_off.copy_(torch.tensor(off, dtype=torch.int32))
    g.shared.copy_(torch.tensor(shared, dtype=torch.int32))
    p.attn(None, g)
    assert p.status() == ERR["ROWS"] and (p.out == 7).all()


def test_bad_selections():
    p = Pools([100, 200, -1], 32, (24, 4, 256), max_len=320)
    sel = torch.zeros(3, 4, 5, dtype=torch.int32, device="cuda")
    count = torch.full((3, 4), 2, dtype=torch.int32, device="cuda")
    sel[:, :, 1] = 1
    for c in (-1, 6, 1 << 30):
        count[1, 2] = c
        p.selected(sel, count)
        assert p.status() == ERR["ROWS"]
        p.batch.status.zero_()
        count[1, 2] = 2
    for j in (-1, p.table.shape[1], 1 << 30):
        sel[0, 3, 1] = j
        p.selected(sel, count)
        assert p.status() == ERR["PAGE"]
        p.batch.status.zero_()
        sel[0, 3, 1] = 1
    count[2] = 99  # an idle slot's is not read
    p.selected(sel, count)
    assert p.status() == 0


def test_bad_appends():
    p = Pools([100, -1, 300], 32, (4, 2, 64), max_len=319, cols=10, fill=None)
    q_raw, k_raw, v = (torch.randn(20, H, 64, device="cuda").to(BF) for H in (4, 2, 2))
    q = torch.empty_like(q_raw)

    def append(off, n_total=20, n_max=20):
        r = B.PagedRows([5, 0, 5], n_total=n_total, n_max=n_max)
        r.row_off.copy_(torch.tensor(off, dtype=torch.int32))
        K0, V0 = p.K.clone(), p.V.clone()
        B.tv_paged_append(p.layer, p.batch, r, None, None, 0.0, 8, 1e4, q_raw, k_raw, v, q)
        code = p.status()
        p.batch.status.zero_()
        return code, torch.equal(K0, p.K) and torch.equal(V0, p.V)

    for off in ([1, 5, 5, 10], [0, 5, 5, 21], [0, 0, 5, 5]):  # (the last: rows of an idle slot)
        assert append(off) == (ERR["ROWS"], True)
    assert append([0, 3, 3, 13], n_max=9)[0] == ERR["ROWS"]
    assert append([0, 0, 0, 20])[0] == 0        # rows 300 .. 319: the table's last
    p.len[2] = 301
    assert append([0, 0, 0, 20])[0] == ERR["CAPACITY"]
    p.len[2] = 320
    assert append([0, 0, 0, 1])[0] == ERR["LEN"]
    p.len[2] = 300
    keep = int(p.table[0, 3])
    p.table[0, 3] = p.n_pages
    assert append([0, 1, 1, 1]) == (ERR["PAGE"], True)
    p.table[0, 3] = keep
    assert append([0, 1, 1, 1])[0] == 0
    # bounds and the advance refuse alike
    code, exp = torch.zeros(p.n_pages, 2, 2, 64, dtype=torch.int8, device="cuda"), torch.zeros(p.n_pages, 2, dtype=torch.int32, device="cuda")
    r = B.PagedRows([60, 0, 0], n_total=60, n_max=60)
    r.row_off.copy_(torch.tensor([0, 61, 61, 61], dtype=torch.int32))
    B.tv_paged_bounds(p.layer, p.batch, r, code, exp)
    assert p.status() == ERR["ROWS"] and not code.any()
    p.batch.status.zero_()
    B.tv_paged_advance(p.batch, r)
    assert p.status() == ERR["ROWS"] and p.len.tolist()[0] == 100


def test_rows_that_are_not_finite():
    """Infinities and NaN among rows that are seen reach what the formula lets them reach, and no more."""
    inf, nan = float("inf"), float("nan")
    p = Pools([500, 500, 500, 40], 32, (24, 4, 256), seed=6)
    base = p.attn().clone()

    def page_row(s, t):
        return p.rows[s][t // 32], t % 32

    pg, r = page_row(0, 77)
    p.V[pg, 1, r, 5] = inf       # slot 0, heads 6 .. 11, column 5: infinite
    p.V[pg, 1, r, 9] = nan       # column 9: NaN
    pg, r = page_row(1, 300)
    p.K[pg, 2, r, 0] = nan       # slot 1, heads 12 .. 17: NaN throughout
    got = p.attn()
    assert (got[0, 6:12, 5] == inf).all() and got[0, 6:12, 9].isnan().all()
    keep = torch.ones(256, dtype=torch.bool, device="cuda")
    keep[[5, 9]] = False
    assert torch.equal(got[0, 6:12][:, keep], base[0, 6:12][:, keep])
    others = [h for h in range(24) if not 6 <= h < 12]
    assert torch.equal(got[0, others], base[0, others])
    assert got[1, 12:18].isnan().all()
    others = [h for h in range(24) if not 12 <= h < 18]
    assert torch.equal(got[1, others], base[1, others])
    assert torch.equal(got[2:], base[2:])
    assert p.status() == 0


def test_scores_of_minus_infinity():
    """Keys whose every score is -inf have no weight; a row with nothing else is 0 / 0."""
    p = Pools([200, 90], 16, (8, 2, 64), seed=7)
    p.q[:] = p.q.abs() + 0.1
    for t in range(0, 150):
        p.K[p.rows[0][t // 16], :, t % 16] = -float("inf")
    for t in range(0, 91):
        p.K[p.rows[1][t // 16], 1, t % 16] = -float("inf")
    got = f64(p.attn())
    K, V, q = f64(p.K), f64(p.V), f64(p.q)
    with np.errstate(invalid="ignore"):
        for h in range(8):
            g = h // 4
            k, v = (np.concatenate([x[p.rows[0][j], g] for j in range(13)])[150:201] for x in (K, V))
            w = np.exp((k @ q[0, h]) * p.scale)
            ref = (w / w.sum()) @ v
            assert np.abs(got[0, h] - ref).max() <= 2 * HALF[BF] * 1.1 * np.abs(v).max()
    assert np.isfinite(got[1, :4]).all() and np.isnan(got[1, 4:]).all()
    assert p.status() == 0


@pytest.mark.parametrize("dtype,heads,lens", [(F32, (4, 2, 64), [300, 90]), (BF, (24, 4, 256), [20000, 70]), (BF, (16, 2, 128), [9000, 500])])
def test_infinite_values_without_weight(dtype, heads, lens):
    """An infinite value whose score is -inf is 0 times infinity wherever it lies: among scores of -inf alone, too."""
    for slot, first, n in ((0, 0, 8), (0, lens[0] // 8, lens[0] // 4), (1, 40, 8)):
        p = Pools(lens, 32, heads, dtype, seed=9)
        p.q[:] = p.q.abs() + 0.1
        for t in range(first, first + n):
            p.K[p.rows[slot][t // 32], 1, t % 32] = -float("inf")
        pg, r = p.rows[slot][(first + n // 2) // 32], (first + n // 2) % 32
        p.V[pg, 1, r, 3] = float("inf")
        got, G = p.attn(), heads[0] // heads[1]
        assert got[slot, G:2 * G, 3].isnan().all()
        got[slot, G:2 * G, 3] = 0
        assert got.isfinite().all() and p.status() == 0


def test_far_pages():
    """Offsets in the pools past 2^31 bytes and elements."""
    Hkv, page, D = 4, 128, 256
    n_pages = 17000  # 2.2e9 elements a pool
    K, V = (torch.empty(n_pages, Hkv, page, D, dtype=BF, device="cuda") for _ in range(2))
    ids = [n_pages - 1, 16500, 3, n_pages - 2]
    gen = torch.Generator(device="cuda").manual_seed(8)
    for i in ids:
        K[i], V[i] = (torch.randn((Hkv, page, D), generator=gen, device="cuda").to(BF) for _ in range(2))
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    L = 3 * page + 50
    layer, batch = B.PagedLayer(K, V, 24), B.PagedBatch(table, torch.tensor([L], dtype=torch.int32, device="cuda"), L)
    k_raw, v, q_raw = (torch.randn((1, H, D), generator=gen, device="cuda").to(BF) for H in (4, 4, 24))
    q = torch.empty_like(q_raw)
    B.tv_paged_append(layer, batch, None, None, None, 0.0, 0, 1e4, q_raw, k_raw, v, q)
    assert torch.equal(K[ids[3], :, 50], k_raw[0]) and torch.equal(V[ids[3], :, 50], v[0]) and torch.equal(q, q_raw)
    out = torch.empty_like(q)
    ws = torch.empty(B.tv_paged_attn_workspace_bytes(layer, batch), dtype=torch.uint8, device="cuda")
    B.tv_paged_attn(layer, batch, None, q, None, out, 0.0625, ws)
    Ks, Vs = f64(K[ids]), f64(V[ids])
    ref, mag, prod = O.attend(Ks, Vs, [0, 1, 2, 3], L, f64(q[0]), 0.0625)
    assert (np.abs(f64(out[0]) - ref) <= HALF[BF] * 1.01 * (mag + np.abs(ref)) + 2.0 ** -24 * (512 * prod + 600) * mag).all()
    code = torch.zeros(n_pages, Hkv, 2, D, dtype=torch.int8, device="cuda")
    exp = torch.zeros(n_pages, Hkv, dtype=torch.int32, device="cuda")
    batch.len.fill_(0)
    B.tv_paged_bounds(layer, batch, B.PagedRows([3 * page]), code, exp)
    for i in ids[:3]:
        for g in range(Hkv):
            want, e = O.bounds(f64(K[i, g]))
            assert int(exp[i, g]) == e and (code[i, g].cpu().numpy() == want).all()
    assert batch.status_code() == 0
