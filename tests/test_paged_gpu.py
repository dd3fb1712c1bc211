"""Calls over caches in pages against the fp64 oracle: types, head layouts, page
sizes, lengths from zero to long ones, idle slots, what no slot sees set to NaN."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.paged as O
from speculative_tree_verify_masked_gb300 import binding as B
from tests.paged_helpers import HALF, Pools, f64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HEADS = [(24, 4, 256), (16, 2, 128), (8, 8, 64), (32, 1, 64), (2, 1, 256), (128, 1, 128), (3, 3, 128)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", HEADS)
def test_attn_lengths(heads, page):
    p = Pools([0, 1, page - 1, page, -1, 63, 64, 500, 130, 127], page, heads, seed=page)
    p.expect(p.attn())
    assert p.status() == 0


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("heads", [(2, 1, 64), (8, 2, 128), (6, 2, 256)])
def test_attn_fp32(heads, page):
    p = Pools([0, 1, page - 1, page, -1, 200, 31], page, heads, F32, seed=page)
    p.expect(p.attn())
    p.expect(p.attn(p.gate), p.gate)
    assert p.status() == 0


@pytest.mark.parametrize("heads", HEADS[:4])
def test_attn_gate(heads):
    p = Pools([5, 70, -1, 1000], 32, heads, seed=3)
    p.expect(p.attn(p.gate), p.gate)
    g = p.gate.clone()
    p.expect(p.attn(p.gate), g)  # (again, from the same buffers)
    p.out = p.gate  # the gate's own memory
    ws = p.space(B.tv_paged_attn_workspace_bytes(p.layer, p.batch, None))
    B.tv_paged_attn(p.layer, p.batch, None, p.q, p.gate, p.out, p.scale, ws)
    p.expect(p.out, g, slots=[0, 1, 3])


@pytest.mark.parametrize("heads,lens", [((24, 4, 256), [20000]), ((8, 8, 64), [9001, 3]), ((16, 2, 128), [70] * 150),
                                        ((24, 4, 256), [0] * 40), ((2, 1, 128), list(range(300))), ((24, 4, 256), [12000, 1, 1, 900])])
def test_attn_splits(heads, lens):
    """One long slot over every CTA, many short ones, cuts at uneven places."""
    p = Pools(lens, 64, heads, seed=len(lens))
    p.expect(p.attn(), slots=range(0, len(lens), max(1, len(lens) // 12)))
    assert p.status() == 0


@pytest.mark.parametrize("heads,n,most", [((24, 4, 256), 200, 255), ((24, 4, 256), 3, 255), ((16, 2, 128), 90, 254), ((40, 2, 64), 70, 511),
                                          ((8, 8, 64), 40, 511), ((34, 2, 256), 60, 100), ((8, 1, 128), 500, 40)])
@pytest.mark.parametrize("idle", [0, 1])
def test_attn_items_uncut(heads, n, most, idle):
    """Slots short enough for ranges that end with items: more items than CTAs and fewer, idle slots in runs."""
    rng = np.random.default_rng(n + most)
    lens = rng.integers(0, most + 1, n)
    lens[rng.integers(0, n)] = most
    if idle:
        lens[n // 4:n - n // 4] = -1
    p = Pools(lens.tolist(), 32, heads, seed=n)
    p.expect(p.attn())
    assert p.status() == 0


@pytest.mark.parametrize("heads,page", [((24, 4, 256), 64), ((16, 2, 128), 32), ((8, 8, 64), 128)])
def test_attn_long_pieces(heads, page):
    """Hundreds of tiles a CTA, some from memory and some from L2: copies land out of order."""
    p = Pools([8192 + 13 * i for i in range(48)], page, heads, seed=4, groups=[(48, 8192)])
    first = p.attn().clone()
    p.expect(first, slots=(0, 20, 47))
    for _ in range(20):
        assert torch.equal(first, p.attn())
    assert p.status() == 0


# (small savings are left alone: 200 MB of keys and values of a 24 + 4 head layer of 256 are 51,200 rows)
GROUPS = [
    ("one group", [2048 + 7 * i for i in range(56)], [(56, 2048)]),
    ("groups and lone slots", [700] * 20 + [5, 64] + [1300] * 60 + [30] + [2000] * 3, [(20, 640), (1, 0), (1, 64), (60, 1280), (1, 0), (3, 1920)]),
    ("idle members, an empty group", [-1, 400, 384, -1] + [2500] * 50 + [-1, 300, 384, -1], [(3, 384), (0, 128), (52, 2432), (3, 0)]),
    ("one active member", [-1, 6000, -1] + [2600] * 40, [(3, 5888), (40, 2560)]),
    ("nothing shared", [400, 0, 1, -1], [(2, 0), (2, 0)]),
    ("too little shared", [400, 300, 280], [(3, 256)]),
    ("long", [20000 + 128 * 3 + i for i in range(9)], [(9, 19968)]),
    ("many groups", [1024 + i % 3 for i in range(240)], [(4, 1024)] * 60),
]


@pytest.mark.parametrize("name,lens,groups", GROUPS, ids=[g[0] for g in GROUPS])
@pytest.mark.parametrize("heads,page", [((24, 4, 256), 64), ((24, 4, 256), 16), ((16, 8, 128), 32), ((16, 8, 128), 128), ((16, 16, 64), 64),
                                        ((40, 4, 256), 16)])
def test_attn_groups(heads, page, name, lens, groups):
    if page == 128:
        groups = [(m, s // 128 * 128) for m, s in groups]
    p = Pools(lens, page, heads, seed=page, groups=groups)
    slots = [i for i in range(len(lens)) if i < 3 or i % 13 == 0 or lens[i] < 100]
    gate = p.gate if "long" in name else None
    p.expect(p.attn(gate, p.groups), gate, slots=slots)
    got = p.out.clone()
    p.out.fill_(7.0)
    for _ in range(3):
        assert torch.equal(got, p.attn(gate, p.groups))
    assert p.status() == 0


def test_attn_groups_prefix_tiles_end_inside():
    """Prefixes that end at every page of a tile of keys, in tiles cut in two and three rows of queries."""
    for n in range(64, 73):
        lens = [16 * n + i % 50 for i in range(90)]
        p = Pools(lens, 16, (24, 4, 256), seed=n, groups=[(90, 16 * n)])
        p.expect(p.attn(None, p.groups), slots=(0, 21, 42, 89))
        assert p.status() == 0


def test_attn_groups_fp32():
    p = Pools([300, 256, 256 + 17], 32, (4, 2, 128), F32, groups=[(3, 256)])
    p.expect(p.attn(p.gate, p.groups), p.gate)


def test_attn_many_slots():
    p = Pools([(i * 37) % 90 for i in range(1024)], 16, (4, 2, 64), seed=1)
    p.expect(p.attn(), slots=range(0, 1024, 53))
    assert p.status() == 0


def _append(p, rows, norm, rot, theta=1e7, seed=0, in_place=False):
    n = p.batch.n_seq if rows is None else rows.n_total
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    q_raw, k_raw, v = ((r(n, H, p.D) * c).to(p.dtype) for H, c in ((p.Hq, 3), (p.Hkv, 0.5), (p.Hkv, 1)))
    wq, wk = (1 + 0.1 * r(p.D), 1 + 0.1 * r(p.D)) if norm else (None, None)
    q = q_raw.clone() if in_place else torch.full_like(q_raw, 7.0)
    B.tv_paged_append(p.layer, p.batch, rows, wq, wk, 1e-6, rot, theta, q if in_place else q_raw, k_raw, v, q)
    return q_raw, k_raw, v, wq, wk, q


def _check_append(p, lens, counts, packed, K0, V0, q_raw, k_raw, v, wq, wk, q, rot, theta=1e7):
    """Rows in their places and nothing else changed (bit for bit)."""
    want_K, want_V, at = K0.clone(), V0.clone(), 0
    for i, (L, n) in enumerate(zip(lens, counts)):
        a = at if packed else i
        at += n
        if L < 0 or n == 0:
            continue
        pos = np.arange(L, L + n)
        yq, yk = O.append(f64(q_raw[a:a + n]), f64(k_raw[a:a + n]), pos, None if wq is None else f64(wq),
                          None if wk is None else f64(wk), 1e-6, rot, theta)
        got_k = torch.stack([p.K[p.rows[i][x // p.page], :, x % p.page] for x in pos])
        for y, got in ((yq, q[a:a + n]), (yk, got_k)):
            # the rounding, and some ten fp32 steps of the head's largest value (norm, angle, products)
            tol = HALF[p.dtype] * np.abs(y) * 1.01 + 16 * 2.0 ** -24 * np.abs(y).max(-1, keepdims=True) + 1e-37
            assert (np.abs(f64(got) - y) <= tol).all(), (i, float((np.abs(f64(got) - y) - tol).max()))
        for x in pos:
            want_K[p.rows[i][x // p.page], :, x % p.page] = p.K[p.rows[i][x // p.page], :, x % p.page]
            want_V[p.rows[i][x // p.page], :, x % p.page] = v[a + x - L]
    bits = torch.int16 if p.dtype == BF else torch.int32
    assert torch.equal(p.K.view(bits), want_K.view(bits)) and torch.equal(p.V.view(bits), want_V.view(bits))
    assert p.status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads,rot,norm", [((24, 4, 256), 64, True), ((16, 2, 128), 128, True), ((8, 8, 64), 6, False), ((2, 1, 64), 0, True)])
def test_append_step(dtype, heads, rot, norm):
    lens = [0, 131071, -1, 15, 16, 63, 64, 4000, -1]
    p = Pools([-1] * len(lens), 16, heads, dtype, max_len=131071, cols=8192, spare=len(lens))
    for i, L in enumerate(lens):  # each slot's page of its next row, and no other
        if L >= 0:
            p.rows[i][L // 16] = i
    p.table.copy_(torch.tensor(p.rows, dtype=torch.int32))
    p.len.copy_(torch.tensor(lens, dtype=torch.int32))
    K0, V0 = p.K.clone(), p.V.clone()
    x = _append(p, None, norm, rot)
    _check_append(p, lens, [int(L >= 0) for L in lens], False, K0, V0, *x, rot)
    assert (x[5][2] == 7).all() and (x[5][8] == 7).all()  # idle slots' rows


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("n_seq", [4, 40, 65])
def test_append_rows(dtype, page, n_seq):
    lens = [(i * 29) % 200 if i % 7 else 0 for i in range(n_seq)]
    counts = [(0, 1, 17, 130)[i % 4] for i in range(n_seq)]
    lens[4 % n_seq] = -1 if n_seq > 4 else lens[0]
    p = Pools(lens, page, (8, 2, 128), dtype, extra=130, max_len=max(lens), fill=None)
    n = sum(counts)
    rows = B.PagedRows(counts, n_total=n + 5)  # five rows of padding
    K0, V0 = p.K.clone(), p.V.clone()
    x = _append(p, rows, True, 64, in_place=n_seq == 40)
    if n_seq == 40:  # in place: form it apart, too, and compare
        y = _append(p, rows, True, 64)
        assert torch.equal(x[5][:n], y[5][:n]) and (y[5][n:] == 7).all()
        x = y
    _check_append(p, lens, counts, True, K0, V0, *x, 64)
    assert (x[5][n:] == 7).all()


def test_append_equals_contiguous():
    """The rows that tv_attn_prompt_front writes, bit for bit, in pages."""
    lens, counts = [100, 0, 7], [33, 64, 5]
    p = Pools(lens, 32, extra=64, fill=None)
    K, V = ([torch.zeros(4, 256, 256, dtype=BF, device="cuda") for _ in lens] for _ in range(2))
    x = _append(p, B.PagedRows(counts), True, 64)
    q = torch.empty_like(x[0])
    B.tv_attn_prompt_front(B.AttnLayer(K, V, 24), B.Prompt(counts), p.len, p.max_len, x[3], x[4], 1e-6, 64, 1e7, x[0], x[1], x[2], q)
    assert torch.equal(q, x[5])
    for i, (L, n) in enumerate(zip(lens, counts)):
        for t in range(L, L + n):
            assert torch.equal(K[i][:, t], p.K[p.rows[i][t // 32], :, t % 32])
            assert torch.equal(V[i][:, t], p.V[p.rows[i][t // 32], :, t % 32])


def test_advance():
    p = Pools([3, -1, 0, 70], 16, (2, 1, 64), F32)
    B.tv_paged_advance(p.batch)
    assert p.len.tolist() == [4, -1, 1, 71]
    p.len.copy_(torch.tensor([3, -1, 0, 70], dtype=torch.int32))
    B.tv_paged_advance(p.batch, B.PagedRows([2, 0, 5, 0]))
    assert p.len.tolist() == [5, -1, 5, 70] and p.status() == 0


def _bounds(p, rows=None):
    code = torch.full((p.n_pages, p.Hkv, 2, p.D), 99, dtype=torch.int8, device="cuda")
    exp = torch.full((p.n_pages, p.Hkv), 99, dtype=torch.int32, device="cuda")
    B.tv_paged_bounds(p.layer, p.batch, rows, code, exp)
    return code, exp


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [(24, 4, 256), (4, 2, 128), (2, 1, 64)])
def test_bounds(dtype, page, heads):
    lens = [0, page - 1, 2 * page - 1, -1, 5, page + 3, 3 * page]
    counts = [page, 1, 0, 0, page - 6, 3 * page, 2 * page - 1]
    p = Pools(lens, page, heads, dtype, extra=3 * page, seed=page, fill=None)
    scale = torch.tensor([1.0, 1e-30, 3e4, 127.0, 1e-38, 1e20][:6], device="cuda")
    p.K.copy_((p.K.float() * scale[torch.arange(p.n_pages, device="cuda") % 6][:, None, None, None]).to(dtype))
    p.K[p.rows[5][2], 0] = 0.0                   # all zero
    p.K[p.rows[5][3], 0, 3, 7] = float("inf")    # not finite
    p.K[p.rows[6][3], 0, page - 1, 0] = float("nan")
    p.K[p.rows[0][0], 0] = 127.0                 # the largest code itself
    p.K[p.rows[1][0], 0] = -127.5
    for rows, c in ((B.PagedRows(counts), counts), (None, [1] * len(lens))):
        code, exp = _bounds(p, rows)
        done = {p.rows[i][j] for i, (L, n) in enumerate(zip(lens, c)) if L >= 0 for j in range(L // page, (L + n) // page)}
        assert done
        for x in range(p.n_pages):
            for g in range(p.Hkv):
                if x not in done:
                    assert (code[x] == 99).all() and (exp[x] == 99).all()
                    continue
                want, e = O.bounds(f64(p.K[x, g]))
                assert int(exp[x, g]) == e and (code[x, g].cpu().numpy() == want).all(), (x, g, int(exp[x, g]), e)
    assert p.status() == 0


def _select(p, code, exp, first, last, n_sel):
    sel = torch.full((len(p.lens), p.Hkv, n_sel), 77, dtype=torch.int32, device="cuda")
    count = torch.full((len(p.lens), p.Hkv), 77, dtype=torch.int32, device="cuda")
    ws = p.space(B.tv_paged_select_workspace_bytes(p.layer, p.batch))
    B.tv_paged_select(p.layer, p.batch, code, exp, first, last, p.q, sel, count, ws)
    return sel, count


def _want(p, code, exp, first, last, n_sel, i, g):
    nb = p.lens[i] // p.page + 1
    ids = p.rows[i][first:nb - last] if nb > n_sel else []
    G = p.Hq // p.Hkv
    return O.select(f64(p.q[i, g * G:(g + 1) * G]), code[ids, g].cpu().numpy().astype(np.int64), exp[ids, g].cpu().numpy(), nb,
                    first, last, n_sel)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", [(24, 4, 256), (32, 1, 64), (4, 4, 128), (2, 1, 64)])
@pytest.mark.parametrize("first,last,n_sel", [(1, 2, 8), (0, 1, 1), (3, 2, 5), (0, 3, 200), (0, 1, 130)])
def test_select(dtype, heads, first, last, n_sel):
    lens = [0, 100, 128 * 16, -1, 300 * 16 + 5, 130 * 16 - 1, 130 * 16]
    p = Pools(lens, 16, heads, dtype, seed=n_sel, fill=None)
    gen = torch.Generator(device="cuda").manual_seed(5)
    code = torch.randint(-127, 128, (p.n_pages, p.Hkv, 2, p.D), generator=gen, device="cuda", dtype=torch.int8)
    exp = torch.randint(-9, -6, (p.n_pages, p.Hkv), generator=gen, device="cuda", dtype=torch.int32)
    exp[::11] = 128
    code[exp == 128] = 0
    code[5::7] = code[5]  # equal scores
    exp[5::7] = exp[5]
    p.q[1] = 0.0
    if dtype == F32:
        p.q[2, 0, 0] = float("nan")
    sel, count = _select(p, code, exp, first, last, n_sel)
    for i, L in enumerate(lens):
        for g in range(p.Hkv):
            if L < 0:
                assert (sel[i] == 77).all() and (count[i] == 77).all()
                continue
            want = _want(p, code, exp, first, last, n_sel, i, g)
            got = sel[i, g].tolist()
            assert int(count[i, g]) == len(want) and got == want + [-1] * (n_sel - len(want)), (i, g)
    assert p.status() == 0


def test_select_largest_sums():
    """Codes and queries at their ends: scores of 127 * 127 * 256, and neighbours that differ by one step."""
    p = Pools([64 * 16 + 3], 16, (24, 4, 256), seed=1, fill=None)
    gen = torch.Generator(device="cuda").manual_seed(1)
    sign = torch.randint(0, 2, (1, 4, 1, 256), generator=gen, device="cuda") * 2 - 1
    p.q.copy_((sign.expand(1, 4, 6, 256).reshape(1, 24, 256) * 127.0).to(BF))
    code = torch.zeros(p.n_pages, 4, 2, 256, dtype=torch.int8, device="cuda")
    code[:, :, 1], code[:, :, 0] = 127, -127
    for x in range(p.n_pages):  # one column of each page a step or two lower
        code[x, :, :, (7 * x) % 256] = torch.tensor([-127 + x % 3, 127 - x % 3], dtype=torch.int8, device="cuda")
    exp = torch.zeros(p.n_pages, 4, dtype=torch.int32, device="cuda")
    sel, count = _select(p, code, exp, 1, 2, 20)
    for g in range(4):
        assert sel[0, g].tolist() == _want(p, code, exp, 1, 2, 20, 0, g) and int(count[0, g]) == 20


@pytest.mark.parametrize("exps", [range(100, 128), range(-100, -72)], ids=["large", "small"])
def test_select_exponents_at_their_ends(exps):
    """Scores whose sizes leave fp32 are still told apart, and those of 0 are equal, whatever their signs of zero."""
    p = Pools([64 * 16 + 3], 16, (24, 4, 256), seed=2, fill=None)
    gen = torch.Generator(device="cuda").manual_seed(2)
    code = torch.randint(-127, 128, (p.n_pages, 4, 2, 256), generator=gen, device="cuda").sort(2).values.to(torch.int8)
    exp = torch.randint(exps[0], exps[-1] + 1, (p.n_pages, 4), generator=gen, device="cuda", dtype=torch.int32)
    code[torch.arange(0, p.n_pages, 5, device="cuda")] = 0
    for sign in (1.0, -1.0):
        p.q.copy_(sign * p.q.abs())
        for n_sel in (9, 30, 60):
            sel, count = _select(p, code, exp, 1, 2, n_sel)
            for g in range(4):
                assert sel[0, g].tolist() == _want(p, code, exp, 1, 2, n_sel, 0, g) and int(count[0, g]) == n_sel
    assert p.status() == 0


@pytest.mark.parametrize("lens", [[200000, 135008], [16 * 16385 + 30, 400000]])
@pytest.mark.parametrize("Hq", [8, 64])
def test_select_long(lens, Hq):
    """Many pages, all drawn from a few; more than shared memory holds."""
    page, cols, G = 16, 26000, Hq // 2
    K = torch.randn(50, 2, page, 64, device="cuda").to(BF)
    table = torch.randint(0, 50, (2, cols), device="cuda", dtype=torch.int32)
    layer, batch = B.PagedLayer(K, K, Hq), B.PagedBatch(table, torch.tensor(lens, dtype=torch.int32, device="cuda"), 400010 if max(lens) > 200000 else 200010)
    code = torch.randint(-127, 128, (50, 2, 2, 64), device="cuda", dtype=torch.int8)
    exp = torch.randint(-3, 0, (50, 2), device="cuda", dtype=torch.int32)
    q = torch.randn(2, Hq, 64, device="cuda").to(BF)
    for n_sel in (1000, 4096, 40):
        sel, count = torch.zeros(2, 2, n_sel, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, dtype=torch.int32, device="cuda")
        ws = torch.empty(B.tv_paged_select_workspace_bytes(layer, batch), dtype=torch.uint8, device="cuda")
        B.tv_paged_select(layer, batch, code, exp, 1, 2, q, sel, count, ws)
        for i, L in enumerate(lens):
            ids = table[i, 1:L // page - 1].tolist()
            for g in range(2):
                want = O.select(f64(q[i, g * G:g * G + G]), code[ids, g].cpu().numpy().astype(np.int64), exp[ids, g].cpu().numpy(),
                                L // page + 1, 1, 2, n_sel)
                assert sel[i, g].tolist() == want and int(count[i, g]) == n_sel
    assert batch.status_code() == 0


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,dtype", [((24, 4, 256), BF), ((16, 2, 128), BF), ((8, 8, 64), BF), ((40, 2, 64), BF), ((4, 2, 128), F32)])
def test_attn_selected(heads, dtype, page):
    """Lists in any order, with pages twice, pages behind the length, empty ones."""
    lens = [9 * page + 5, 3, -1, 20 * page - 1, 6 * page]
    p = Pools(lens, page, heads, dtype, seed=page)
    for i, L in enumerate(lens):  # (pages behind the length exist)
        if L >= 0:
            for j in range(L // page + 1, len(p.rows[i])):
                p.rows[i][j] = p.n_pages - 1
    p.table.copy_(torch.tensor(p.rows, dtype=torch.int32))
    lists = {0: [[9, 0, 4, 4, 7], [], [12, 9], [15], [2] * 9], 1: [[0], [0, 1], [3, 0, 2]], 3: [list(range(20)), [19, 3], [5, 18, 0, 11]],
             4: [[6], [6, 0, 6], [5, 6, 4, 3, 2, 1, 0]]}
    n_sel = 20
    sel = torch.full((len(lens), p.Hkv, n_sel), -1, dtype=torch.int32)
    count = torch.zeros(len(lens), p.Hkv, dtype=torch.int32)
    places = {}
    for i, options in lists.items():
        places[i] = [options[(g + page // 16) % len(options)] for g in range(p.Hkv)]
        for g, x in enumerate(places[i]):
            sel[i, g, :len(x)] = torch.tensor(x, dtype=torch.int32)
            count[i, g] = len(x)
    sel, count = sel.cuda(), count.cuda()
    p.expect(p.selected(sel, count), places=places)
    p.expect(p.selected(sel, count, p.gate), p.gate, places=places)
    assert p.status() == 0


def test_attn_selected_all_pages_equals_attn():
    """Every page listed in order: the bits of the call without a list."""
    p = Pools([700, 64, 0, 1500], 64, seed=9)
    a = p.attn().clone()
    n = 1500 // 64 + 1
    sel = torch.arange(n, dtype=torch.int32, device="cuda").expand(4, 4, n).contiguous()
    count = (p.len // 64 + 1)[:, None].expand(4, 4).to(torch.int32).contiguous()
    assert torch.equal(a, p.selected(sel, count))
