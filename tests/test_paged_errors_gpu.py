"""Errors that a paged call finds while its other CTAs are at work: what it writes for other slots is
right or left as it was, never half of it, and nothing behind its buffers is touched."""
from __future__ import annotations

import pytest
import torch

from speculative_tree_verify_masked_gb300 import binding as B
from tests.paged_helpers import Pools

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ERR_LEN, ERR_PAGE = 10, 13
MARGIN = 4096  # values before and behind an output


def _framed(shape, dtype, fill):
    """A tensor with margins of the same value, and the whole of it."""
    n = 1
    for x in shape:
        n *= x
    whole = torch.full((n + 2 * MARGIN,), fill, dtype=dtype, device="cuda")
    return whole[MARGIN:MARGIN + n].view(shape), whole


def _margins(whole, fill):
    return bool((whole[:MARGIN] == fill).all()) and bool((whole[-MARGIN:] == fill).all())


def _selected(p, code, exp, n_sel, first=1, last=2):
    """sel, count and whether their margins are as they were."""
    sel, sel_all = _framed((len(p.lens), p.Hkv, n_sel), torch.int32, 77)
    count, count_all = _framed((len(p.lens), p.Hkv), torch.int32, 77)
    ws = p.space(B.tv_paged_select_workspace_bytes(p.layer, p.batch))
    B.tv_paged_select(p.layer, p.batch, code, exp, first, last, p.q, sel, count, ws)
    return sel, count, _margins(sel_all, 77) and _margins(count_all, 77)


def _codes(p, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    code = torch.randint(-127, 128, (p.n_pages, p.Hkv, 2, p.D), generator=gen, device="cuda", dtype=torch.int8)
    return code, torch.randint(-9, -6, (p.n_pages, p.Hkv), generator=gen, device="cuda", dtype=torch.int32)


# many more CTAs than run at once; two an SM; clusters of eight, four and two, where CTAs of one slot may disagree
SELECT = [("many", [16 * (40 + i % 90) + i % 16 for i in range(500)] + [5, -1, 40], (4, 4, 64)),
          ("some", [16 * (200 + i) for i in range(60)], (8, 2, 128)),
          ("clusters", [16 * 4000 + 3, 16 * 2500, 90, 16 * 3999], (8, 2, 64)),
          ("wide", [16 * 900 + i for i in range(20)], (32, 2, 64))]


@pytest.mark.parametrize("name,lens,heads", SELECT, ids=[x[0] for x in SELECT])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_choice_beside_an_entry_that_names_no_page(name, lens, heads, dtype):
    p = Pools(lens, 16, heads, dtype, fill=None)
    code, exp = _codes(p)
    n_sel = 24
    want_sel, want_count, clean = _selected(p, code, exp, n_sel)
    assert clean and p.status() == 0
    for bad in (0, 1, len(lens) // 4 * 3):
        j = lens[bad] // 16 // 2
        keep = int(p.table[bad, j])
        for entry in (p.n_pages, -1, 1 << 30, -(1 << 31)):
            p.table[bad, j] = entry
            sel, count, clean = _selected(p, code, exp, n_sel)
            assert p.status() == ERR_PAGE and clean
            # a list is written whole or not at all; the slot's own is n_sel pages, whichever
            left = (sel == 77).all(-1) & (count == 77)
            right = (sel == want_sel).all(-1) & (count == want_count)
            right[bad] = True
            assert (left | right).all()
            assert ((sel[bad] >= 0) & (sel[bad] <= lens[bad] // 16) | (sel[bad] == 77)).all()
            p.batch.status.zero_()
        p.table[bad, j] = keep
    sel, count, clean = _selected(p, code, exp, n_sel)
    assert torch.equal(sel, want_sel) and torch.equal(count, want_count) and p.status() == 0


def test_choice_beside_a_length_that_is_not_allowed():
    name, lens, heads = SELECT[0]
    p = Pools(lens, 16, heads, BF, fill=None)
    code, exp = _codes(p)
    want_sel, want_count, _ = _selected(p, code, exp, 24)
    for L in (-2, p.max_len + 1, (1 << 31) - 1):
        p.len[7] = L
        sel, count, clean = _selected(p, code, exp, 24)
        left = (sel == 77).all(-1) & (count == 77)
        right = (sel == want_sel).all(-1) & (count == want_count)
        assert p.status() == ERR_LEN and clean and (left | right).all() and left[7].all()
        p.batch.status.zero_()


def test_choice_given_the_word():
    name, lens, heads = SELECT[0]
    p = Pools(lens, 16, heads, BF, fill=None)
    code, exp = _codes(p)
    p.batch.status[0] = ERR_PAGE
    sel, count, clean = _selected(p, code, exp, 24)
    assert (sel == 77).all() and (count == 77).all() and clean and p.status() == ERR_PAGE


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [16, 64])
def test_bounds_beside_an_entry_that_names_no_page(dtype, page):
    """Hundreds of slots' pages, each bound by its keys or not at all."""
    lens = [(37 * i) % 500 for i in range(300)]
    counts = [4 * page + i % 9 for i in range(300)]
    p = Pools(lens, page, (8, 4, 128), dtype, extra=5 * page, fill=None)
    rows = B.PagedRows(counts)

    def run():
        code, code_all = _framed((p.n_pages, p.Hkv, 2, p.D), torch.int8, 99)
        exp, exp_all = _framed((p.n_pages, p.Hkv), torch.int32, 99)
        B.tv_paged_bounds(p.layer, p.batch, rows, code, exp)
        return code, exp, _margins(code_all, 99) and _margins(exp_all, 99)

    want_code, want_exp, clean = run()
    assert clean and p.status() == 0
    for bad in (0, 150, 299):
        j = lens[bad] // page + 1
        keep = int(p.table[bad, j])
        for entry in (p.n_pages, -1, -(1 << 31)):
            p.table[bad, j] = entry
            code, exp, clean = run()
            assert p.status() == ERR_PAGE and clean
            left = (code == 99).all(-1).all(-1) & (exp == 99)
            right = (code == want_code).all(-1).all(-1) & (exp == want_exp)
            assert (left | right).all() and left[keep].all()
            p.batch.status.zero_()
        p.table[bad, j] = keep
    p.batch.status[0] = ERR_PAGE
    code, exp, clean = run()
    assert (code == 99).all() and (exp == 99).all() and clean


@pytest.mark.parametrize("dtype,heads,lens", [(F32, (4, 2, 64), [(61 * i) % 400 for i in range(400)]),
                                              (BF, (8, 2, 128), [(61 * i) % 400 for i in range(400)]),
                                              (BF, (24, 4, 256), [9000, 300, 4001, -1, 64, 20000])])
@pytest.mark.parametrize("chosen", [False, True])
def test_attention_beside_an_entry_that_names_no_page(dtype, heads, lens, chosen):
    """Rows of out as they are without the bad entry, or as they were: cut items, whole ones, every page or listed ones."""
    p = Pools(lens, 16, heads, dtype)
    sel = torch.tensor([[list(range(5))] * p.Hkv] * len(lens), dtype=torch.int32, device="cuda")
    count = torch.tensor([[min(5, L // 16 + 1)] * p.Hkv for L in lens], dtype=torch.int32, device="cuda")

    def run():
        p.out, whole = _framed((len(lens), p.Hq, p.D), dtype, 7.0)
        p.selected(sel, count, p.gate) if chosen else p.attn(p.gate)
        return p.out, _margins(whole, 7.0)

    want, clean = run()
    assert clean and p.status() == 0 and want.isfinite().all()
    for bad in (i for i, L in enumerate(lens) if i in (1, 4, 200, 399) and L >= 16):
        keep = int(p.table[bad, 1])
        for entry in (p.n_pages, -1, -(1 << 31)):
            p.table[bad, 1] = entry
            out, clean = run()
            assert p.status() == ERR_PAGE and clean
            ok = (out == 7).all(-1) | (out == want).all(-1)
            ok[bad] = True
            assert ok.all()
            p.batch.status.zero_()
        p.table[bad, 1] = keep
    out, _ = run()
    assert torch.equal(out, want) and p.status() == 0
    p.batch.status[0] = ERR_PAGE
    out, clean = run()
    assert (out == 7).all() and clean
