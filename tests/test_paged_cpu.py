"""Calls over caches in pages: what the host refuses (nothing is enqueued), workspace
sizes, and pins of the oracle against brute force."""
from __future__ import annotations

import ctypes
import os
import subprocess
from ctypes import c_void_p as vp

import numpy as np
import pytest
import torch

import oracle.paged as O
from oracle.prompt import attn_prompt
from speculative_tree_verify_masked_gb300 import binding as B

ref = ctypes.byref
ARG, SHAPE, DTYPE, ALIGN, WORKSPACE = 1, 2, 3, 4, 8


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        from speculative_tree_verify_masked_gb300 import build

        build.build()
    return B.lib()


K, V, Q, K_RAW, V_RAW, OUT, FAR = 1 << 30, 2 << 30, 3 << 30, 4 << 30, 5 << 30, 6 << 30, 7 << 30


def layer(dtype=B.TV_BF16, Hq=24, Hkv=4, D=256, page=64, n_pages=100, k=K, v=V):
    return B.tv_paged_layer(dtype, Hq, Hkv, D, page, n_pages, k, v)


def batch(n_seq=8, cols=16, max_len=1000, table=0x1000, len_=0x2000, status=0x3000):
    return B.tv_paged(n_seq, cols, max_len, table, len_, status)


def rows(n_total=20, n_max=10, off=0x4000):
    return B.tv_paged_rows(n_total, n_max, off)


def groups(n=2, off=0x5000, shared=0x6000):
    return B.tv_paged_groups(n, off, shared)


def append(L, l=None, b=None, r=None, qn=0x7000, kn=0x8000, eps=1e-6, rot=64, theta=1e7, q_raw=Q, k_raw=K_RAW, v=V_RAW, q=OUT):
    l, b = layer() if l is None else l, batch() if b is None else b
    return L.tv_paged_append(ref(l), ref(b), ref(r) if r is not None else None, vp(qn), vp(kn), eps, rot, theta, vp(q_raw),
                             vp(k_raw), vp(v), vp(q), None)


def attn(L, l=None, b=None, g=None, q=Q, gate=0, out=OUT, scale=0.1, ws=FAR, n=1 << 30):
    l, b = layer() if l is None else l, batch() if b is None else b
    return L.tv_paged_attn(ref(l), ref(b), ref(g) if g is not None else None, vp(q), vp(gate), vp(out), scale, vp(ws), n, None)


def selected(L, l=None, b=None, sel=0x7000, cnt=0x8000, n_sel=8, q=Q, gate=0, out=OUT, scale=0.1, ws=FAR, n=1 << 30):
    l, b = layer() if l is None else l, batch() if b is None else b
    return L.tv_paged_attn_selected(ref(l), ref(b), vp(sel), vp(cnt), n_sel, vp(q), vp(gate), vp(out), scale, vp(ws), n, None)


def bounds(L, l=None, b=None, r=None, code=OUT, exp=FAR):
    l, b = layer() if l is None else l, batch() if b is None else b
    return L.tv_paged_bounds(ref(l), ref(b), ref(r) if r is not None else None, vp(code), vp(exp), None)


def select(L, l=None, b=None, code=K_RAW, exp=V_RAW, first=1, last=2, n_sel=8, q=Q, sel=0x7000, cnt=0x8000, ws=FAR, n=1 << 30):
    l, b = layer() if l is None else l, batch() if b is None else b
    return L.tv_paged_select(ref(l), ref(b), vp(code), vp(exp), first, last, n_sel, vp(q), vp(sel), vp(cnt), vp(ws), n, None)


@pytest.mark.parametrize("name", ["tv_paged_layer", "tv_paged", "tv_paged_rows", "tv_paged_groups"])
def test_struct_layout_matches_c(name, tmp_path):
    s = getattr(B, name)
    names = [f for f, _ in s._fields_]
    src = f'#include <stdio.h>\n#include <stddef.h>\n#include "tv.h"\nint main(void) {{\n printf("%zu\\n", sizeof({name}));\n'
    src += "".join(f' printf("%zu\\n", offsetof({name}, {n}));\n' for n in names) + " return 0; }\n"
    (tmp_path / "l.c").write_text(src)
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c11", "-I", inc, str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(s)] + [getattr(s, n).offset for n in names]


CALLS = [append, attn, selected, bounds, select]


@pytest.mark.parametrize("call", CALLS)
def test_layers_and_batches_refused(L, call):
    for bad in ({"Hq": 25}, {"Hq": 0}, {"Hkv": 0}, {"D": 96}, {"page": 0}, {"page": 48}, {"page": 8}, {"page": 256}, {"Hq": 129, "Hkv": 1}):
        assert call(L, l=layer(**bad)) == SHAPE, bad
    assert call(L, l=layer(dtype=2)) == DTYPE
    assert call(L, l=layer(Hq=4096, Hkv=4096), b=batch(n_seq=16)) == SHAPE
    for bad in ({"n_pages": 0}, {"n_pages": 1 << 24}):
        assert call(L, l=layer(**bad)) == ARG, bad
    for bad in ({"n_seq": 0}, {"n_seq": 1025}, {"cols": 0}, {"cols": 15}, {"max_len": -1}, {"max_len": 1024}, {"table": 0}, {"len_": 0},
                {"status": 0}, {"cols": (1 << 24) + 1}):
        assert call(L, b=batch(**bad)) == ARG, bad
    for bad in ({"table": 0x1008}, {"len_": 0x2004}, {"status": 0x3008}):
        assert call(L, b=batch(**bad)) == ALIGN, bad
    assert call(L, l=layer(k=K + 8)) == ALIGN
    assert call(L, l=layer(k=0)) == ARG or call is select


@pytest.mark.parametrize("call", [append, bounds])
def test_rows_refused(L, call):
    for r in (rows(-1), rows(20, 21), rows(20, -1), rows(1 << 21, 4), rows(off=0)):
        assert call(L, r=r) == ARG
    assert call(L, r=rows(off=0x4004)) == ALIGN
    assert call(L, r=rows(0, 0)) == 0  # nothing to do


def test_append_refused(L):
    for bad in ({"q_raw": 0}, {"k_raw": 0}, {"v": 0}, {"q": 0}, {"rot": 63}, {"rot": 258}, {"rot": -2}, {"theta": 1.0},
                {"theta": float("inf")}, {"eps": 0.0}, {"qn": 0}, {"kn": 0}):
        assert append(L, **bad) == ARG, bad
    for bad in ({"q_raw": Q + 8}, {"k_raw": K_RAW + 2}, {"v": V_RAW + 4}, {"q": OUT + 8}, {"qn": 0x7004}):
        assert append(L, **bad) == ALIGN, bad
    nq, nk, pool = 8 * 24 * 256 * 2, 8 * 4 * 256 * 2, 100 * 4 * 64 * 256 * 2
    for q in (Q + 16, Q - nq + 16, K_RAW, K_RAW + nk - 16, V_RAW - nq + 16, K + pool - 16, V):
        assert append(L, q=q) == ARG, hex(q)
    for k in (K, K + pool - 16, V - nk + 16):
        assert append(L, k_raw=k) == ARG and append(L, v=k) == ARG and append(L, q_raw=k) == ARG
    assert append(L, l=layer(v=K)) == ARG and append(L, l=layer(v=K + pool - 16)) == ARG


@pytest.mark.parametrize("call", [attn, selected])
def test_attn_refused(L, call):
    for bad in ({"q": 0}, {"out": 0}, {"scale": 0.0}, {"scale": -1.0}, {"scale": float("nan")}, {"scale": float("inf")}):
        assert call(L, **bad) == ARG, bad
    n = 8 * 24 * 256 * 2
    for out in (Q, Q + 16, Q - n + 16):
        assert call(L, out=out) == ARG
    for out in (K, K + 100 * 4 * 64 * 256 * 2 - 16, V - n + 16):
        assert call(L, out=out) == ARG
    for gate in (OUT + 16, OUT - 16, OUT + n - 16):
        assert call(L, gate=gate) == ARG
    for bad in ({"q": Q + 8}, {"out": OUT + 8}, {"gate": Q + 8}, {"ws": FAR + 8}):
        assert call(L, **bad) == ALIGN, bad
    need = L.tv_paged_attn_workspace_bytes(ref(layer()), ref(batch()), None)
    assert need > 0 and need == L.tv_paged_attn_selected_workspace_bytes(ref(layer()), ref(batch()), 8)
    assert call(L, n=need - 1) == WORKSPACE and call(L, ws=0) == WORKSPACE
    assert L.tv_paged_attn_workspace_bytes(ref(layer(dtype=B.TV_F32)), ref(batch()), None) == 0
    assert L.tv_paged_attn_workspace_bytes(ref(layer(D=96)), ref(batch()), None) == 0


def test_groups_and_lists_refused(L):
    for g in (groups(0), groups(9), groups(off=0), groups(shared=0)):
        assert attn(L, g=g) == ARG
    for g in (groups(off=0x5004), groups(shared=0x6008)):
        assert attn(L, g=g) == ALIGN
    assert selected(L, out=0x7000 - 16) == ARG and selected(L, out=0x8010) == ARG
    for bad in ({"sel": 0}, {"cnt": 0}, {"n_sel": 0}, {"n_sel": 4097}):
        assert selected(L, **bad) == ARG, bad
    for bad in ({"sel": 0x7008}, {"cnt": 0x8004}):
        assert selected(L, **bad) == ALIGN, bad


def test_select_and_bounds_refused(L):
    for bad in ({"first": -1}, {"last": 0}, {"first": 7}, {"first": 1, "last": 8}, {"n_sel": 0}, {"n_sel": 4097}, {"code": 0}, {"exp": 0},
                {"q": 0}, {"sel": 0}, {"cnt": 0}, {"first": (1 << 31) - 1, "last": (1 << 31) - 1}):
        assert select(L, **bad) == ARG, bad
    for bad in ({"code": K_RAW + 4}, {"exp": V_RAW + 4}, {"q": Q + 8}, {"sel": 0x7004}, {"cnt": 0x8004}, {"ws": FAR + 4}):
        assert select(L, **bad) == ALIGN, bad
    for bad in ({"sel": 0x8000, "cnt": 0x8010}, {"sel": K_RAW}, {"cnt": V_RAW + 16}, {"sel": Q}, {"cnt": 0x2010}, {"sel": 0x1010}):
        assert select(L, **bad) == ARG, bad
    need = L.tv_paged_select_workspace_bytes(ref(layer()), ref(batch()))
    assert need == 0  # up to 16,384 pages
    far = dict(l=layer(page=16), b=batch(cols=20000, max_len=16384 * 16))
    need = L.tv_paged_select_workspace_bytes(ref(far["l"]), ref(far["b"]))
    assert need == 8 * 4 * 16385 * 4
    far.update(sel=9 << 30, cnt=10 << 30)
    assert select(L, n=need - 1, **far) == WORKSPACE and select(L, ws=0, **far) == WORKSPACE
    for bad in ({"code": 0}, {"exp": 0}, {"code": K}, {"exp": K + 16}, {"exp": OUT + 16}):
        assert bounds(L, **bad) == ARG, bad
    assert bounds(L, code=OUT + 8) == ALIGN


def test_advance_refused(L):
    def adv(b=None, r=None, len_=0x2000):
        return L.tv_paged_advance(ref(batch() if b is None else b), ref(r) if r is not None else None, vp(len_), None)
    for bad in ({"n_seq": 0}, {"n_seq": 1025}, {"max_len": -1}, {"max_len": 1 << 30}, {"len_": 0}, {"status": 0}):
        assert adv(batch(**bad)) == ARG, bad
    assert adv(len_=0) == ARG and adv(len_=0x2010) == ARG
    assert adv(batch(len_=0x2004), len_=0x2004) == ALIGN and adv(r=rows(off=0)) == ARG


TABLE, LEN, WORD = 0x1000, 0x2000, 0x3000


@pytest.mark.parametrize("where", [TABLE, TABLE + 8 * 16 * 4 - 16, LEN, LEN + 16, WORD])
def test_writes_into_the_batch_refused(L, where):
    for call in (attn, selected):
        assert call(L, out=where) == ARG and call(L, ws=where) == ARG
    assert append(L, q=where) == ARG and append(L, l=layer(k=where)) == ARG and append(L, l=layer(v=where)) == ARG
    assert bounds(L, code=where) == ARG and bounds(L, exp=where) == ARG
    assert select(L, sel=where) == ARG and select(L, cnt=where) == ARG


def test_workspaces_apart(L):
    need = L.tv_paged_attn_workspace_bytes(ref(layer()), ref(batch()), None)
    n, pool = 8 * 24 * 256 * 2, 100 * 4 * 64 * 256 * 2
    for ws in (Q, Q + n - 16, OUT - need + 16, K + pool - 16, V):
        assert attn(L, ws=ws) == ARG and selected(L, ws=ws) == ARG
    assert attn(L, gate=FAR + 16) == ARG and selected(L, sel=FAR) == ARG and selected(L, cnt=FAR + need // 16 * 16 - 16) == ARG
    assert attn(L, g=groups(), out=0x5000) == ARG and attn(L, g=groups(shared=1 << 20), out=(1 << 20) - n + 16) == ARG
    far = dict(l=layer(page=16), b=batch(cols=20000, max_len=16384 * 16), sel=9 << 30, cnt=10 << 30)
    for ws in (9 << 30, 10 << 30, K_RAW, V_RAW, Q + n - 16, TABLE):
        assert select(L, ws=ws, **far) == ARG


def test_bindings_refuse_host_memory():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    b = B.PagedBatch(torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 32)
    assert not B.PagedLayer(k, k, 4).sound and not b.sound
    with pytest.raises(ValueError):
        B.PagedGroups([1, 2], [16], device="cpu")
    r = B.PagedRows([3, 0, 2], device="cpu", n_total=9, n_max=4)
    r.set_rows([4, 4, 1])
    assert r.row_off.tolist() == [0, 4, 8, 9]
    for bad in ([5, 0, 0], [4, 4, 2], [1, 1]):
        with pytest.raises(ValueError):
            r.set_rows(bad)


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------
def _pools(rng, n_pages=12, Hkv=2, page=16, D=8):
    return (rng.standard_normal((n_pages, Hkv, page, D)) for _ in range(2))


def test_attend_equals_contiguous():
    rng = np.random.default_rng(0)
    Kp, Vp = _pools(rng)
    table, Ln = [7, 2, 9, 11, 0], 16 * 3 + 5
    q, gate = rng.standard_normal((4, 8)), rng.standard_normal((4, 8))
    k, v = (np.concatenate([x[p] for p in table], 1) for x in (Kp, Vp))
    out, _, _ = O.attend(Kp, Vp, table, Ln, q, 0.3, gate)
    t64 = torch.from_numpy
    want = attn_prompt(t64(k), t64(v), Ln, t64(q[None]), 0.3, t64(gate[None]))[0].numpy().reshape(4, 8)
    assert np.abs(out - want).max() < 1e-12
    # listed pages: all of them in another order are the same rows; a page twice counts twice; none: zeros
    again, _, _ = O.attend(Kp, Vp, table, Ln, q, 0.3, gate, [[3, 0, 2, 1], [1, 3, 0, 2]])
    assert np.abs(out - again).max() < 1e-12
    one, _, _ = O.attend(Kp, Vp, table, 15, q, 0.3, None, [[0, 0], [0]])
    assert np.abs(one - O.attend(Kp, Vp, table, 15, q, 0.3)[0]).max() < 1e-12
    none, _, _ = O.attend(Kp, Vp, table, 15, q, 0.3, None, [[], [1, 4]])
    assert not none.any()


def test_append_positions():
    """A turned row's norm stays, position 0 turns nothing, and scores depend on the distance alone."""
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
    dots = []
    for p in (0, 5, 1000):
        yq, _ = O.append(q, k, [p + 7], None, None, 0, 8, 100.0)
        _, yk = O.append(q, k, [p], None, None, 0, 8, 100.0)
        dots.append((yq * yk).sum())
        assert abs(np.linalg.norm(yk) - np.linalg.norm(k)) < 1e-12
    assert np.ptp(dots) < 1e-10
    assert np.array_equal(O.append(q, k, [0], None, None, 0, 8, 100.0)[0], q)


def test_scores_bound_every_key():
    rng = np.random.default_rng(2)
    for scale in (1e-3, 1.0, 37.0):
        keys, q = scale * rng.standard_normal((5, 16, 8)), rng.standard_normal((3, 8))
        code, e = zip(*(O.bounds(x) for x in keys))
        s = O.scores(q, np.array(code), np.array(e))
        u = O.query_codes(q)
        for j in range(5):
            assert (u @ keys[j].T).max() <= s[j] + 1e-9
            assert (code[j][0] * 2.0 ** e[j] <= keys[j].min(0)).all() and (code[j][1] * 2.0 ** e[j] >= keys[j].max(0)).all()
            assert np.abs(code[j]).max() > 63  # the least exponent
    assert O.bounds(np.full((4, 2), 127.0))[1] == 0 and O.bounds(np.full((4, 2), 127.5))[1] == 1
    assert O.bounds(np.zeros((4, 2)))[1] == -100 and O.bounds(np.array([[1.0, np.nan]]))[1] == 128


def test_select_by_hand():
    q = np.array([[2.0, 0.0]])  # codes 64, 0
    code = np.array([[[0, 0], [c, 9]] for c in (5, 7, 7, 1, 7)])
    e = np.zeros(5, int)
    assert O.select(q, code, e, 8, 1, 2, 5) == [0, 2, 3, 6, 7]   # pages 2, 3 and 5 tie: the lower two
    assert O.select(q, code, e, 8, 1, 2, 3) == [0, 6, 7]
    assert O.select(q, code, e, 8, 1, 2, 8) == list(range(8))
    e[0] = 128
    assert O.select(q, code, e, 8, 1, 2, 4) == [0, 1, 6, 7]      # an infinite score
