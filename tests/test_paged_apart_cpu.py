"""Paged calls refuse whatever they write, their workspace and the status word among it, where it shares
memory with anything else that they write or read: every pair of each call's buffers, its first and last bytes."""
from __future__ import annotations

import ctypes
from ctypes import c_void_p as vp

import pytest

from speculative_tree_verify_masked_gb300 import binding as B
from tests.test_paged_cpu import L  # noqa: F401  (the library)

ref = ctypes.byref
ARG, CUDA = 1, 7
N_SEQ, COLS, MAX_LEN, HQ, HKV, D, PAGE, PAGES, ROWS, N_SEL = 8, 16, 1000, 24, 4, 256, 64, 100, 20, 8
POOL = PAGES * HKV * PAGE * D * 2
# bytes of each buffer a call may be given
SIZE = {"K": POOL, "V": POOL, "table": N_SEQ * COLS * 4, "len": N_SEQ * 4, "status": 4, "row_off": (N_SEQ + 1) * 4, "group_off": 3 * 4,
        "shared": 2 * 4, "q_norm": D * 4, "k_norm": D * 4, "q_raw": ROWS * HQ * D * 2, "k_raw": ROWS * HKV * D * 2, "v": ROWS * HKV * D * 2,
        "q": ROWS * HQ * D * 2, "aq": N_SEQ * HQ * D * 2, "gate": N_SEQ * HQ * D * 2, "out": N_SEQ * HQ * D * 2,
        "code": PAGES * HKV * 2 * D, "exp": PAGES * HKV * 4, "sel": N_SEQ * HKV * N_SEL * 4, "count": N_SEQ * HKV * 4}
HOME = {k: (i + 1) << 32 for i, k in enumerate(list(SIZE) + ["ws"])}


def _layer(at):
    return B.tv_paged_layer(B.TV_BF16, HQ, HKV, D, PAGE, PAGES, at["K"], at["V"])


def _batch(at):
    return B.tv_paged(N_SEQ, COLS, MAX_LEN, at["table"], at["len"], at["status"])


def _rows(at):
    return ref(B.tv_paged_rows(ROWS, 10, at["row_off"]))


def _groups(at):
    return B.tv_paged_groups(2, at["group_off"], at["shared"])


def append(lib, at):
    return lib.tv_paged_append(ref(_layer(at)), ref(_batch(at)), _rows(at), vp(at["q_norm"]), vp(at["k_norm"]), 1e-6, 64, 1e7,
                               vp(at["q_raw"]), vp(at["k_raw"]), vp(at["v"]), vp(at["q"]), None)


def attn(lib, at):
    return lib.tv_paged_attn(ref(_layer(at)), ref(_batch(at)), ref(_groups(at)), vp(at["aq"]), vp(at["gate"]), vp(at["out"]), 0.1,
                             vp(at["ws"]), 1 << 32, None)


def selected(lib, at):
    return lib.tv_paged_attn_selected(ref(_layer(at)), ref(_batch(at)), vp(at["sel"]), vp(at["count"]), N_SEL, vp(at["aq"]),
                                      vp(at["gate"]), vp(at["out"]), 0.1, vp(at["ws"]), 1 << 32, None)


def bounds(lib, at):
    return lib.tv_paged_bounds(ref(_layer(at)), ref(_batch(at)), _rows(at), vp(at["code"]), vp(at["exp"]), None)


def select(lib, at):
    return lib.tv_paged_select(ref(_layer(at)), ref(_batch(at)), vp(at["code"]), vp(at["exp"]), 1, 2, N_SEL, vp(at["aq"]), vp(at["sel"]),
                               vp(at["count"]), vp(at["ws"]), 1 << 32, None)


def advance(lib, at):
    return lib.tv_paged_advance(ref(_batch(at)), _rows(at), vp(at["len"]), None)


# what each call writes, what it reads, and the pairs that may be one buffer
CALLS = [(append, ["K", "V", "q", "status"], ["q_raw", "k_raw", "v", "q_norm", "k_norm", "row_off", "table", "len"], {("q", "q_raw")}),
         (attn, ["out", "ws", "status"], ["K", "V", "aq", "gate", "group_off", "shared", "table", "len"], {("out", "gate")}),
         (selected, ["out", "ws", "status"], ["K", "V", "aq", "gate", "sel", "count", "table", "len"], {("out", "gate")}),
         (bounds, ["code", "exp", "status"], ["K", "row_off", "table", "len"], set()),
         (select, ["sel", "count", "status"], ["code", "exp", "aq", "table", "len"], set()),
         (advance, ["len", "status"], ["row_off"], set())]


@pytest.mark.parametrize("call,writes,reads,same", CALLS, ids=[c[0].__name__ for c in CALLS])
def test_every_pair_refused(L, call, writes, reads, same):  # noqa: F811
    size = dict(SIZE, ws=max(16, L.tv_paged_attn_workspace_bytes(ref(_layer(HOME)), ref(_batch(HOME)), ref(_groups(HOME)) if call is attn else None)))
    assert call(L, HOME) != ARG  # all apart
    for i, w in enumerate(writes):
        for r in writes[i + 1:] + reads:
            last = (size[r] - 1) // 16 * 16         # the last 16 bytes that r has any of
            mine = (size[w] - 1) // 16 * 16
            for at in (HOME[r], HOME[r] + last, HOME[r] - mine):
                got = call(L, dict(HOME, **{w: at}))
                assert got == ARG or (at == HOME[r] and (w, r) in same), (w, r, hex(at), got)
            # side by side is apart
            assert call(L, dict(HOME, **{w: HOME[r] + last + 16})) != ARG, (w, r)


def test_select_workspace_apart(L):  # noqa: F811
    """A workspace of the choice is one only where shared memory does not hold the keys."""
    layer, cols = B.tv_paged_layer(B.TV_BF16, HQ, HKV, D, 16, PAGES, HOME["K"], HOME["V"]), 20000
    b = B.tv_paged(2, cols, 16384 * 16, HOME["table"], HOME["len"], HOME["status"])
    need = L.tv_paged_select_workspace_bytes(ref(layer), ref(b))
    assert need > 0
    size = {"sel": 2 * HKV * N_SEL * 4, "count": 2 * HKV * 4, "code": PAGES * HKV * 2 * D, "exp": PAGES * HKV * 4, "aq": 2 * HQ * D * 2,
            "table": 2 * cols * 4, "len": 8, "status": 4}

    def call(ws):
        return L.tv_paged_select(ref(layer), ref(b), vp(HOME["code"]), vp(HOME["exp"]), 1, 2, N_SEL, vp(HOME["aq"]), vp(HOME["sel"]),
                                 vp(HOME["count"]), vp(ws), need, None)
    assert call(HOME["ws"]) != ARG
    for r, n in size.items():
        for at in (HOME[r], HOME[r] + (n - 1) // 16 * 16, HOME[r] - (need - 1) // 16 * 16):
            assert call(at) == ARG, (r, hex(at))


def test_advance_without_rows(L):  # noqa: F811
    for word in (HOME["len"], HOME["len"] + 16):
        assert L.tv_paged_advance(ref(_batch(dict(HOME, status=word))), None, vp(HOME["len"]), None) == ARG
