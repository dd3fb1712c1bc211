"""The books of PagedCaches (pages, users, lengths, the table), which are kept on the host: what they refuse
leaves them as they were."""
from __future__ import annotations

import os

import pytest
import torch

from speculative_tree_verify_masked_gb300 import binding as B
from speculative_tree_verify_masked_gb300.paged import PagedCaches


@pytest.fixture(scope="module", autouse=True)
def library():
    if not os.path.exists(B.LIB_PATH):
        from speculative_tree_verify_masked_gb300 import build

        build.build()


def caches(n_slots=4, n_pages=20, page=16, max_len=100):
    return PagedCaches(1, n_pages, page, 4, 2, 64, n_slots, max_len, torch.float32, device="cpu")


def books(c):
    return [list(x) for x in c.pages], list(c.lens), list(c.users), list(c.free), c.table.tolist(), c.len.tolist()


def sound(c):
    """Every page free or counted once for each slot that holds it; the device's table and lengths as the host's."""
    held = [p for x in c.pages for p in x]
    assert all(c.users[p] == held.count(p) for p in range(len(c.users)))
    assert sorted(c.free + list(set(held))) == list(range(len(c.users)))
    for s, ids in enumerate(c.pages):
        assert c.table[s].tolist() == ids + [-1] * (c.table.shape[1] - len(ids)) and int(c.len[s]) == c.lens[s]


def test_slots_that_are_not_there():
    c = caches()
    c.admit(0)
    c.grow([40, 0, 0, 0])
    c.len[0] = c.lens[0] = 40
    before = books(c)
    for slot in (-1, -4, 4, 99):
        with pytest.raises(ValueError):
            c.admit(slot)
        with pytest.raises(ValueError):
            c.retire(slot)
        with pytest.raises(ValueError):
            c.admit(1, like=slot, rows=16)
        with pytest.raises(ValueError):
            c.admit(1, like=slot)
    assert books(c) == before
    sound(c)


def test_prefixes_that_are_not_there():
    c = caches()
    c.admit(0)
    c.grow([40, 0, 0, 0])
    c.len[0] = c.lens[0] = 40
    before = books(c)
    for like, rows in ((0, -16), (0, -32), (0, 8), (0, 48), (2, 16), (2, 0), (None, 16), (None, -16), (1, 0)):
        with pytest.raises(ValueError):
            c.admit(1, like=like, rows=rows)
    assert books(c) == before
    c.admit(1, like=0, rows=32)
    sound(c)
    c.retire(0)
    sound(c)
    c.retire(1)
    sound(c)
    assert len(c.free) == 20
