"""The choice of pages for more slots than run at once, against the oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.paged as O
from tests.paged_helpers import Pools, f64
from tests.test_paged_errors_gpu import _codes, _selected

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", [(4, 4, 64), (24, 4, 256), (48, 4, 128)])
def test_choice_for_more_slots_than_run_at_once(dtype, heads):
    """CTAs of half the threads, a KV head of up to twelve query heads: the oracle's lists."""
    lens = [16 * ((7 * i) % 150) + i % 16 for i in range(400)]
    p = Pools(lens, 16, heads, dtype, fill=None) if heads[2] < 256 else Pools(lens[:110], 16, heads, dtype, fill=None)
    code, exp = _codes(p)
    exp[::13] = 128
    code[::13] = 0
    sel, count, clean = _selected(p, code, exp, 24)
    assert clean and p.status() == 0
    G = p.Hq // p.Hkv
    for i in range(0, len(p.lens), 7):
        nb = p.lens[i] // 16 + 1
        ids = p.rows[i][1:nb - 2] if nb > 24 else []
        for g in range(p.Hkv):
            want = O.select(f64(p.q[i, g * G:(g + 1) * G]), code[ids, g].cpu().numpy().astype(np.int64), exp[ids, g].cpu().numpy(), nb, 1, 2, 24)
            assert sel[i, g].tolist() == want + [-1] * (24 - len(want)) and int(count[i, g]) == len(want), (i, g)
