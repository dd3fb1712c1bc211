"""Prompt calls run over and over give the same bits: nothing in flight on the
chip (tiles, queries, partial results) is overwritten before it has been read.
Between runs the outputs and the workspace are filled with other values, and now
and then the L2 cache with other lines."""
from __future__ import annotations

import pytest
import torch

from tests.test_prompt_gpu import Attn, Gdn

pytestmark = pytest.mark.gpu


def repeat(n, run, tensors, ws):
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    run()
    ref = [t.clone() for t in tensors]
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(n):
        if i % 8 == 0:
            flush.zero_()
        if i % 4 == 0:
            ws.fill_(0xFF)
        tensors[0].fill_(7.0)
        run()
        for t, r in zip(tensors, ref):
            bad += (t != r).any()
    assert int(bad) == 0


@pytest.mark.parametrize("kw", [dict(rows=[1500], ctx=[0], gate=True), dict(rows=[700, 30, 900], ctx=[0, 2000, 333]),
                                dict(rows=[1500], ctx=[77], Hq=8, Hkv=8, D=64, gate=True),
                                dict(rows=[3, 1, 700], ctx=[5000, 127, 0], Hq=32, Hkv=4, D=128)])
def test_attn_prompt_repeats(kw):
    a = Attn(seed=9, **kw)
    repeat(3000, a.run, [a.out], a.ws)
    assert a.prompt.status_code() == 0


@pytest.mark.parametrize("kw", [dict(rows=[2000, 700], Hk=4, Hv=8), dict(rows=[300, 63, 1]), dict(rows=[900], Hk=2, Hv=4, dk=64, dv=64)])
def test_gdn_prompt_repeats(kw):
    g = Gdn(seed=3, **kw)

    def run():
        for s, z in zip(g.S, g.S0):
            s.copy_(z)
        g.run()

    repeat(1000, run, [g.out] + g.S, g.ws)
    assert g.prompt.status_code() == 0


def test_calls_on_two_streams_at_once():
    """Two batches of each kind side by side, each with its own buffers, give what each gives alone."""
    runs = [Attn([900], [300], seed=4, gate=True), Attn([40, 500], [3000, 0], Hq=16, Hkv=2, D=128, seed=5),
            Gdn([700, 20], Hk=4, Hv=8, seed=6), Gdn([30], Hk=2, Hv=4, dk=64, dv=64, seed=7)]

    def go(x, stream=None):
        if isinstance(x, Gdn):
            for s, z in zip(x.S, x.S0):
                s.copy_(z)
        x.run(stream)

    refs = []
    for x in runs:
        go(x)
        refs.append([x.out.clone()] + [s.clone() for s in getattr(x, "S", [])])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(50):
        for x, s in zip(runs, streams):
            with torch.cuda.stream(s):
                x.out.fill_(7.0)
                go(x)
    torch.cuda.synchronize()
    for x, ref in zip(runs, refs):
        assert x.prompt.status_code() == 0
        for a, b in zip([x.out] + list(getattr(x, "S", [])), ref):
            assert torch.equal(a, b)
