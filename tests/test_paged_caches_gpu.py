"""PagedCaches on the GPU: what a capture may not hold, and prefixes that pay for being read once, in steps
that are run and in captured ones."""
from __future__ import annotations

import pytest
import torch

from speculative_tree_verify_masked_gb300 import binding as B
from speculative_tree_verify_masked_gb300.paged import PagedCaches

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _raw(gen, n, H, D, dt=BF):
    return torch.randn((n, H, D), generator=gen, device="cuda").to(dt)


def test_books_inside_a_capture():
    """What writes from the host is refused there, before the books change; so is a whole step, which counts rows that have not run."""
    c = PagedCaches(1, 30, 16, 4, 2, 64, 3, 100)
    c.admit(0)
    c.grow([16, 0, 0])
    c.len[0] = c.lens[0] = 16
    c.admit(1, like=0, rows=16)
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = {"q": _raw(gen, 3, 4, 64), "k": _raw(gen, 3, 2, 64), "v": _raw(gen, 3, 2, 64), "out": torch.zeros(3, 4, 64, dtype=BF, device="cuda")}

    def books():
        return [list(p) for p in c.pages], list(c.lens), list(c.users), list(c.free)

    before, table, other = books(), c.table.clone(), torch.zeros(4, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (None, stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            other.add_(1)
            for refused in (lambda: c.grow(stream=given), lambda: c.admit(2, stream=given), lambda: c.retire(1, stream=given),
                            lambda: c.decode([x], stream=given)):
                with pytest.raises(RuntimeError):
                    refused()
                assert books() == before
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.table, table) and c.len.tolist() == [16, 16, -1]
    c.grow()  # pages for the two slots' next rows
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=stream):
        other.add_(1)
        c.grow()  # none are needed: nothing to write
        with pytest.raises(RuntimeError):
            c.decode([x])
    assert c.lens == [16, 16, -1]
    c.decode([x])
    assert c.lens == [17, 17, -1] and c.len.tolist() == [17, 17, -1] and c.status() == 0
