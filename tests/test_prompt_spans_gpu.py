"""Spans of a PromptPass fed one behind the other: on a stream of their own,
without waits between them, and spans that are refused."""
from __future__ import annotations

import pytest
import torch

from tests.test_prompt_pass_gpu import BF, F32, Stack

pytestmark = pytest.mark.gpu


def held(st, n):
    """What a prompt of `n` rows a sequence leaves: caches, states, tails."""
    r = st.r
    return ([t[:, :m].clone() for a in r.attn.values() for kv in (a["layer"].K, a["layer"].V) for t, m in zip(kv, n)]
            + [t.clone() for g in r.gdn.values() for t in g["layer"].S] + [t.clone() for ts in st.tails.values() for t in ts])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("handle", [False, True])
def test_spans_on_a_stream_of_their_own(dtype, handle):
    """set_rows for the next span while the span before still waits in the stream."""
    st = Stack(dtype, [130, 71])
    p = st.make(201, 130)
    spans = [[(0, 64), (0, 0)], [(64, 65), (0, 50)], [(65, 130), (50, 71)]]
    inputs = []
    for sp in spans:
        _, x = st.rows_of(sp)
        n = sum(b - a for a, b in sp)
        inputs.append({li: {k: (v if k == "w_norm" else torch.cat([v, v.new_zeros((201 - n, *v.shape[1:]))]))
                            for k, v in xs.items()} for li, xs in x.items()})
    for sp, x in zip(spans, inputs):  # one at a time, on the current stream
        p.set_rows([b - a for a, b in sp])
        p.run(x)
        torch.cuda.synchronize()
    assert p.status() == 0 and st.r.len.tolist() == [130, 71]
    ref = held(st, [130, 71])
    outs = [{li: v["out"].clone() for li, v in x.items()} for x in inputs]
    st.reset()
    for x in inputs:
        for v in x.values():
            v["out"].zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    arg = s.cuda_stream if handle else s
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # (some 10 ms: everything below is enqueued meanwhile)
    for sp, x in zip(spans, inputs):
        p.set_rows([b - a for a, b in sp], arg)
        p.run(x, arg)
    torch.cuda.synchronize()
    assert p.status() == 0 and st.r.len.tolist() == [130, 71]
    for a, b in zip(ref, held(st, [130, 71])):
        assert torch.equal(a, b)
    for sp, x, o in zip(spans, inputs, outs):
        n = sum(b - a for a, b in sp)
        for li, v in x.items():
            assert torch.equal(v["out"][:n], o[li][:n]), li


def test_rows_are_not_set_inside_a_capture():
    st = Stack(F32, [20, 10])
    p = st.make(30, 20)
    p.set_rows([20, 10])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run(st.x)
        with pytest.raises(RuntimeError):
            p.set_rows([5, 5])
    g.replay()
    torch.cuda.synchronize()
    assert p.status() == 0 and st.r.len.tolist() == [20, 10]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("why,code", [("len", 10), ("capacity", 6), ("rows", 12), ("len below 0", 10)])
def test_a_refused_span_moves_nothing(dtype, why, code):
    """GDN layers come first here: they must not move either; cleared, the span runs."""
    st = Stack(dtype, [65, 40])
    r = st.r
    p = st.make(105, 65)
    for a in r.attn.values():  # (NaN is not equal to itself)
        for t in a["layer"].K + a["layer"].V:
            t.fill_(3.0)
    p.set_rows([65, 40])
    L = {"len": [0, r.max_len + 1], "capacity": [r.max_len, 0], "rows": [7, 9], "len below 0": [-1, 0]}[why]
    assert r.cap == r.max_len + 64
    if why == "rows":
        p.prompt.row_off.copy_(torch.tensor([0, 65, 50], dtype=torch.int32))
    r.len.copy_(torch.tensor(L, dtype=torch.int32))
    full = [t.clone() for a in r.attn.values() for t in a["layer"].K + a["layer"].V] + held(st, [0, 0])
    for _ in range(2):  # (the word stays: the second one is a no-op too)
        p.run(st.x)
    torch.cuda.synchronize()
    assert p.status() == code and r.len.tolist() == L
    now = [t for a in r.attn.values() for t in a["layer"].K + a["layer"].V] + held(st, [0, 0])
    assert all(torch.equal(a, b) for a, b in zip(full, now))
    p.prompt.status.zero_()
    p.set_rows([65, 40])
    st.reset()
    p.run(st.x)
    torch.cuda.synchronize()
    assert p.status() == 0 and r.len.tolist() == [65, 40]
    assert all(bool(torch.isfinite(t).all()) for t in held(st, [65, 40]))


def test_span_check_and_advance_by_themselves():
    from speculative_tree_verify_masked_gb300 import binding as B

    ln = torch.tensor([5, 10, 0], dtype=torch.int32, device="cuda")
    p = B.Prompt([3, 0, 4], n_total=9, n_max=6)
    B.tv_prompt_check(p, ln, 10, 13)
    B.tv_prompt_advance(p, ln)
    torch.cuda.synchronize()
    assert p.status_code() == 0 and ln.tolist() == [8, 10, 4]
    B.tv_prompt_check(p, ln, 10, 10)  # 8 + 3 rows
    B.tv_prompt_advance(p, ln)
    torch.cuda.synchronize()
    assert p.status_code() == 6 and ln.tolist() == [8, 10, 4]
    p.status.zero_()
    B.tv_prompt_check(p, ln, 9, 100)
    torch.cuda.synchronize()
    assert p.status_code() == 10
    p.status.zero_()
    p.row_off.copy_(torch.tensor([0, 7, 7, 9]))
    B.tv_prompt_advance(p, ln)  # more than n_max rows
    torch.cuda.synchronize()
    assert p.status_code() == 12 and ln.tolist() == [8, 10, 4]
