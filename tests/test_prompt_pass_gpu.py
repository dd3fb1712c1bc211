"""Prompts brought into a verify round's caches and states, and the round or
decode step that goes on from there (prompt.py), against the fp64 definitions.

Tolerances: outputs as the verify tests hold them (gpu_helpers.check_close).
fp32 chains two calls whose errors are near 1e-6 each; its bounds leave ten
times that.  bf16 runs are compared with the oracle where one call follows
from what is in memory, and bit for bit with each other.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.gdn_front as GF
import oracle.prompt as OP
import oracle.tree_verify as O
from speculative_tree_verify_masked_gb300 import binding as B
from speculative_tree_verify_masked_gb300 import synth
from speculative_tree_verify_masked_gb300.prompt import PromptPass
from speculative_tree_verify_masked_gb300.round import VerifyRound
from tests.gpu_helpers import check_close, f64, oracle_attn, oracle_gdn, seq_slice

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ROT, THETA, EPS, W = 32, 1e4, 1e-6, 4


class Stack:
    """A four-layer round whose contexts are still empty, and a prompt's raw
    projections for it."""

    def __init__(self, dtype, rows, pad=0, D=64, Hk=2, Hv=4, d=64):
        s = synth.Shapes(Hq=4, Hkv=2, D=D, Hk=Hk, Hv=Hv, dk=d, dv=d, kv_dtype=dtype)
        cfg = synth.Workload("prompt, then a round", 90, s, [300, 200], [("merged", 12, 6), ("chain", 5)], 4,
                             attn_layers=[1, 3], accept=[("random",)] * 2)
        self.rows, self.s, n = rows, s, sum(rows) + pad
        self.r = r = VerifyRound(cfg)
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        C = 2 * Hk * d + Hv * d

        def rnd(*shape, dt=F32):
            return torch.randn(*shape, generator=g, device="cuda").to(dt)

        self.w = {li: rnd(C, W) * W ** -0.5 for li in r.gdn}
        self.tails = {li: [torch.zeros(W - 1, C, device="cuda", dtype=dtype) for _ in rows] for li in r.gdn}
        self.norms = {1: (1 + 0.1 * rnd(D), 1 + 0.1 * rnd(D))}
        self.x = {}
        for li in r.layers:
            if li in r.attn:
                self.x[li] = dict(q=rnd(n, 4, D, dt=dtype), k=rnd(n, 2, D, dt=dtype), v=rnd(n, 2, D, dt=dtype),
                                  out=torch.zeros(n, 4, D, device="cuda", dtype=dtype))
                if li == 3:
                    self.x[li]["gate"] = rnd(n, 4, D, dt=dtype)
            else:
                self.x[li] = dict(x=rnd(n, C, dt=dtype), a=rnd(n, Hv), b=rnd(n, Hv), z=rnd(n, Hv, d, dt=dtype),
                                  w_norm=1 + 0.1 * rnd(d), out=torch.zeros(n, Hv, d, device="cuda", dtype=dtype))
        self.reset()

    def reset(self):
        r = self.r
        r.len.zero_()
        for a in r.attn.values():
            for t in a["layer"].K + a["layer"].V:
                t.fill_(float("nan"))
        for t in [t for g in r.gdn.values() for t in g["layer"].S] + [t for ts in self.tails.values() for t in ts]:
            t.zero_()
        for x in self.x.values():
            x["out"].zero_()

    def make(self, n_total, n_max):
        conv = {li: (self.w[li], self.tails[li]) for li in self.r.gdn}
        return PromptPass(self.r, n_total, n_max, conv, self.norms, ROT, THETA, EPS)

    def rows_of(self, spans):
        """The span inputs: each sequence's rows [a, b) of every layer, packed."""
        off = np.concatenate([[0], np.cumsum(self.rows)])
        idx = torch.cat([torch.arange(off[s] + a, off[s] + b) for s, (a, b) in enumerate(spans)]).cuda()
        return idx, {li: {k: (v if k == "w_norm" else v[idx].contiguous()) for k, v in x.items()} for li, x in self.x.items()}

    def oracle(self, li, s):
        """(outputs of sequence s's rows, (K, V) or S or after them) from the raw projections, fp64."""
        sl = slice(sum(self.rows[:s]), sum(self.rows[:s + 1]))
        x, m = self.x[li], self.s
        if li in self.r.attn:
            n = self.rows[s]
            wq, wk = self.norms.get(li, (None, None))
            pos = torch.arange(n, device="cuda")
            q = OP.norm_rope(x["q"][sl], wq, pos, EPS, ROT, THETA)
            K = OP.norm_rope(x["k"][sl], wk, pos, EPS, ROT, THETA).transpose(0, 1)
            V = x["v"][sl].double().transpose(0, 1)
            gate = x.get("gate")
            out, _ = OP.attn_prompt(K, V, 0, q, m.D ** -0.5, None if gate is None else gate[sl])
            return f64(out), (f64(K), f64(V))
        tail = torch.zeros(W - 1, x["x"].shape[1], device="cuda", dtype=x["x"].dtype)
        q, k, v, al, be, _ = OP.gdn_prompt_front(x["x"][sl], tail, self.w[li], x["a"][sl], x["b"][sl], m.Hk, m.dk, m.Hv, m.dv)
        o, S = OP.gdn_prompt(torch.zeros(m.Hv, m.dv, m.dk, device="cuda"), q, k, v, al, be, m.dk ** -0.5)
        return GF.gated_rmsnorm(f64(o), f64(x["z"][sl]), f64(x["w_norm"])), f64(S)


@pytest.mark.parametrize("spans", [[[(0, 130), (0, 71)]], [[(0, 64), (0, 0)], [(64, 65), (0, 71)], [(65, 130), (71, 71)]]])
def test_prompt_then_round_fp32(spans):
    st = Stack(F32, [130, 71])
    r = st.r
    p = st.make(201, 130)
    for sp in spans:
        idx, x = st.rows_of(sp)
        p.set_rows([b - a for a, b in sp])
        n = len(idx)
        full = {li: {k: (v if k == "w_norm" else torch.cat([v, v.new_full((201 - n, *v.shape[1:]), float("nan"))]))
                     for k, v in xs.items()} for li, xs in x.items()}  # padding behind the span
        p.run(full)
        for li in r.layers:
            st.x[li]["out"][idx] = full[li]["out"][:n]
    torch.cuda.synchronize()
    assert p.status() == 0 and r.len.tolist() == [130, 71]
    held = {(li, s): st.oracle(li, s) for li in r.layers for s in range(2)}
    for (li, s), (out, _) in held.items():
        check_close(st.x[li]["out"][sum(st.rows[:s]):sum(st.rows[:s + 1])], out, f"prompt, layer {li}, sequence {s}")
    r.run(reset_len=False)
    torch.cuda.synchronize()
    assert r.status() == 0
    for (li, s), (_, mem) in held.items():
        lo, hi = seq_slice(r, s)
        if li in r.attn:
            a = r.attn[li]
            ref = O.attn_tree_verify(*mem, st.rows[s], f64(a["q"][lo:hi]), f64(a["k_t"][lo:hi]), f64(a["v_t"][lo:hi]),
                                     r.parents[s], r.attn_scale)
            check_close(a["out"][lo:hi], ref, f"round, layer {li}, sequence {s}")
        else:
            g = r.gdn[li]
            ref = O.gdn_tree_verify(mem, *(f64(g[k][lo:hi]) for k in ("q", "k", "v", "alpha", "beta")), r.parents[s],
                                    r.gdn_scale)
            check_close(g["out"][lo:hi], ref, f"round, layer {li}, sequence {s}")
    assert r.len.tolist() == [130 + len(r.expected_paths[0]), 71 + len(r.expected_paths[1])]


def test_prompt_then_decode_fp32():
    """The prompt's last rows fed as decode steps: the same outputs as in the prompt."""
    st = Stack(F32, [40, 33])
    r = st.r
    p = st.make(73, 40)
    _, x = st.rows_of([(0, 39), (0, 32)])
    p2 = st.make(71, 39)
    p2.set_rows([39, 32])
    p2.run(x)
    _, x = st.rows_of([(39, 40), (32, 33)])
    pl = B.plan(512)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.zeros(max(16, B.tv_attn_workspace_bytes(pl, r.attn[1]["layer"], 2, 1, r.max_len)), dtype=torch.uint8,
                     device="cuda")
    for li in r.layers:
        y = x[li]
        if li in r.attn:
            layer = r.attn[li]["layer"]
            wq, wk = st.norms.get(li, (None, None))
            q, k = torch.empty_like(y["q"]), torch.empty_like(y["k"])
            B.tv_attn_norm_rope(layer, None, 2, r.len, r.max_len, wq, wk, EPS, ROT, THETA, y["q"], y["k"], q, k, status)
            if "gate" in y:
                B.tv_attn_decode_gated(pl, layer, 2, r.len, r.max_len, q, k, y["v"], y["gate"], y["out"], r.attn_scale, ws,
                                       status)
            else:
                B.tv_decode_step(pl, layer, None, 2, r.len, r.max_len, q, k, y["v"], None, None, y["out"], r.attn_scale,
                                 ws, status)
        else:
            B.tv_gdn_decode_fused(r.gdn[li]["layer"], p.fronts[li], 2, y["x"], y["a"], y["b"], y["z"], y["w_norm"],
                                  y["out"], r.gdn_scale, status)
            B.tv_gdn_conv_commit(p.fronts[li], None, 2, y["x"], status=status)
    B.tv_len_advance(r.len, None, 1, 2)
    torch.cuda.synchronize()
    assert p2.status() == 0 and int(status[0]) == 0 and r.len.tolist() == [40, 33]
    for li in r.layers:
        for s in range(2):
            out, mem = st.oracle(li, s)
            check_close(x[li]["out"][s], out[-1], f"decode, layer {li}, sequence {s}")
            if li in r.gdn:
                err = np.linalg.norm(f64(r.gdn[li]["layer"].S[s]) - mem) / np.linalg.norm(mem)
                assert err <= 2e-5, (li, s, err)


@pytest.mark.parametrize("D,d,Hv", [(64, 64, 4), (256, 128, 6)])
def test_prompt_graph_then_round_bf16(D, d, Hv):
    """A captured pass gives the eager pass's bits, also after other rows, and the round goes on from it."""
    st = Stack(BF, [150, 99], pad=15, D=D, d=d, Hv=Hv)
    r = st.r
    p = st.make(264, 200)
    p.set_rows(st.rows)

    def held():
        return ([x["out"][:249].clone() for x in st.x.values()]
                + [t[:, :n].clone() for a in r.attn.values() for kv in (a["layer"].K, a["layer"].V) for t, n in zip(kv, st.rows)]
                + [t.clone() for g in r.gdn.values() for t in g["layer"].S] + [t.clone() for ts in st.tails.values() for t in ts])

    p.run(st.x)
    torch.cuda.synchronize()
    ref = held()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(st.x)
    for rows in ([20, 200], [0, 7], st.rows):
        st.reset()
        p.set_rows(rows)
        graph.replay()
        torch.cuda.synchronize()
        assert p.status() == 0 and r.len.tolist() == list(rows)
    for a, b in zip(ref, held()):
        assert torch.equal(a, b)
    S0 = {(li, s): g["layer"].S[s].clone() for li, g in r.gdn.items() for s in range(2)}
    r.verify()
    torch.cuda.synchronize()
    assert r.status() == 0
    for s in range(2):
        lo, hi = seq_slice(r, s)
        for li, a in r.attn.items():
            check_close(a["out"][lo:hi], oracle_attn(r, li, s, L=st.rows[s]), f"round, layer {li}, sequence {s}")
        for li, g in r.gdn.items():
            check_close(g["out"][lo:hi], oracle_gdn(r, li, s, S0=S0[li, s]), f"round, layer {li}, sequence {s}")
