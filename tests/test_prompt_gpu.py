"""The prompt calls on the GPU against their fp64 definitions (oracle/prompt.py):
head norms with rotation, causal attention over packed prompts, the Gated
DeltaNet front end and the gated delta rule; plus padding, refusals, capture
into graphs and streams.

Tolerances, derived before the first run.  A rounding to a type is off by at
most half a step, eps/2 of the value: bf16 u = 2^-8, fp32 2^-24.
 * attention, bf16: the output rounding (u |ref|), the probabilities' rounding
   acting on |V| (u reach), the row sum of rounded probabilities (u |ref|), and
   fp32 scores: D products of unit normal values leave the scaled score within
   2e-4, so 4e-4 reach for weight and sum together; a gate multiplies all of it
   and adds fp32 roundings only.  fp32: scores within D 2^-24 sum|q k| scale
   < 4e-5 give 8e-5 reach at most; the output rounding is far below.
 * norm and rotation: u |ref| for the final rounding plus fp32 arithmetic of a
   head's values, whose errors are within 16 steps (2^-20) of its largest one.
 * delta rule: outputs as the verify tests hold them (gpu_helpers.check_close),
   states to 2e-5 in rel-L2: operands split into two bf16 parts leave 2^-17 of
   each product, some four products deep.
 * front end: u |ref| + 2e-6 max|ref| (SiLU's fast exponential and divide are a
   few fp32 steps), gates 2e-6.
"""
from __future__ import annotations

import math

import pytest
import torch

import oracle.prompt as OP
from speculative_tree_verify_masked_gb300 import binding as B
from tests.gpu_helpers import check_close, f64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
STATE_REL = 2e-5
NAN = float("nan")


def rnd(gen, *shape, dtype=F32):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def within(got, ref, bound, what):
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    over = (got - ref).abs() - bound
    assert float(over.max()) <= 0, f"{what}: {float(over.max()):.3e} over its bound at {int(over.argmax())}"


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
class Attn:
    """One attention call's buffers.  Everything no row may see is NaN: cache
    rows behind each sequence, packed rows behind the last one."""

    def __init__(self, rows, ctx, Hq=24, Hkv=4, D=256, dtype=BF, gate=False, seed=1, pad=0, cap=None, n_max=None):
        g = gen_of(seed)
        self.rows, self.ctx, self.dtype, n = rows, ctx, dtype, sum(rows)
        self.cap = cap or max(L + m for L, m in zip(ctx, rows)) + 7
        self.K, self.V = [], []
        for L, m in zip(ctx, rows):
            for kv in (self.K, self.V):
                t = torch.full((Hkv, self.cap, D), NAN, device="cuda", dtype=dtype)
                t[:, :L + m] = rnd(g, Hkv, L + m, D, dtype=dtype)
                kv.append(t)
        self.q = torch.full((n + pad, Hq, D), NAN, device="cuda", dtype=dtype)
        self.q[:n] = rnd(g, n, Hq, D, dtype=dtype)
        self.gate = rnd(g, n + pad, Hq, D, dtype=dtype) if gate else None
        self.out = torch.full_like(self.q, 7.0)
        self.scale = D ** -0.5
        self.layer = B.AttnLayer(self.K, self.V, Hq)
        self.prompt = B.Prompt(rows, n_total=n + pad, n_max=n_max)
        self.len = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.max_len = max(ctx)
        self.ws = torch.full((max(16, B.tv_attn_prompt_workspace_bytes(self.layer, self.prompt, self.max_len)),), 0xFF,
                             dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        B.tv_attn_prompt(self.layer, self.prompt, self.len, self.max_len, self.q, self.gate, self.out, self.scale,
                         self.ws, stream)

    def check(self, what=""):
        torch.cuda.synchronize()
        assert self.prompt.status_code() == 0
        off = 0
        for s, (L, n) in enumerate(zip(self.ctx, self.rows)):
            gate = None if self.gate is None else self.gate[off:off + n]
            ref, reach = OP.attn_prompt(self.K[s], self.V[s], L, self.q[off:off + n], self.scale, gate)
            if n:
                noise = 4e-4 if self.dtype == BF else 8e-5
                u = U[self.dtype]
                within(self.out[off:off + n], ref, 2 * u * ref.abs() + (u + noise) * reach + 1e-30,
                       f"{what} sequence {s}")
            off += n
        assert bool((self.out[off:] == 7.0).all()), "rows behind the last sequence were written"


LAYOUTS = [(24, 4, 256, BF), (2, 1, 64, F32), (16, 2, 128, BF), (8, 8, 64, BF), (6, 2, 256, F32), (5, 1, 128, F32),
           (128, 1, 64, BF), (7, 1, 256, BF)]
BATCHES = [([1], [0]), ([1], [1000]), ([2, 1], [0, 63]), ([63, 64, 65], [0, 1, 64]), ([127, 0, 1, 129], [5, 9, 128, 0]),
           ([0, 300], [77, 511]), ([21, 22, 43], [640, 0, 127])]


@pytest.mark.parametrize("Hq,Hkv,D,dtype", LAYOUTS)
@pytest.mark.parametrize("rows,ctx", BATCHES)
def test_attn_prompt_matches_oracle(Hq, Hkv, D, dtype, rows, ctx):
    a = Attn(rows, ctx, Hq, Hkv, D, dtype, gate=len(rows) % 2 == 0, seed=len(rows), pad=3)
    a.run()
    a.check()


@pytest.mark.parametrize("rows,ctx", [([1500], [0]), ([700, 30, 900], [0, 2000, 333]), ([24], [20000]), ([1], [40001]),
                                      ([200, 200], [6000, 6000])])
def test_attn_prompt_long(rows, ctx):
    a = Attn(rows, ctx, gate=True, seed=9)
    a.run()
    a.check()


def test_attn_prompt_full_cache_and_eight_sequences():
    rows, ctx = [1, 2, 3, 130, 5, 60, 7, 8], [255, 254, 253, 126, 251, 196, 249, 248]
    a = Attn(rows, ctx, 8, 2, 128, BF, seed=3, cap=256, n_max=200)
    a.run()
    a.check()


def test_attn_prompt_large_scores_and_equal_rows():
    """Scores far apart (one key wins, the rest vanish) and all equal (a plain mean)."""
    a = Attn([200], [100], 4, 1, 128, BF, seed=4)
    a.q *= 30
    a.run()
    torch.cuda.synchronize()
    ref, reach = OP.attn_prompt(a.K[0], a.V[0], 100, a.q, a.scale)
    # scores of size 30 |q.k| scale: their fp32 errors grow by as much
    within(a.out, ref, 2 * U[BF] * ref.abs() + (U[BF] + 30 * 4e-4) * reach, "large scores")
    a.q.zero_()
    a.run()
    a.check("equal scores")


def test_attn_prompt_slices_agree_with_the_whole():
    a = Attn([777], [0], seed=5)
    a.run()
    torch.cuda.synchronize()
    whole = a.out.clone()
    a.out.fill_(7.0)
    for r0, r1 in [(0, 1), (1, 129), (129, 600), (600, 777)]:
        p = B.Prompt([r1 - r0])
        L = torch.tensor([r0], dtype=torch.int32, device="cuda")
        ws = torch.empty(max(16, B.tv_attn_prompt_workspace_bytes(a.layer, p, r0)), dtype=torch.uint8, device="cuda")
        B.tv_attn_prompt(a.layer, p, L, r0, a.q[r0:r1], None, a.out[r0:r1], a.scale, ws)
    a.check("slices")
    ref, reach = OP.attn_prompt(a.K[0], a.V[0], 0, a.q, a.scale)
    within(whole, ref, 2 * U[BF] * ref.abs() + (U[BF] + 4e-4) * reach, "whole")


@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF, 256)])
def test_attn_prompt_device_errors_write_nothing(dtype, D):
    for rows, ctx, change, code in [([5, 6], [3, 4], lambda a: a.prompt.row_off.copy_(torch.tensor([0, 7, 5])), 12),
                                    ([5, 6], [3, 4], lambda a: a.prompt.row_off.copy_(torch.tensor([1, 5, 11])), 12),
                                    ([5, 6], [3, 4], lambda a: a.prompt.row_off.copy_(torch.tensor([0, 5, 12])), 12),
                                    ([5, 6], [3, 4], lambda a: a.prompt.row_off.copy_(torch.tensor([0, -1, 11])), 12),
                                    ([5, 6], [3, 4], lambda a: a.prompt.row_off.copy_(torch.tensor([0, 0, 11])), 12),
                                    ([5, 6], [3, 4], lambda a: a.len.copy_(torch.tensor([-1, 4])), 10),
                                    ([5, 6], [3, 4], lambda a: a.len.copy_(torch.tensor([3, 5])), 10)]:
        a = Attn(rows, ctx, 4, 2, D, dtype, seed=6)
        change(a)
        a.run()
        torch.cuda.synchronize()
        assert a.prompt.status_code() == code
        assert bool((a.out == 7.0).all())
    a = Attn([5, 6], [3, 4], 4, 2, D, dtype, seed=6, cap=11)
    a.max_len = 6
    a.len.copy_(torch.tensor([3, 6]))
    a.run()
    torch.cuda.synchronize()
    assert a.prompt.status_code() == 6 and bool((a.out == 7.0).all())
    a.len.copy_(torch.tensor([3, 4]))
    a.run()  # the word still holds the error
    torch.cuda.synchronize()
    assert bool((a.out == 7.0).all())
    a.prompt.status.zero_()
    a.run()
    a.check()


def test_attn_prompt_graph_replays_other_batches_on_another_stream():
    """One captured call serves every batch inside its bounds; two graphs that
    share a workspace run one behind the other."""
    a = Attn([300, 200, 4], [1000, 0, 77], 24, 4, 256, BF, seed=7, pad=60, n_max=400)
    b = Attn([90], [3000], 24, 4, 256, BF, seed=8)
    need = max(a.ws.numel(), b.ws.numel())
    a.ws = b.ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    graphs = []
    for x in (a, b):
        x.run(st)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            x.run()
        graphs.append(g)
    for x in (a, b):
        x.out.fill_(7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        graphs[0].replay()
        graphs[1].replay()
    a.check("first batch")
    b.check("second graph")
    a.out.fill_(7.0)
    a.rows = [150, 0, 4]  # fewer rows: sequence 2's move up, the last rows become padding
    a.prompt.set_rows(a.rows)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        graphs[1].replay()
        graphs[0].replay()
    torch.cuda.synchronize()
    a.check("second batch")


# ---------------------------------------------------------------------------
# norms and rotation
# ---------------------------------------------------------------------------
EPS, THETA = 1e-6, 1e7


def nr_bound(ref, dtype):
    return U[dtype] * ref.abs() + 2.0 ** -20 * ref.abs().amax(-1, keepdim=True) + 1e-30


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(24, 4, 256, BF), (2, 1, 64, F32), (16, 2, 128, BF), (3, 3, 64, BF), (5, 1, 256, F32)])
@pytest.mark.parametrize("rot", [0, 2, 6, 16, 20, 32, 64, "all"])
@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope_prompt_and_decode(Hq, Hkv, D, dtype, rot, norm):
    rot = D if rot == "all" else rot
    g = gen_of(11)
    rows, ctx = [3, 0, 1, 9], [0, 5, (1 << 20) - 1, 4095]
    n, pad = sum(rows), 2
    cap = max(L + m for L, m in zip(ctx, rows)) if D == 64 else 8192
    if D != 64:
        ctx[2] = 8191
    q_raw, k_raw, v = (rnd(g, n + pad, H, D, dtype=dtype) for H in (Hq, Hkv, Hkv))
    q_raw *= 5
    w = [1 + 0.2 * rnd(g, D) if norm else None for _ in range(2)]
    K, V = ([torch.full((Hkv, cap, D), 7.0, device="cuda", dtype=dtype) for _ in rows] for _ in range(2))
    layer, prompt = B.AttnLayer(K, V, Hq), B.Prompt(rows, n_total=n + pad)
    L = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    q = torch.full_like(q_raw, 7.0)
    B.tv_attn_prompt_front(layer, prompt, L, max(ctx), w[0], w[1], EPS, rot, THETA, q_raw, k_raw, v, q)
    torch.cuda.synchronize()
    assert prompt.status_code() == 0
    pos = torch.tensor([c + i for c, m in zip(ctx, rows) for i in range(m)], device="cuda")
    rq = OP.norm_rope(q_raw[:n], w[0], pos, EPS, rot, THETA)
    rk = OP.norm_rope(k_raw[:n], w[1], pos, EPS, rot, THETA)
    within(q[:n], rq, nr_bound(rq, dtype), "q")
    assert bool((q[n:] == 7.0).all())
    off = 0
    for s, (c, m) in enumerate(zip(ctx, rows)):
        r = rk[off:off + m].transpose(0, 1)
        if m:
            within(K[s][:, c:c + m], r, nr_bound(r, dtype), "k")
            assert torch.equal(V[s][:, c:c + m], v[off:off + m].transpose(0, 1))
        for t in (K[s], V[s]):
            assert bool((t[:, :c] == 7.0).all()) and bool((t[:, c + m:] == 7.0).all())
        off += m
    # decode form: the same rows one at a time, in place, give the same bits
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    first = [i for i, (o, m) in enumerate(zip([0, 3, 3, 4], rows)) if m]
    at = torch.tensor([sum(rows[:i]) for i in first], device="cuda")
    lens = torch.tensor([ctx[i] for i in first], dtype=torch.int32, device="cuda")
    dq, dk = q_raw[at].clone(), k_raw[at].clone()
    B.tv_attn_norm_rope(layer, None, len(first), lens, max(ctx), w[0], w[1], EPS, rot, THETA, dq, dk, dq, dk, status)
    torch.cuda.synchronize()
    assert int(status[0]) == 0 and torch.equal(dq, q[at])
    for j, i in enumerate(first):
        assert torch.equal(dk[j], K[i][:, ctx[i]])


def test_norm_rope_tree_rows_equal_decode_rows():
    g = gen_of(12)
    parents = [[-1, 0, 0, 1, 3], [-1, 0]]
    Hq, Hkv, D = 6, 2, 128
    K = [torch.zeros(Hkv, 256, D, device="cuda", dtype=BF) for _ in parents]
    layer, tree = B.AttnLayer(K, K, Hq), B.Tree(parents)
    L = torch.tensor([100, 31], dtype=torch.int32, device="cuda")
    q_raw, k_raw = rnd(g, 7, Hq, D, dtype=BF), rnd(g, 7, Hkv, D, dtype=BF)
    w = [1 + 0.2 * rnd(g, D) for _ in range(2)]
    q, k = torch.empty_like(q_raw), torch.empty_like(k_raw)
    B.tv_tree_prepare(tree)
    B.tv_attn_norm_rope(layer, tree, 2, L, 200, w[0], w[1], EPS, 32, THETA, q_raw, k_raw, q, k)
    depth = [0, 1, 1, 2, 3, 0, 1]
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    for i in range(7):
        at = torch.tensor([(100 if i < 5 else 31) + depth[i]], dtype=torch.int32, device="cuda")
        dq, dk = torch.empty_like(q[:1]), torch.empty_like(k[:1])
        B.tv_attn_norm_rope(layer, None, 1, at, 200, w[0], w[1], EPS, 32, THETA, q_raw[i:i + 1].contiguous(),
                            k_raw[i:i + 1].contiguous(), dq, dk, status)
        torch.cuda.synchronize()
        assert torch.equal(dq[0], q[i]) and torch.equal(dk[0], k[i])
    assert tree.status_code() == 0 and int(status[0]) == 0


def test_prompt_front_device_errors_write_nothing():
    K, V = [torch.full((2, 16, 64), 7.0, device="cuda")], [torch.full((2, 16, 64), 7.0, device="cuda")]
    layer = B.AttnLayer(K, V, 2)
    q_raw, k_raw, v = (torch.ones(9, 2, 64, device="cuda") for _ in range(3))
    for L, mx, code in ((8, 8, 6), (9, 8, 10), (-1, 8, 10)):
        prompt, q = B.Prompt([9]), torch.full_like(q_raw, 7.0)
        ln = torch.tensor([L], dtype=torch.int32, device="cuda")
        B.tv_attn_prompt_front(layer, prompt, ln, mx, None, None, EPS, 64, THETA, q_raw, k_raw, v, q)
        torch.cuda.synchronize()
        assert prompt.status_code() == code
        assert all(bool((t == 7.0).all()) for t in (q, K[0], V[0]))


# ---------------------------------------------------------------------------
# Gated DeltaNet front end
# ---------------------------------------------------------------------------
class Front:
    def __init__(self, rows, Hk, Hv, d, W, dtype, seed=1, pad=0):
        g = gen_of(seed)
        n = sum(rows) + pad
        self.rows, self.dims, C = rows, (Hk, d, Hv, d), 2 * Hk * d + Hv * d
        self.x = rnd(g, n, C, dtype=dtype)
        self.a, self.b = 3 * rnd(g, n, Hv), 3 * rnd(g, n, Hv)
        self.w = rnd(g, C, W) * W ** -0.5
        self.tails = [rnd(g, W - 1, C, dtype=dtype) for _ in rows]
        self.q, self.k = (torch.full((n, Hk, d), 7.0, device="cuda", dtype=dtype) for _ in range(2))
        self.v = torch.full((n, Hv, d), 7.0, device="cuda", dtype=dtype)
        self.alpha, self.beta = (torch.full((n, Hv), 7.0, device="cuda") for _ in range(2))
        self.layer = B.GdnFrontLayer(Hk, Hv, d, d, self.w, self.tails, dtype)
        self.prompt = B.Prompt(rows, n_total=n)

    def outs(self):
        return self.q, self.k, self.v, self.alpha, self.beta

    def run(self, stream=None):
        B.tv_gdn_prompt_front(self.layer, self.prompt, self.x, self.a, self.b, *self.outs(), stream=stream)


@pytest.mark.parametrize("Hk,Hv,d,dtype", [(16, 48, 128, BF), (2, 2, 64, F32), (3, 6, 64, BF), (1, 5, 128, F32)])
@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("rows", [[1], [2, 0, 1, 3], [67, 33, 1, 160]])
def test_gdn_prompt_front_matches_oracle(Hk, Hv, d, dtype, W, rows):
    f = Front(rows, Hk, Hv, d, W, dtype, seed=W, pad=2)
    old = [t.clone() for t in f.tails]
    f.run()
    torch.cuda.synchronize()
    assert f.prompt.status_code() == 0
    off = 0
    for s, n in enumerate(rows):
        sl = slice(off, off + n)
        if n:
            q, k, v, al, be, tail = OP.gdn_prompt_front(f.x[sl], old[s], f.w, f.a[sl], f.b[sl], *f.dims)
            for got, ref, name in ((f.q, q, "q"), (f.k, k, "k"), (f.v, v, "v")):
                within(got[sl], ref, U[dtype] * ref.abs() + 2e-6 * ref.abs().max(), name)
            within(f.alpha[sl], al, 2e-6 + 0 * al, "alpha")
            within(f.beta[sl], be, 2e-6 + 0 * be, "beta")
        else:
            tail = old[s]
        assert torch.equal(f.tails[s], tail)
        off += n
    for t in f.outs():
        assert bool((t[off:] == 7.0).all())


def test_gdn_prompt_front_slices_give_the_same_bits():
    a, b = (Front([200], 4, 8, 128, 4, BF, seed=21) for _ in range(2))
    a.run()
    for r0, r1 in ((0, 1), (1, 3), (3, 70), (70, 200)):
        B.tv_gdn_prompt_front(b.layer, B.Prompt([r1 - r0]), b.x[r0:r1], b.a[r0:r1], b.b[r0:r1],
                              *(t[r0:r1] for t in b.outs()))
    torch.cuda.synchronize()
    for x, y in zip(a.outs() + tuple(a.tails), b.outs() + tuple(b.tails)):
        assert torch.equal(x, y)


def test_gdn_prompt_front_device_errors_write_nothing():
    f = Front([4, 5], 2, 2, 64, 4, F32)
    old = [t.clone() for t in f.tails]
    f.prompt.row_off.copy_(torch.tensor([0, 6, 5]))
    f.run()
    torch.cuda.synchronize()
    assert f.prompt.status_code() == 12
    assert all(bool((t == 7.0).all()) for t in f.outs()) and all(torch.equal(x, y) for x, y in zip(old, f.tails))


# ---------------------------------------------------------------------------
# gated delta rule
# ---------------------------------------------------------------------------
class Gdn:
    def __init__(self, rows, Hk=16, Hv=48, dk=128, dv=128, dtype=BF, seed=1, pad=0, spread=6.0, n_max=None):
        g = gen_of(seed)
        n = sum(rows)
        self.rows, self.dtype = rows, dtype
        self.q, self.k = (torch.full((n + pad, Hk, dk), NAN, device="cuda", dtype=dtype) for _ in range(2))
        for t in (self.q, self.k):
            t[:n] = torch.nn.functional.normalize(rnd(g, n, Hk, dk), dim=-1).to(dtype)
        self.v = torch.full((n + pad, Hv, dv), NAN, device="cuda", dtype=dtype)
        self.v[:n] = rnd(g, n, Hv, dv, dtype=dtype)
        a = rnd(g, n + pad, Hv) - spread * torch.rand(Hv, generator=g, device="cuda")
        self.alpha = torch.exp(-torch.nn.functional.softplus(a))
        self.beta = torch.sigmoid(rnd(g, n + pad, Hv))
        self.S = [0.1 * rnd(g, Hv, dv, dk) for _ in rows]
        self.S0 = [t.clone() for t in self.S]
        self.out = torch.full_like(self.v, 7.0)
        self.scale = dk ** -0.5
        self.layer, self.prompt = B.GdnLayer(self.S, Hk, dtype), B.Prompt(rows, n_total=n + pad, n_max=n_max)
        self.ws = torch.full((max(16, B.tv_gdn_prompt_workspace_bytes(self.layer, self.prompt)),), 0xFF,
                             dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        B.tv_gdn_prompt(self.layer, self.prompt, self.q, self.k, self.v, self.alpha, self.beta, self.out, self.scale,
                        self.ws, stream)

    def check(self, what=""):
        torch.cuda.synchronize()
        assert self.prompt.status_code() == 0
        off = 0
        for s, n in enumerate(self.rows):
            sl = slice(off, off + n)
            ref, S = OP.gdn_prompt(self.S0[s], self.q[sl], self.k[sl], self.v[sl], self.alpha[sl], self.beta[sl], self.scale)
            if n:
                check_close(self.out[sl], f64(ref), f"{what} out {s}")
                err = float((self.S[s].double() - S).norm() / S.norm())
                assert err <= STATE_REL, f"{what}: state {s} rel-L2 {err:.2e}"
            else:
                assert torch.equal(self.S[s], self.S0[s])
            off += n
        assert bool((self.out[off:] == 7.0).all()), "rows behind the last sequence were written"


GDN_SHAPES = [(16, 48, 128, 128, BF), (2, 2, 64, 64, F32), (4, 8, 64, 64, BF), (1, 3, 128, 256, BF), (2, 2, 128, 24, BF),
              (3, 3, 64, 100, F32), (2, 4, 64, 96, BF)]


@pytest.mark.parametrize("Hk,Hv,dk,dv,dtype", GDN_SHAPES)
@pytest.mark.parametrize("rows", [[1], [2, 0, 3], [63, 64, 65], [128, 1, 0, 200], [300]])
def test_gdn_prompt_matches_oracle(Hk, Hv, dk, dv, dtype, rows):
    x = Gdn(rows, Hk, Hv, dk, dv, dtype, seed=len(rows) + rows[0], pad=3)
    x.run()
    x.check()


def test_gdn_prompt_long_memory():
    """Decays close to 1 over many blocks: errors of early rows would last."""
    x = Gdn([2000, 700], 4, 8, seed=31, spread=12.0)
    x.run()
    x.check()


def test_gdn_prompt_eight_sequences():
    x = Gdn([1, 70, 0, 129, 64, 5, 256, 33], 2, 6, seed=32, n_max=300)
    x.run()
    x.check()


@pytest.mark.parametrize("rows", [[200]])
def test_gdn_prompt_extreme_gates(rows):
    """alpha 0 and 1, beta 0 and 1, keys repeated: the state is cleared, kept,
    overwritten; decays inside a block under- and overflow nothing."""
    x = Gdn(rows, 2, 4, seed=33)
    x.alpha[::7] = 0.0
    x.alpha[1::7] = 1.0
    x.alpha[50:120, 0] = 1.0
    x.alpha[50:120, 1] = 1e-30
    x.beta[::5] = 1.0
    x.beta[2::5] = 0.0
    x.k[60:90] = x.k[60]
    x.run()
    x.check()


def test_gdn_prompt_slices_agree_with_the_whole():
    a, b = (Gdn([500], 4, 8, seed=34) for _ in range(2))
    a.run()
    a.check("whole")
    for r0, r1 in ((0, 1), (1, 130), (130, 194), (194, 500)):
        p = B.Prompt([r1 - r0])
        ws = torch.empty(max(16, B.tv_gdn_prompt_workspace_bytes(b.layer, p)), dtype=torch.uint8, device="cuda")
        B.tv_gdn_prompt(b.layer, p, b.q[r0:r1], b.k[r0:r1], b.v[r0:r1], b.alpha[r0:r1], b.beta[r0:r1], b.out[r0:r1],
                        b.scale, ws)
    b.check("slices")


def test_gdn_prompt_fp32_rows_equal_decode_steps():
    x = Gdn([40], 2, 4, 64, 64, F32, seed=35)
    S = [x.S0[0].clone()]
    layer, status = B.GdnLayer(S, 2, F32), torch.zeros(4, dtype=torch.int32, device="cuda")
    x.run()
    for t in range(40):
        o = torch.empty(1, 4, 64, device="cuda")
        B.tv_decode_step(None, None, layer, 1, None, 0, x.q[t:t + 1].contiguous(), x.k[t:t + 1].contiguous(),
                         x.v[t:t + 1].contiguous(), x.alpha[t:t + 1].contiguous(), x.beta[t:t + 1].contiguous(), o,
                         x.scale, None, status)
        torch.cuda.synchronize()
        assert torch.equal(o[0], x.out[t])
    assert torch.equal(S[0], x.S[0])


def test_gdn_prompt_graph_other_batches_and_stream():
    x = Gdn([150, 80], 4, 8, seed=36, pad=70, n_max=220)
    st = torch.cuda.Stream()
    x.run(st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        x.run()
    for rows in ([150, 80], [3, 220], [0, 129]):
        for s in range(2):
            x.S[s].copy_(x.S0[s])
        n = sum(rows)
        for t, fill in ((x.q, 0.05), (x.k, 0.05), (x.v, 0.5)):
            bad = torch.isnan(t)
            t[bad] = fill
        x.out.fill_(7.0)
        x.rows = rows
        x.prompt.set_rows(rows)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        x.check(str(rows))


def test_gdn_prompt_device_errors_write_nothing():
    x = Gdn([70, 80], 2, 4, seed=37)
    x.prompt.row_off.copy_(torch.tensor([0, 90, 80]))
    x.run()
    torch.cuda.synchronize()
    assert x.prompt.status_code() == 12
    assert bool((x.out == 7.0).all()) and all(torch.equal(a, b) for a, b in zip(x.S, x.S0))
