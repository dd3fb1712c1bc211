"""The prompt calls without a GPU: descriptor layout, argument errors that the
host sees, and the fp64 prompt oracle pinned against the tree and decode
oracles (a prompt is a chain of decoded tokens)."""
from __future__ import annotations

import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import oracle.attn_front as OA
import oracle.gdn_front as OG
import oracle.prompt as OP
import oracle.tree_verify as OT
from speculative_tree_verify_masked_gb300 import binding as B
from speculative_tree_verify_masked_gb300 import build as BUILD

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "tv.h")
vp = ctypes.c_void_p
ref = ctypes.byref


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        BUILD.build()
    return B.lib()


def test_prompt_struct_layout_matches_c():
    names = [f for f, _ in B.tv_prompt._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "tv.h"\nint main(void) {\n printf("%zu\\n", sizeof(tv_prompt));\n'
    src += "".join(f' printf("%zu\\n", offsetof(tv_prompt, {n}));\n' for n in names) + " return 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-std=c11", "-I", os.path.dirname(HEADER), c, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(B.tv_prompt)] + [getattr(B.tv_prompt, n).offset for n in names]


def prompts_refused():
    """Descriptors every prompt call answers with TV_ERR_ARG."""
    ok = dict(n_seq=1, n_total=8, n_max=8, row_off=0x1000, status=0x2000)
    for change in (dict(n_seq=0), dict(n_seq=9), dict(n_total=-1), dict(n_total=(1 << 20) + 1), dict(n_max=9),
                   dict(n_max=-1), dict(row_off=None), dict(status=None), dict(row_off=0x1004), dict(status=0x2008)):
        d = {**ok, **change}
        yield B.tv_prompt(d["n_seq"], d["n_total"], d["n_max"], d["row_off"], d["status"])


def good_prompt(n_total=8):
    return B.tv_prompt(1, n_total, n_total, 0x1000, 0x2000)


def attn_layer(dtype=B.TV_BF16, Hq=24, Hkv=4, D=256, cap=64, k=0x3000, v=0x4000):
    return B.tv_attn_layer(dtype, Hq, Hkv, D, cap, (vp * 8)(*[k] * 8), (vp * 8)(*[v] * 8))


def test_attn_prompt_refusals(L):
    big = 1 << 40

    def call(layer=None, pr=None, ln=vp(16), ml=8, q=vp(16), gate=None, out=vp(16), scale=0.1, ws=vp(256), wb=big):
        layer = attn_layer() if layer is None else layer
        return L.tv_attn_prompt(ref(layer), ref(pr or good_prompt()), ln, ml, q, gate, out, scale, ws, wb, None)

    assert L.tv_attn_prompt(None, ref(good_prompt()), vp(16), 8, vp(16), None, vp(16), 0.1, vp(256), big, None) == 1
    assert L.tv_attn_prompt(ref(attn_layer()), None, vp(16), 8, vp(16), None, vp(16), 0.1, vp(256), big, None) == 1
    for pr in prompts_refused():
        assert call(pr=pr) == 1
    for kw in (dict(ln=None), dict(q=None), dict(out=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(ml=-1), dict(ml=65), dict(layer=attn_layer(cap=0)),
               dict(layer=attn_layer(k=None)), dict(layer=attn_layer(v=None))):
        assert call(**kw) == 1, kw
    for kw in (dict(ln=vp(20)), dict(q=vp(24)), dict(gate=vp(24)), dict(out=vp(8)), dict(layer=attn_layer(k=0x3008))):
        assert call(**kw) == 4, kw
    assert call(layer=attn_layer(dtype=3)) == 3
    for bad in (dict(D=96), dict(Hq=23), dict(Hq=0), dict(Hkv=0), dict(Hq=129, Hkv=1)):
        assert call(layer=attn_layer(**bad)) == 2, bad
    assert call(pr=good_prompt(0), q=None, out=None, ws=None, wb=0) == 0  # no rows: nothing to do


def test_norm_rope_refusals(L):
    def prompt(layer=None, pr=None, ln=vp(16), ml=8, qn=vp(16), kn=vp(16), eps=1e-6, rot=64, th=1e7, q=vp(16), v=vp(16)):
        layer = attn_layer() if layer is None else layer
        return L.tv_attn_prompt_front(ref(layer), ref(pr or good_prompt()), ln, ml, qn, kn, eps, rot, th, q, vp(16), v,
                                      vp(16), None)

    def decode(layer=None, n=1, ln=vp(16), ml=8, qn=vp(16), kn=vp(16), eps=1e-6, rot=64, th=1e7, q=vp(16), st=vp(16)):
        layer = attn_layer() if layer is None else layer
        return L.tv_attn_norm_rope(ref(layer), None, n, ln, ml, qn, kn, eps, rot, th, q, vp(16), vp(16), vp(16), st, None)

    for call in (prompt, decode):
        for kw in (dict(ln=None), dict(q=None), dict(ml=-1), dict(ml=65), dict(qn=None), dict(kn=None), dict(eps=0.0),
                   dict(eps=float("nan")), dict(eps=float("inf")), dict(rot=63), dict(rot=-2), dict(rot=258), dict(th=1.0),
                   dict(th=float("inf"))):
            assert call(**kw) == 1, (call, kw)
        for kw in (dict(ln=vp(20)), dict(q=vp(24)), dict(qn=vp(20))):
            assert call(**kw) == 4, (call, kw)
        assert call(layer=attn_layer(dtype=9)) == 3
        for bad in (dict(D=32), dict(Hq=23), dict(Hkv=0)):
            assert call(layer=attn_layer(**bad)) == 2, bad
    for pr in prompts_refused():
        assert prompt(pr=pr) == 1
    assert prompt(layer=attn_layer(v=None)) == 1 and prompt(layer=attn_layer(v=0x4004)) == 4 and prompt(v=None) == 1
    assert prompt(pr=good_prompt(0), q=None, v=None) == 0
    assert decode(n=0) == 1 and decode(n=9) == 1 and decode(st=None) == 1 and decode(st=vp(20)) == 4
    tree = B.tv_tree(1, 0, 0, None, None, None, None)
    assert L.tv_attn_norm_rope(ref(attn_layer()), ref(tree), 1, vp(16), 8, None, None, 0.0, 64, 1e7, vp(16), vp(16),
                               vp(16), vp(16), None, None) == 1


def test_gdn_prompt_refusals(L):
    big = 1 << 40

    def layer(dtype=B.TV_BF16, Hk=4, Hv=8, dk=128, dv=128, S=0x3000):
        return B.tv_gdn_layer(dtype, Hk, Hv, dk, dv, (vp * 8)(*[S] * 8))

    def call(lay=None, pr=None, args=None, scale=0.1, ws=vp(256), wb=big):
        args = args or [vp(16)] * 6
        return L.tv_gdn_prompt(ref(lay or layer()), ref(pr or good_prompt()), *args, scale, ws, wb, None)

    for pr in prompts_refused():
        assert call(pr=pr) == 1
    for i in range(6):
        assert call(args=[None if j == i else vp(16) for j in range(6)]) == 1
        assert call(args=[vp(24) if j == i else vp(16) for j in range(6)]) == 4
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == 1
    assert call(lay=layer(S=None)) == 1 and call(lay=layer(S=0x3004)) == 4 and call(lay=layer(dtype=5)) == 3
    for bad in (dict(Hk=3), dict(Hk=0), dict(dk=32), dict(dk=256), dict(dv=0), dict(dv=257)):
        assert call(lay=layer(**bad)) == 2, bad
    assert call(pr=good_prompt(0), args=[None] * 6, ws=None, wb=0) == 0


def test_gdn_prompt_front_refusals(L):
    def layer(dtype=B.TV_BF16, Hk=4, Hv=8, dk=128, dv=128, W=4, wconv=0x2000, tail=0x3000):
        return B.tv_gdn_front_layer(dtype, Hk, Hv, dk, dv, W, wconv, (vp * 8)(*[tail] * 8))

    def call(lay=None, pr=None, args=None):
        return L.tv_gdn_prompt_front(ref(lay or layer()), ref(pr or good_prompt()), *(args or [vp(16)] * 8), None)

    for pr in prompts_refused():
        assert call(pr=pr) == 1
    for i in range(8):
        assert call(args=[None if j == i else vp(16) for j in range(8)]) == 1
        assert call(args=[vp(24) if j == i else vp(16) for j in range(8)]) == 4
    assert call(lay=layer(tail=None)) == 1 and call(lay=layer(tail=0x3004)) == 4 and call(lay=layer(dtype=5)) == 3
    assert call(lay=layer(wconv=0x2004)) == 4
    for bad in (dict(W=0), dict(W=9), dict(dk=96, dv=96), dict(dv=64), dict(Hk=0)):
        assert call(lay=layer(**bad)) == 2, bad
    assert call(pr=good_prompt(0), args=[None] * 8) == 0


def test_binding_refuses_wrong_buffers():
    """The wrappers look at dtype, contiguity, size and place before the C call takes raw pointers."""
    S = [torch.zeros(2, 64, 64)]
    layer = B.GdnLayer(S, 2, torch.float32)
    prompt = B.Prompt([4], device="cpu")
    good = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):  # not on a GPU
        B.tv_gdn_prompt(layer, prompt, good, good, good, good, good, good, 0.1, None, stream=0)
    with pytest.raises(ValueError):
        prompt.set_rows([5])
    with pytest.raises(ValueError):
        prompt.set_rows([1, 1])


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------
def test_oracle_attention_is_a_chain_of_decodes():
    rng = np.random.default_rng(1)
    Hq, Hkv, D, L0, n = 4, 2, 8, 5, 7
    K, V = rng.normal(size=(2, Hkv, L0 + n + 1, D))
    q = rng.normal(size=(n, Hq, D))
    out, reach = OP.attn_prompt(torch.tensor(K), torch.tensor(V), L0, torch.tensor(q), 0.3)
    for i in range(n):
        Kc, Vc = K.copy(), V.copy()
        want = OT.attn_decode(Kc, Vc, L0 + i, q[i], K[:, L0 + i], V[:, L0 + i], 0.3)
        assert np.abs(out[i].numpy() - want).max() < 1e-12
    assert bool((reach >= out.abs() - 1e-15).all())


def test_oracle_delta_rule_is_the_tree_verify_of_a_chain():
    rng = np.random.default_rng(2)
    Hk, Hv, dk, dv, n = 2, 4, 8, 6, 9
    S = rng.normal(size=(Hv, dv, dk))
    q, k = rng.normal(size=(2, n, Hk, dk))
    v, alpha, beta = rng.normal(size=(n, Hv, dv)), rng.uniform(size=(n, Hv)), rng.uniform(size=(n, Hv))
    parent = [-1] + list(range(n - 1))
    want = OT.gdn_tree_verify(S, q, k, v, alpha, beta, parent, 0.5)
    state = OT.commit_gdn(S, k, v, alpha, beta, list(range(n)))
    out, got = OP.gdn_prompt(*(torch.tensor(x) for x in (S, q, k, v, alpha, beta)), 0.5)
    assert np.abs(out.numpy() - want).max() < 1e-12 and np.abs(got.numpy() - state).max() < 1e-12


def test_oracle_front_ends_are_the_tree_forms_of_a_chain():
    rng = np.random.default_rng(3)
    Hk, Hv, d, W, n = 2, 3, 4, 4, 6
    C = 2 * Hk * d + Hv * d
    x, tail, w = rng.normal(size=(n, C)), rng.normal(size=(W - 1, C)), rng.normal(size=(C, W))
    a, b = rng.normal(size=(2, n, Hv))
    parent = [-1] + list(range(n - 1))
    want = OG.gdn_front(x, tail, w, a, b, parent, Hk, d, Hv, d)
    got = OP.gdn_prompt_front(*(torch.tensor(t) for t in (x, tail, w, a, b)), Hk, d, Hv, d)
    for g, r in zip(got, want):
        assert np.abs(g.numpy() - r).max() < 1e-12
    assert np.array_equal(got[5].numpy(), OG.commit_tail(tail, x, list(range(n))))
    h = rng.normal(size=(n, 2, 8))
    turned = OP.norm_rope(torch.tensor(h), None, torch.arange(n) + 11, 1e-6, 6, 1e4)
    for i in range(n):
        assert np.abs(turned[i].numpy() - OA.rope(h[i], 11 + i, 6, 1e4)).max() < 1e-12
    unit = OP.norm_rope(torch.tensor(h), torch.ones(8), torch.zeros(n), 1e-12, 0, 1e4)
    assert np.abs((unit.numpy() ** 2).mean(-1) - 1).max() < 1e-9


def test_shared_memory_refused(L):
    """Outputs that share memory with inputs other rows still read: TV_ERR_ARG, before anything is launched."""
    q, n = 1 << 20, 8
    a = attn_layer()
    row = 24 * 256 * 2
    for out in (q, q + 16, q + n * row - 16, q - n * row + 16):
        assert L.tv_attn_prompt(ref(a), ref(good_prompt(n)), vp(16), 8, vp(q), None, vp(out), 0.1, None, 0, None) == 1
    for out in (q + n * row, q - n * row):  # side by side: on to the next check (here the missing workspace)
        big = B.tv_attn_layer(B.TV_BF16, 24, 4, 256, 1 << 20, (vp * 8)(*[0x3000] * 8), (vp * 8)(*[0x4000] * 8))
        assert L.tv_attn_prompt(ref(big), ref(good_prompt(n)), vp(16), 1 << 19, vp(q), None, vp(out), 0.1, None, 0, None) == 8
    g = B.tv_gdn_layer(B.TV_BF16, 4, 8, 128, 128, (vp * 8)(*[0x3000] * 8))
    k, v, far = q + (1 << 20), q + (2 << 20), 1 << 30
    for out in (q + 16, k, v - 16):
        assert L.tv_gdn_prompt(ref(g), ref(good_prompt(n)), vp(q), vp(k), vp(v), vp(far), vp(far), vp(out), 0.1, None, 0, None) == 1
    f = B.tv_gdn_front_layer(B.TV_BF16, 4, 8, 128, 128, 4, 0x2000, (vp * 8)(*[0x3000] * 8))
    c = 2 * 4 * 128 + 8 * 128
    for i in range(3):
        outs = [q, k, v]
        x = outs[i] - n * c * 2 + 16
        assert L.tv_gdn_prompt_front(ref(f), ref(good_prompt(n)), vp(x), vp(far), vp(far), *map(vp, outs), vp(far), vp(far), None) == 1


def test_binding_refuses_host_memory():
    """Buffers that are not GPU memory never reach the library."""
    with pytest.raises(ValueError):
        B._ws_bytes(torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B._need("call", q=(torch.zeros(16), torch.float32, 16))
    assert B._ws_bytes(None) == 0
