"""Refusals of the prompt calls that the host sees: spans, and buffers of the wrong kind."""
from __future__ import annotations

from tests.test_prompt_cpu import L, good_prompt, prompts_refused, ref, vp  # noqa: F401 (L is a fixture)


def test_span_call_refusals(L):  # noqa: F811
    for pr in prompts_refused():
        assert L.tv_prompt_check(ref(pr), vp(16), 8, 64, None) == 1
        assert L.tv_prompt_advance(ref(pr), vp(16), None) == 1
    assert L.tv_prompt_check(None, vp(16), 8, 64, None) == 1 and L.tv_prompt_advance(None, vp(16), None) == 1
    assert L.tv_prompt_check(ref(good_prompt()), None, 8, 64, None) == 1
    assert L.tv_prompt_advance(ref(good_prompt()), None, None) == 1
    for ml, cap in ((-1, 64), (65, 64), (0, 0)):
        assert L.tv_prompt_check(ref(good_prompt()), vp(16), ml, cap, None) == 1
    assert L.tv_prompt_check(ref(good_prompt()), vp(20), 8, 64, None) == 4
    assert L.tv_prompt_advance(ref(good_prompt()), vp(20), None) == 4
    assert L.tv_prompt_check(ref(good_prompt(0)), vp(16), 8, 64, None) == 0
    assert L.tv_prompt_advance(ref(good_prompt(0)), vp(16), None) == 0


def test_norm_rope_shared_memory_refused(L):  # noqa: F811
    """Rows formed in place, or apart from the raw ones: nothing between, before anything is launched."""
    from tests.test_prompt_cpu import attn_layer

    a, n = attn_layer(), 8
    qb, kb = n * 24 * 256 * 2, n * 4 * 256 * 2  # bytes of the packed rows
    Q, K, V, far = 1 << 24, 1 << 26, 1 << 27, 1 << 28

    def prompt(q):
        return L.tv_attn_prompt_front(ref(a), ref(good_prompt(n)), vp(16), 8, None, None, 0.0, 64, 1e7, vp(Q), vp(K), vp(V), vp(q), None)

    for q in (Q + 16, Q - 16, Q + qb - 16, Q - qb + 16, K, K + kb - 16, K - qb + 16, V, V + 16):
        assert prompt(q) == 1, hex(q)

    def decode(q, k):
        return L.tv_attn_norm_rope(ref(a), None, n, vp(16), 8, None, None, 0.0, 64, 1e7, vp(Q), vp(K), vp(q), vp(k), vp(16), None)

    for q, k in ((Q + 16, far), (K, far), (far, K + 16), (far, Q + 512), (far, far + 16), (Q, Q), (K, Q)):
        assert decode(q, k) == 1, (hex(q), hex(k))


def test_gates_and_shared_memory_refused(L):  # noqa: F811
    import ctypes

    from speculative_tree_verify_masked_gb300 import binding as B
    from tests.test_prompt_cpu import attn_layer

    a, n, far = attn_layer(), 8, 1 << 30
    rows = n * 24 * 256 * 2
    for gate in (far + 16, far - 16, far + rows - 16, far - rows + 16):
        assert L.tv_attn_prompt(ref(a), ref(good_prompt(n)), vp(16), 8, vp(1 << 20), vp(gate), vp(far), 0.1, None, 0, None) == 1
    g = B.tv_gdn_layer(B.TV_BF16, 4, 8, 128, 128, (ctypes.c_void_p * 8)(*[0x3000] * 8))
    q, k, v = 1 << 20, 2 << 20, 3 << 20
    for al, be in ((far, 5 << 20), (5 << 20, far + 16), (far - n * 8 * 4 + 16, 5 << 20), (far + n * 8 * 128 * 2 - 16, 5 << 20)):
        assert L.tv_gdn_prompt(ref(g), ref(good_prompt(n)), vp(q), vp(k), vp(v), vp(al), vp(be), vp(far), 0.1, None, 0, None) == 1
    f = B.tv_gdn_front_layer(B.TV_BF16, 4, 8, 128, 128, 4, 0x2000, (ctypes.c_void_p * 8)(*[0x3000] * 8))
    x, ar, br, al, be = far, 5 << 20, 6 << 20, 7 << 20, 8 << 20

    def front(x=x, ar=ar, br=br, q=q, k=k, v=v, al=al, be=be):
        return L.tv_gdn_prompt_front(ref(f), ref(good_prompt(n)), *map(vp, (x, ar, br, q, k, v, al, be)), None)

    for kw in (dict(ar=q), dict(br=k + 16), dict(ar=v), dict(al=x), dict(be=x + 16), dict(al=ar + 16), dict(be=ar - 16),
               dict(al=br + 16), dict(be=br + 32)):
        assert front(**kw) == 1, kw
