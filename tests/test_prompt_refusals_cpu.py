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
