"""A prompt call over more sequences than its layer holds, or over a layer whose
tensors are not alike, is refused before the library sees a pointer."""
from __future__ import annotations

import pytest
import torch

from speculative_tree_verify_masked_gb300 import binding as B


def prompt(n):
    return B.Prompt([4] * n, device="cpu")


def layers(n):
    kv = [torch.zeros(2, 16, 64) for _ in range(n)]
    return (B.AttnLayer(kv, kv, 2), B.GdnLayer([torch.zeros(2, 64, 64) for _ in range(n)], 2, torch.float32),
            B.GdnFrontLayer(2, 2, 64, 64, torch.zeros(384, 4), [torch.zeros(3, 384) for _ in range(n)], torch.float32))


def calls(a, g, f, p):
    t, ln = torch.zeros(64, 2, 64), torch.zeros(8, dtype=torch.int32)
    yield lambda: B.tv_attn_prompt_front(a, p, ln, 8, None, None, 1e-6, 64, 1e4, t, t, t, t, stream=0)
    yield lambda: B.tv_attn_prompt(a, p, ln, 8, t, None, t, 0.1, None, stream=0)
    yield lambda: B.tv_gdn_prompt(g, p, t, t, t, t, t, t, 0.1, None, stream=0)
    yield lambda: B.tv_gdn_prompt_front(f, p, t, t, t, t, t, t, t, t, stream=0)


def test_more_sequences_than_the_layer_holds():
    for call in calls(*layers(2), prompt(3)):
        with pytest.raises(ValueError, match="3 sequences, but the layer holds 2"):
            call()


def test_layers_must_be_alike_gpu_memory():
    for call in calls(*layers(2), prompt(2)):  # (host memory here)
        with pytest.raises(ValueError, match="one GPU"):
            call()


def test_alike():
    class Gpu(torch.Tensor):
        def get_device(self):
            return 1 if self.numel() == 77 else 0

    def gpu(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(Gpu)

    assert not B._alike([gpu(2), gpu(77)], (2,), torch.float32) and B._alike([gpu(77), gpu(77)], (77,), torch.float32)

    assert B._alike([gpu(2, 16, 64), gpu(2, 16, 64)], (2, 16, 64), torch.float32)
    for bad in (gpu(2, 15, 64), gpu(2, 16, 64, dtype=torch.bfloat16), gpu(2, 64, 16).transpose(1, 2)):
        assert not B._alike([gpu(2, 16, 64), bad], (2, 16, 64), torch.float32)
    assert not B._alike([torch.zeros(2, 16, 64)], (2, 16, 64), torch.float32)


def test_buffers_of_another_gpu_are_refused(monkeypatch):
    class Gpu(torch.Tensor):
        def get_device(self):
            return 1

    t = torch.zeros(16).as_subclass(Gpu)
    monkeypatch.setattr(B, "_current_gpu", lambda: 0)
    with pytest.raises(ValueError, match="on GPU 1, the current one is 0"):
        B._need("call", q=(t, torch.float32, 16))
    monkeypatch.setattr(B, "_current_gpu", lambda: 1)
    B._need("call", q=(t, torch.float32, 16), gate=(None, torch.float32, 16))


def test_layers_and_rows_of_another_gpu_are_refused(monkeypatch):
    p = prompt(2)
    for layer in layers(2):
        layer.sound, layer.gpu = True, 1
        for here in (0, 1):  # (the rows are host memory)
            monkeypatch.setattr(B, "_current_gpu", lambda: here)
            with pytest.raises(ValueError, match="the layer is on GPU 1"):
                B._need_layer("call", layer, p)
