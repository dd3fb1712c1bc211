"""Prompts brought into a verify round's caches and states, through the C ABI.

A VerifyRound starts from resident contexts.  PromptPass fills them: it feeds
the raw projections of a span of prompt rows (whole prompts, or slices of
them, of the round's sequences) through every mixer of the round's layers,

  attention: tv_attn_prompt_front, tv_attn_prompt
  GDN:       tv_gdn_prompt_front, tv_gdn_prompt, tv_gdn_out_norm

and then advances the round's lengths, so that the next verify round or decode
step goes on behind the span.  A span that does not fit (malformed rows, a length
above the round's bound, rows past a cache's end) is refused before its first
layer: status() names the reason, and caches, states, tails and lengths stay.  ("How ignis serves a request", "The shape of
the process": one call per prefill span; "One request, end to end", 2.5.)

The pass owns what lies between the calls of one layer (rotated queries,
convolved rows, gates, one workspace for the longest need); layers run one
after another on one stream and share it.  Two passes that may run at the same
time each need their own.
"""
from __future__ import annotations

import torch

from . import binding as B
from .round import VerifyRound


class PromptPass:
    """Spans of up to n_total rows, n_max a sequence, into a round's layers.

    conv: the GDN layers' (wconv [C][W] fp32, [a tail [W-1][C] per sequence]);
    norms: the attention layers' (q_norm, k_norm) head weights [D] fp32, None
    for none; both by layer index."""

    def __init__(self, r: VerifyRound, n_total: int, n_max: int, conv: dict, norms: dict | None = None,
                 rot_dims: int = 0, theta: float = 10000.0, eps: float = 1e-6):
        self.r, self.rot_dims, self.theta, self.eps = r, rot_dims, theta, eps
        s, dev, dt = r.cfg.shapes, r.device, r.cfg.shapes.kv_dtype
        self.norms = norms or {}
        self.prompt = B.Prompt([0] * r.cfg.n_seq, device=dev, n_total=n_total, n_max=n_max)
        self.fronts = {li: B.GdnFrontLayer(s.Hk, s.Hv, s.dk, s.dv, conv[li][0], conv[li][1], dt) for li in r.gdn}
        ws = 0
        if r.attn:
            self.q_attn = torch.empty((n_total, s.Hq, s.D), dtype=dt, device=dev)
            layer = next(iter(r.attn.values()))["layer"]
            ws = max(ws, B.tv_attn_prompt_workspace_bytes(layer, self.prompt, r.max_len))
        if r.gdn:
            self.q, self.k = (torch.empty((n_total, s.Hk, s.dk), dtype=dt, device=dev) for _ in range(2))
            self.v, self.o = (torch.empty((n_total, s.Hv, s.dv), dtype=dt, device=dev) for _ in range(2))
            self.alpha, self.beta = (torch.empty((n_total, s.Hv), device=dev) for _ in range(2))
            layer = next(iter(r.gdn.values()))["layer"]
            ws = max(ws, B.tv_gdn_prompt_workspace_bytes(layer, self.prompt))
        self.ws = torch.empty(ws, dtype=torch.uint8, device=dev) if ws else None

    def set_rows(self, rows, stream=None):
        """The next span's rows per sequence (0: none), written to the device.
        With the stream that run() gets, behind what that holds, so spans can
        be fed one behind the other without waiting; without, on the current
        stream, which is waited for (no earlier span may run on another)."""
        self.prompt.set_rows(rows, stream)

    def check(self, stream=None):
        """Refuses a span that does not fit; before its first layer.  (Without
        attention layers only its offsets can be wrong.)"""
        most = (1 << 31) - 1
        B.tv_prompt_check(self.prompt, self.r.len, *((self.r.max_len, self.r.cap) if self.r.attn else (most, most)),
                          stream)

    def layer(self, li, x: dict, stream=None):
        """One layer over the span.  Attention: x holds q, k, v, out and, for
        a gated layer, gate; GDN: x, a, b, z, w_norm, out; each with n_total
        rows (rows behind the span's last are not read; a GDN layer's gated
        norm writes whatever they give)."""
        r = self.r
        if li in r.attn:
            layer = r.attn[li]["layer"]
            qn, kn = self.norms.get(li, (None, None))
            B.tv_attn_prompt_front(layer, self.prompt, r.len, r.max_len, qn, kn, self.eps, self.rot_dims, self.theta,
                                   x["q"], x["k"], x["v"], self.q_attn, stream)
            B.tv_attn_prompt(layer, self.prompt, r.len, r.max_len, self.q_attn, x.get("gate"), x["out"], r.attn_scale,
                             self.ws, stream)
        else:
            f = self.fronts[li]
            B.tv_gdn_prompt_front(f, self.prompt, x["x"], x["a"], x["b"], self.q, self.k, self.v, self.alpha,
                                  self.beta, stream)
            B.tv_gdn_prompt(r.gdn[li]["layer"], self.prompt, self.q, self.k, self.v, self.alpha, self.beta, self.o,
                            r.gdn_scale, self.ws, stream)
            B.tv_gdn_out_norm(f, self.prompt.n_total, self.o, x["z"], x["w_norm"], x["out"], stream)

    def advance(self, stream=None):
        """The round's lengths past the span, unless it was refused; after its last layer."""
        B.tv_prompt_advance(self.prompt, self.r.len, stream)

    def run(self, inputs: dict, stream=None):
        """One span through every layer (inputs by layer index, as layer()
        takes them), then the lengths.  With a KV pool the rows that the span
        writes are committed first (VerifyRound.commit_kv).  After a refused
        span nothing runs until its status is cleared (prompt.status.zero_());
        the layers' outputs then hold nothing of use."""
        self.check(stream)
        for li in self.r.layers:
            self.layer(li, inputs[li], stream)
        self.advance(stream)

    def status(self) -> int:
        return self.prompt.status_code()
