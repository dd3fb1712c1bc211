"""Plain oracle for the prompt calls: packed rows of several sequences through
the attention front end, causal attention over the cache, the Gated DeltaNet
front end and the gated delta rule.

TEST INFRASTRUCTURE ONLY (as oracle/tree_verify.py): fp64, shares no code with
the CUDA path.  Written with torch so that long prompts run on the device the
inputs are on; every function takes one sequence.

Source (page title, section): "How ignis serves a request", "The shape of the
process" (one call per prefill span); the mixers' formulas are those of
oracle/tree_verify.py, attn_front.py and gdn_front.py with a chain in the place
of a tree.  Pinned against them in tests/test_prompt_cpu.py.
"""
from __future__ import annotations

import math

import torch


def norm_rope(x, w, pos, eps, rot, theta):
    """x [n, H, D] at positions pos [n] -> normalised (w not None) and rotated, fp64."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w.double()
    if rot == 0:
        return x
    h = rot // 2
    f = torch.tensor([theta ** (-2.0 * j / rot) for j in range(h)], dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None, None] * f
    a, b = x[..., :h], x[..., h:rot]
    return torch.cat([a * torch.cos(ang) - b * torch.sin(ang), b * torch.cos(ang) + a * torch.sin(ang), x[..., rot:]], -1)


def attn_prompt(K, V, L, q, scale, gate=None):
    """Rows q [n, Hq, D] behind L cache rows, K, V [Hkv, >= L + n, D] holding
    the prompt's rows: (out [n, Hq, D], reach [n, Hq, D]) in fp64, where reach
    is the same average of |V| (what rounded probabilities act on)."""
    n, Hq, D = q.shape
    G = Hq // K.shape[0]
    out = torch.empty(n, Hq, D, dtype=torch.float64, device=q.device)
    reach = torch.empty_like(out)
    seen = torch.arange(L + n, device=q.device)[None, :] <= torch.arange(n, device=q.device)[:, None] + L
    for h in range(Hq):
        k, v = K[h // G, :L + n].double(), V[h // G, :L + n].double()
        s = (q[:, h].double() @ k.T) * scale
        p = torch.softmax(torch.where(seen, s, torch.full_like(s, -math.inf)), -1)
        out[:, h] = p @ v
        reach[:, h] = p @ v.abs()
    if gate is not None:
        f = torch.sigmoid(gate.double())
        out, reach = out * f, reach * f
    return out, reach


def gdn_prompt(S, q, k, v, alpha, beta, scale):
    """The recurrence row by row from S [Hv, dv, dk]: (out [n, Hv, dv], the state after the last row)."""
    r = v.shape[1] // k.shape[1]
    S = S.double().clone()
    out = torch.empty(v.shape, dtype=torch.float64, device=v.device)
    for t in range(v.shape[0]):
        kt, qt = (x[t].double().repeat_interleave(r, 0)[:, None, :] for x in (k, q))
        S = S * alpha[t].double()[:, None, None]
        c = beta[t].double()[:, None] * (v[t].double() - (S * kt).sum(-1))
        S = S + c[..., None] * kt
        out[t] = scale * (S * qt).sum(-1)
    return out, S


def gdn_prompt_front(x, tail, wconv, a_raw, b_raw, Hk, dk, Hv, dv):
    """Raw rows x [n, C] behind tail [W-1, C]: q, k, v, alpha, beta in fp64 and the new tail."""
    n, W1 = x.shape[0], tail.shape[0]
    z = torch.cat([tail, x]).double()
    u = sum(z[j:j + n] * wconv[:, j].double() for j in range(W1 + 1))
    u = u / (1 + torch.exp(-u))
    q, k, v = u.split([Hk * dk, Hk * dk, Hv * dv], -1)
    q, k = (t.reshape(n, Hk, dk) for t in (q, k))
    q, k = (t / torch.sqrt(t.pow(2).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    a = a_raw.double()
    alpha = torch.exp(-torch.logaddexp(a, torch.zeros_like(a)))
    return q, k, v.reshape(n, Hv, dv), alpha, torch.sigmoid(b_raw.double()), torch.cat([tail, x])[n:]
