"""What the prompt operators are measured on: attention over a prompt's rows
and the cache before them, the query/key head norms with the rotation, the
Gated DeltaNet front end and the gated delta rule over whole prompts.

A prompt here is a packed batch: sequence s owns `rows[s]` new rows behind
`ctx[s]` rows that its caches and states already hold.  `run` computes one
operator either in its plain form (elementary torch operations in 32 bits) or,
where `own` is true, through the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
THETA = 1e7
EPS = 1e-6
CHUNK = 64  # rows of one block of the plain delta rule


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attn(name, rows, ctx, Hq=24, Hkv=4, D=256, dtype="bf16", gate=False):
    return {"name": name, "op": "attn", "rows": rows, "ctx": ctx, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype,
            "gate": gate}


def _qk(name, mode, rows, ctx, Hq=24, Hkv=4, D=256, rot=64, dtype="bf16"):
    return {"name": name, "op": "qk_front", "mode": mode, "rows": rows, "ctx": ctx, "Hq": Hq, "Hkv": Hkv, "D": D,
            "rot": rot, "dtype": dtype}


def _gdn(name, op, rows, Hk=16, Hv=48, d=128, dtype="bf16", width=4):
    return {"name": name, "op": op, "rows": rows, "Hk": Hk, "Hv": Hv, "d": d, "dtype": dtype, "width": width}


def listed():
    return [
        # four sequences decoding one token each at far positions: latency alone
        _qk("qk front, 4 decode tokens", "decode", "1,1,1,1", "65536,8192,8191,131071"),
        # one prompt of ordinary length into an empty cache
        _qk("qk front, 8192 rows", "prompt", "8192", "0"),
        # the small fp32 model of the tests: two short prompts in one call
        _attn("attn fp32, 256 + 37 rows", "256,37", "0,219", Hq=2, Hkv=1, D=64, dtype="fp32"),
        # a server's mixed batch: long, odd and one-row prompts, some behind a context, gated output
        _attn("attn packed, 6659 rows", "2047,1,515,4096", "0,4095,1023,300", gate=True),
        # a whole prompt at once
        _attn("attn, 8192 rows", "8192", "0"),
        # one slice of a very long prompt that is fed slice by slice
        _attn("attn, 1024 rows at 130048", "1024", "130048", gate=True),
        # a short follow-up turn behind a long context: few rows, a long axis
        _attn("attn, 24 rows at 65536", "24", "65536"),
        # a mixed batch's raw projections
        _gdn("gdn front packed, 731 rows", "gdn_front", "515,1,17,198"),
        # a whole prompt's raw projections
        _gdn("gdn front, 8192 rows", "gdn_front", "8192"),
        # the small fp32 model of the tests
        _gdn("gdn fp32, 256 + 37 rows", "gdn", "256,37", Hk=2, Hv=2, d=64, dtype="fp32"),
        # the server's mixed batch through one recurrent layer
        _gdn("gdn packed, 6659 rows", "gdn", "2047,1,515,4096"),
        # a whole prompt through one recurrent layer
        _gdn("gdn, 8192 rows", "gdn", "8192"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split_rows(rng, total, n_seq):
    """`total` rows dealt to n_seq sequences of at least one row each."""
    cuts = sorted(rng.sample(range(1, total), n_seq - 1)) if n_seq > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def draw(rng):
    op = rng.choice(["qk_front", "attn", "attn", "gdn_front", "gdn", "gdn"])
    fp32 = rng.random() < 0.2
    total = _log_int(rng, 1, 512 if fp32 else 8192)
    rows = _split_rows(rng, total, min(total, rng.choice([1, 1, 2, 4, 8])))
    text = ",".join(map(str, rows))
    if op in ("gdn_front", "gdn"):
        Hk, Hv, d = rng.choice([(2, 2, 64), (4, 8, 128)]) if fp32 else rng.choice([(16, 48, 128), (16, 32, 128), (4, 8, 64)])
        c = _gdn("", op, text, Hk, Hv, d, "fp32" if fp32 else "bf16", rng.choice([2, 4, 4, 5]))
    else:
        Hq, Hkv, D = rng.choice([(2, 1, 64), (8, 2, 128)]) if fp32 else rng.choice(
            [(24, 4, 256), (24, 4, 256), (16, 2, 128), (8, 8, 64), (32, 4, 128)])
        far = _log_int(rng, 1, 512 if fp32 else 131072) - 1
        if op == "attn":  # no dearer than the largest listed case
            far = max(0, min(far, int(3.0e12 / (4 * Hq * D * total)) - total))
        ctx = ",".join(str(rng.randint(0, far)) if i else str(far) for i in range(len(rows)))
        if op == "attn":
            c = _attn("", text, ctx, Hq, Hkv, D, "fp32" if fp32 else "bf16", rng.random() < 0.5)
        else:
            mode = "prompt"
            if total <= 8:
                mode, text = "decode", ",".join("1" * total)
                ctx = ",".join(str(rng.randint(0, far)) for _ in range(total))
            c = _qk("", mode, text, ctx, Hq, Hkv, D, rng.choice([D, D // 2, D // 4]), "fp32" if fp32 else "bf16")
    del c["name"]
    return c


def _ints(text):
    return [int(x) for x in text.split(",")]


def _dt(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = _dt(case)

    def rand(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)

    rows = _ints(case["rows"])
    n = sum(rows)
    s = {"case": case, "rows": rows, "n": n, "dt": dt}
    if case["op"] in ("attn", "qk_front"):
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        s["ctx"] = _ints(case["ctx"])
        cap = max(L + m for L, m in zip(s["ctx"], rows)) + 64
        s["len"] = torch.tensor(s["ctx"], dtype=torch.int32, device=DEV)
        if case["op"] == "qk_front":
            # projections as they come: rows of unequal size
            s["q_raw"] = rand(n, Hq, D) * 3
            s["k_raw"] = rand(n, Hkv, D) * 0.5
            s["v"] = rand(n, Hkv, D)
            s["q"] = torch.zeros(n, Hq, D, dtype=dt, device=DEV)
            s["k"] = torch.zeros(n, Hkv, D, dtype=dt, device=DEV)
            s["q_norm"] = 1 + 0.1 * rand(D, dtype=torch.float32)
            s["k_norm"] = 1 + 0.1 * rand(D, dtype=torch.float32)
            s["K"] = [torch.zeros(Hkv, cap, D, dtype=dt, device=DEV) for _ in rows]
            s["V"] = [torch.zeros(Hkv, cap, D, dtype=dt, device=DEV) for _ in rows]
        else:
            # the caches already hold the prompt's own rows, as the front end leaves them
            s["K"] = [rand(Hkv, cap, D) for _ in rows]
            s["V"] = [rand(Hkv, cap, D) for _ in rows]
            s["q"] = rand(n, Hq, D)
            s["gate"] = rand(n, Hq, D) if case["gate"] else None
            s["out"] = torch.empty(n, Hq, D, dtype=dt, device=DEV)
            s["scale"] = D ** -0.5
        return s
    Hk, Hv, d, W = case["Hk"], case["Hv"], case["d"], case["width"]
    # decay rates spread over the heads, from near none to strong
    a_raw = rand(n, Hv, dtype=torch.float32) + torch.linspace(-6, 0, Hv, device=DEV)
    b_raw = rand(n, Hv, dtype=torch.float32)
    s["q"], s["k"] = (torch.empty(n, Hk, d, dtype=dt, device=DEV) for _ in range(2))
    s["v"] = torch.empty(n, Hv, d, dtype=dt, device=DEV)
    if case["op"] == "gdn_front":
        C = 2 * Hk * d + Hv * d
        s["a_raw"], s["b_raw"] = a_raw, b_raw
        s["x"] = rand(n, C)
        s["wconv"] = rand(C, W, dtype=torch.float32) * W ** -0.5
        s["tail"] = [rand(W - 1, C) for _ in rows]
        s["alpha"], s["beta"] = torch.empty_like(a_raw), torch.empty_like(b_raw)
    else:
        for x in ("q", "k"):
            s[x] = torch.nn.functional.normalize(rand(n, Hk, d, dtype=torch.float32), dim=-1).to(dt)
        s["v"] = rand(n, Hv, d)
        s["alpha"] = torch.exp(-torch.nn.functional.softplus(a_raw))
        s["beta"] = torch.sigmoid(b_raw)
        s["S"] = [rand(Hv, d, d, dtype=torch.float32) * 0.1 for _ in rows]
        s["out"] = torch.empty(n, Hv, d, dtype=dt, device=DEV)
        s["scale"] = d ** -0.5
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _handles(s)
    return s


def _handles(s):
    """The descriptors and the workspace that a user's program keeps beside a model."""
    from speculative_tree_verify_masked_gb300 import binding as B

    c = s["case"]
    s["B"] = B
    s["prompt"] = B.Prompt(s["rows"], device=DEV)
    if c["op"] in ("attn", "qk_front"):
        s["layer"] = B.AttnLayer(s["K"], s["V"], c["Hq"])
        s["max_len"] = max(s["ctx"])
        s["status"] = torch.zeros(4, dtype=torch.int32, device=DEV)
        if c["op"] == "attn":
            need = B.tv_attn_prompt_workspace_bytes(s["layer"], s["prompt"], s["max_len"])
            s["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
    elif c["op"] == "gdn":
        s["layer"] = B.GdnLayer(s["S"], c["Hk"], s["dt"])
        need = B.tv_gdn_prompt_workspace_bytes(s["layer"], s["prompt"])
        s["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
    else:
        s["layer"] = B.GdnFrontLayer(c["Hk"], c["Hv"], c["d"], c["d"], s["wconv"], s["tail"], s["dt"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    c, B = s["case"], s["B"]
    if c["op"] == "attn":
        B.tv_attn_prompt(s["layer"], s["prompt"], s["len"], s["max_len"], s["q"], s["gate"], s["out"], s["scale"],
                         s["ws"])
        return s["out"]
    if c["op"] == "qk_front":
        if c["mode"] == "decode":
            B.tv_attn_norm_rope(s["layer"], None, len(s["rows"]), s["len"], s["max_len"], s["q_norm"], s["k_norm"],
                                EPS, c["rot"], THETA, s["q_raw"], s["k_raw"], s["q"], s["k"], s["status"])
            return {"q": s["q"], "k": s["k"]}
        B.tv_attn_prompt_front(s["layer"], s["prompt"], s["len"], s["max_len"], s["q_norm"], s["k_norm"], EPS,
                               c["rot"], THETA, s["q_raw"], s["k_raw"], s["v"], s["q"])
        return {"q": s["q"], "K": s["K"], "V": s["V"]}
    if c["op"] == "gdn_front":
        B.tv_gdn_prompt_front(s["layer"], s["prompt"], s["x"], s["a_raw"], s["b_raw"], s["q"], s["k"], s["v"],
                              s["alpha"], s["beta"])
        return {x: s[x] for x in ("q", "k", "v", "alpha", "beta", "tail")}
    B.tv_gdn_prompt(s["layer"], s["prompt"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["out"], s["scale"],
                    s["ws"])
    return {"out": s["out"], "S": s["S"]}


def _run_plain(s):
    return {"attn": _plain_attn, "qk_front": _plain_qk_front, "gdn_front": _plain_gdn_front, "gdn": _plain_gdn}[
        s["case"]["op"]](s)


def _plain_attn(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    off = 0
    for K, V, L, n in zip(s["K"], s["V"], s["ctx"], s["rows"]):
        q = s["q"][off:off + n].float().view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
        p = torch.matmul(q, K[:, :L + n].float().transpose(1, 2)).mul_(s["scale"]).view(Hkv, G, n, L + n)
        row = torch.arange(n, device=DEV)[:, None] + L
        p.masked_fill_(torch.arange(L + n, device=DEV)[None, :] > row, -math.inf)
        p = p.sub_(p.amax(-1, keepdim=True)).exp_()
        z = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(Hkv, G * n, L + n), V[:, :L + n].float()).view(Hkv, G, n, D) / z
        o = o.permute(2, 0, 1, 3).reshape(n, Hq, D)
        if c["gate"]:
            o = o / (1 + torch.exp(-s["gate"][off:off + n].float()))
        s["out"][off:off + n] = o.to(s["dt"])
        off += n
    return s["out"]


def _norm_rope(x, w, pos, rot):
    """x [n, H, D] in 32 bits: each head over its RMS, times w, its first `rot` dimensions turned."""
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    h = rot // 2
    ang = pos.double()[:, None] * THETA ** (-2.0 * torch.arange(h, device=DEV, dtype=torch.float64) / rot)
    cs, sn = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    a, b = x[..., :h], x[..., h:rot]
    return torch.cat([a * cs - b * sn, b * cs + a * sn, x[..., rot:]], -1)


def _plain_qk_front(s):
    c, dt = s["case"], s["dt"]
    pos = torch.cat([torch.arange(n, device=DEV) + L for L, n in zip(s["ctx"], s["rows"])])
    s["q"].copy_(_norm_rope(s["q_raw"].float(), s["q_norm"], pos, c["rot"]).to(dt))
    k = _norm_rope(s["k_raw"].float(), s["k_norm"], pos, c["rot"]).to(dt)
    if c["mode"] == "decode":
        s["k"].copy_(k)
        return {"q": s["q"], "k": s["k"]}
    off = 0
    for K, V, L, n in zip(s["K"], s["V"], s["ctx"], s["rows"]):
        K[:, L:L + n] = k[off:off + n].transpose(0, 1)
        V[:, L:L + n] = s["v"][off:off + n].transpose(0, 1)
        off += n
    return {"q": s["q"], "K": s["K"], "V": s["V"]}


def _plain_gdn_front(s):
    c, dt = s["case"], s["dt"]
    Hk, Hv, d, W = c["Hk"], c["Hv"], c["d"], c["width"]
    off = 0
    for tail, n in zip(s["tail"], s["rows"]):
        z = torch.cat([tail, s["x"][off:off + n]])
        zf = z.float()
        u = sum(zf[j:j + n] * s["wconv"][:, j] for j in range(W))
        u = u / (1 + torch.exp(-u))
        qk = u[:, :2 * Hk * d].view(n, 2, Hk, d)
        qk = (qk / torch.sqrt((qk * qk).sum(-1, keepdim=True) + EPS)).to(dt)
        s["q"][off:off + n] = qk[:, 0]
        s["k"][off:off + n] = qk[:, 1]
        s["v"][off:off + n] = u[:, 2 * Hk * d:].view(n, Hv, d).to(dt)
        tail.copy_(z[n:])
        off += n
    a = s["a_raw"]
    s["alpha"].copy_(torch.exp(-(torch.clamp(a, min=0) + torch.log1p(torch.exp(-a.abs())))))
    s["beta"].copy_(1 / (1 + torch.exp(-s["b_raw"])))
    return {x: s[x] for x in ("q", "k", "v", "alpha", "beta", "tail")}


def _plain_gdn(s):
    """The gated delta rule block by block: within a block of CHUNK rows the
    corrections solve a unit triangular system, between blocks the state passes."""
    c = s["case"]
    Hk, Hv, d = c["Hk"], c["Hv"], c["d"]
    N, nb = len(s["rows"]), -(-max(s["rows"]) // CHUNK)

    def blocks(x, fill=0.0):  # [n, H, ...] -> [N, H, nb, CHUNK, ...], short sequences filled up
        z = x.new_full((N, nb * CHUNK) + tuple(x.shape[1:]), fill, dtype=torch.float32)
        for i, part in enumerate(x.split(s["rows"])):
            z[i, :part.shape[0]] = part
        return z.transpose(1, 2).reshape((N, x.shape[1], nb, CHUNK) + tuple(x.shape[2:]))

    q, k = (blocks(s[x]).repeat_interleave(Hv // Hk, 1) for x in ("q", "k"))
    v, beta = blocks(s["v"]), blocks(s["beta"])
    # decays from 64-bit sums of logarithms: their differences reach far below the sums
    g = torch.log(blocks(s["alpha"], 1.0).double()).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    decay = torch.exp((g[..., :, None] - g[..., None, :]).masked_fill_(~low, -math.inf).float())
    head, last = torch.exp(g.float()), torch.exp((g[..., -1:] - g).float())
    A = (torch.matmul(k, k.transpose(-1, -2)) * decay * beta[..., None]).tril(-1)
    P = torch.matmul(q, k.transpose(-1, -2)) * decay
    # (I + A)^-1 = (I - A)(I + A^2)(I + A^4) ...: A is strictly lower triangular
    X, B2 = torch.eye(CHUNK, device=DEV) - A, torch.matmul(A, A)
    for _ in range(5):
        X, B2 = X + torch.matmul(X, B2), torch.matmul(B2, B2)
    X = X * beta[..., None, :]
    S = torch.stack(s["S"])
    out = torch.empty(N, Hv, nb, CHUNK, d, device=DEV)
    for b in range(nb):
        kb, qb, hb = k[:, :, b], q[:, :, b], head[:, :, b, :, None]
        St = S.transpose(-1, -2)
        u = torch.matmul(X[:, :, b], v[:, :, b] - hb * torch.matmul(kb, St))
        out[:, :, b] = hb * torch.matmul(qb, St) + torch.matmul(P[:, :, b], u)
        S = S * head[:, :, b, -1, None, None] + torch.matmul((u * last[:, :, b, :, None]).transpose(-1, -2), kb)
    out = (out * s["scale"]).reshape(N, Hv, nb * CHUNK, d).transpose(1, 2)
    off = 0
    for i, n in enumerate(s["rows"]):
        s["S"][i].copy_(S[i])
        s["out"][off:off + n] = out[i, :n].to(s["dt"])
        off += n
    return {"out": s["out"], "S": s["S"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    rows = _ints(case["rows"])
    n, es = sum(rows), 4 if case["dtype"] == "fp32" else 2
    if case["op"] in ("attn", "qk_front"):
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        ctx = _ints(case["ctx"])
        if case["op"] == "qk_front":
            heads = 2 * (Hq + Hkv) + (2 * Hkv if case["mode"] == "prompt" else 0)
            return {"bytes": n * heads * D * es + 8 * D, "flops": n * (Hq + Hkv) * D * 6}
        kv = sum(L + m for L, m in zip(ctx, rows)) * 2 * Hkv * D * es
        pairs = sum(m * L + m * (m + 1) // 2 for L, m in zip(ctx, rows))
        return {"bytes": n * Hq * D * es * (3 if case["gate"] else 2) + kv, "flops": 4 * Hq * D * pairs}
    Hk, Hv, d, W = case["Hk"], case["Hv"], case["d"], case["width"]
    C = 2 * Hk * d + Hv * d
    if case["op"] == "gdn_front":
        return {"bytes": n * (2 * C * es + 16 * Hv) + 4 * C * W + 2 * len(rows) * (W - 1) * C * es,
                "flops": n * C * (2 * W + 6)}
    return {"bytes": n * ((2 * Hk * d + 2 * Hv * d) * es + 8 * Hv) + len(rows) * 8 * Hv * d * d,
            "flops": n * Hv * 6 * d * d}


def exact(case, seed):
    s = _inputs(case, seed)
    return {"attn": _exact_attn, "qk_front": _exact_qk_front, "gdn_front": _exact_gdn_front, "gdn": _exact_gdn}[
        case["op"]](s)


def _exact_attn(s):
    c = s["case"]
    Hq, G, D = c["Hq"], c["Hq"] // c["Hkv"], c["D"]
    out = torch.empty(s["n"], Hq, D, dtype=torch.float64, device=DEV)
    off = 0
    for K, V, L, n in zip(s["K"], s["V"], s["ctx"], s["rows"]):
        for h in range(Hq):
            key, val = K[h // G, :L + n].double(), V[h // G, :L + n].double()
            for r0 in range(0, n, 2048):
                r1 = min(n, r0 + 2048)
                end = L + r1  # no row of this block sees further
                w = s["q"][off + r0:off + r1, h].double() @ key[:end].T * s["scale"]
                seen = torch.arange(end, device=DEV) <= torch.arange(L + r0, L + r1, device=DEV)[:, None]
                w = torch.softmax(torch.where(seen, w, torch.full_like(w, -math.inf)), -1)
                out[off + r0:off + r1, h] = w @ val[:end]
        off += n
    return out * torch.sigmoid(s["gate"].double()) if c["gate"] else out


def _exact_qk_front(s):
    c = s["case"]
    rot = c["rot"]
    pos = torch.tensor([L + i for L, n in zip(s["ctx"], s["rows"]) for i in range(n)], dtype=torch.float64, device=DEV)

    def turned(x, w):
        x = x.double()
        x = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * w.double()
        freq = torch.exp(torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) * (-math.log(THETA) / rot))
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos[:, None] * freq)[:, None]
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
        return torch.cat([z.real, z.imag, x[..., rot:]], -1)

    q, k = turned(s["q_raw"], s["q_norm"]), turned(s["k_raw"], s["k_norm"])
    if c["mode"] == "decode":
        return {"q": q, "k": k}
    K, V = [x.double() for x in s["K"]], [x.double() for x in s["V"]]
    off = 0
    for i, (L, n) in enumerate(zip(s["ctx"], s["rows"])):
        K[i][:, L:L + n] = k[off:off + n].permute(1, 0, 2)
        V[i][:, L:L + n] = s["v"][off:off + n].double().permute(1, 0, 2)
        off += n
    return {"q": q, "K": K, "V": V}


def _exact_gdn_front(s):
    c = s["case"]
    Hk, Hv, d, W = c["Hk"], c["Hv"], c["d"], c["width"]
    us, tails = [], []
    for tail, x in zip(s["tail"], s["x"].split(s["rows"])):
        z = torch.cat([tail, x]).double()
        us.append(torch.nn.functional.conv1d(z.T[None], s["wconv"].double()[:, None], groups=z.shape[1])[0].T)
        tails.append(z[z.shape[0] - (W - 1):])
    u = torch.nn.functional.silu(torch.cat(us))
    q, k, v = u.split([Hk * d, Hk * d, Hv * d], -1)
    q, k = (x.reshape(-1, Hk, d) for x in (q, k))
    q, k = (x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) + EPS) for x in (q, k))
    return {"q": q, "k": k, "v": v.reshape(-1, Hv, d), "alpha": torch.sigmoid(-s["a_raw"].double()),
            "beta": torch.sigmoid(s["b_raw"].double()), "tail": tails}


def _exact_gdn(s):
    """The recurrence itself, row by row; all sequences step together."""
    c = s["case"]
    r = c["Hv"] // c["Hk"]
    N, n_max = len(s["rows"]), max(s["rows"])

    def padded(x, fill=0.0):
        z = torch.full((n_max, N) + tuple(x.shape[1:]), fill, dtype=torch.float64, device=DEV)
        for i, part in enumerate(x.split(s["rows"])):
            z[:part.shape[0], i] = part.double()
        return z

    q, k, v = padded(s["q"]), padded(s["k"]), padded(s["v"])
    alpha, beta = padded(s["alpha"], 1.0), padded(s["beta"])
    S = torch.stack(s["S"]).double()
    out = torch.empty_like(v)
    for t in range(n_max):  # a finished sequence has alpha 1 and beta 0: its state stays
        kt = k[t].repeat_interleave(r, 1)
        S = S * alpha[t][..., None, None]
        err = beta[t][..., None] * (v[t] - (S * kt[..., None, :]).sum(-1))
        S = S + err[..., None] * kt[..., None, :]
        out[t] = (S * q[t].repeat_interleave(r, 1)[..., None, :]).sum(-1)
    out = torch.cat([out[:n, i] for i, n in enumerate(s["rows"])]) * s["scale"]
    return {"out": out, "S": list(S)}
