"""What the paged-cache operators are measured on: appending rows to a cache
in pages, decode attention over such caches (with prefixes that a group of
sequences shares), the pages' bounds, and attention over the pages that a
score by those bounds selects.

A batch has one row of a page table per sequence and `lens[s]` rows already
held (-1: an idle slot).  `run` computes one operator either in its plain form
(elementary torch operations) or, where `own` is true, through the library.
"""
import math
import random

import torch

own = False

DEV = "cuda"
THETA = 1e7
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, lens, page=64, heads=(24, 4, 256), dtype="bf16", **more):
    Hq, Hkv, D = heads
    return {"name": name, "op": op, "lens": _text(lens), "page": page, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype,
            **more}


def _text(values):
    return ",".join(map(str, values))


def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _spread(seed, n, lo, hi):
    rng = random.Random(seed)
    return [_log_int(rng, lo, hi) for _ in range(n)]


def listed():
    return [
        # a decode step of four sequences: latency alone
        _case("append, 4 decode rows", "append", [4095, 0, 131000, 63], rot=64, rows=""),
        # a decode step of a full server, some slots idle
        _case("append, 192 decode rows", "append", [-1 if i % 17 == 5 else x for i, x in enumerate(_spread(1, 192, 1, 65536))],
              page=32, rot=64, rows=""),
        # slices of four prompts, odd and long, into pages of 16
        _case("append, slices of 4629 rows", "append", [0, 1023, 300, 8192], page=16, rot=64, rows="4096,515,1,17"),
        # the pages that a decode step of many sequences completes: few of them
        _case("bounds, 192 decode rows", "bounds", _spread(2, 192, 1, 65536), page=16, rows=""),
        # the pages of two long prompts
        _case("bounds, 16421 rows", "bounds", [0, 37], rows="8192,8229"),
        # the small fp32 model of the tests
        _case("attn fp32, 5 sequences", "attn", [256, 0, 31, 300, 15], page=16, heads=(2, 1, 64), dtype="fp32",
              groups="", shared="", gate=False),
        # a few short chats with a gated output: latency counts
        _case("attn, 4 short sequences", "attn", [0, 63, 500, 1025], groups="", shared="", gate=True),
        # a server's mixed batch: very different lengths, nothing shared
        _case("attn, 96 ragged sequences", "attn", _spread(3, 96, 16, 32768), page=32, heads=(16, 2, 128), groups="",
              shared="", gate=False),
        # many samples of one long prompt, and a second smaller group
        _case("attn, 64 + 6 on shared prefixes", "attn",
              [32768 + x for x in _spread(4, 64, 1, 1024)] + [8192 + x for x in _spread(5, 6, 1, 2048)],
              groups="64,6", shared="32768,8192", gate=True),
        # the small fp32 model, some sequences shorter than their selection
        _case("sparse fp32, 6 sequences", "sparse", [1023, 100, 7, 511, 640, 255], page=16, heads=(2, 1, 64), dtype="fp32",
              n_sel=16, first=1, last=2),
        # one very long context: 4,096 of 131,071 rows are looked at
        _case("sparse, 1 sequence at 131071", "sparse", [131071], n_sel=64, first=1, last=2),
        # a long-context server's batch
        _case("sparse, 24 sequences to 65536", "sparse", _spread(6, 24, 4096, 65536), n_sel=48, first=1, last=2),
    ]


def draw(rng):
    op = rng.choice(["append", "bounds", "attn", "attn", "sparse", "sparse"])
    fp32 = rng.random() < 0.2
    heads = rng.choice([(2, 1, 64), (8, 2, 128)]) if fp32 else rng.choice(
        [(24, 4, 256), (24, 4, 256), (16, 2, 128), (8, 8, 64), (32, 4, 128)])
    Hq, Hkv, D = heads
    page = rng.choice([16, 32, 64, 64, 128])
    n = _log_int(rng, 1, 8 if fp32 else 192)
    far = _log_int(rng, 16, 1024 if fp32 else 131072)
    lens = [rng.randint(0, far - 1) for _ in range(n)]
    dtype = "fp32" if fp32 else "bf16"
    if op in ("append", "bounds"):
        rows = ""
        if rng.random() < 0.5:  # slices of prompts
            n = min(n, 8)
            lens, total = lens[:n], _log_int(rng, n, 512 if fp32 else 8192)
            cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
            rows = _text([b - a for a, b in zip([0] + cuts, cuts + [total])])
        elif rng.random() < 0.4:
            lens[rng.randrange(n)] = -1
        if op == "bounds":  # a page that is completed, at least
            i = rng.choice([i for i, L in enumerate(lens) if L >= 0 and (not rows or _ints(rows)[i])] or [0])
            lens[i] = max(lens[i], 0) // page * page + page - 1
        extra = {"rot": rng.choice([D, D // 2, D // 4])} if op == "append" else {}
        c = _case("", op, lens, page, heads, dtype, rows=rows, **extra)
    else:
        groups = shared = ""
        if op == "attn":
            if rng.random() < 0.5 and n > 2:  # groups on prefixes of whole pages
                k = rng.randint(1, min(4, n // 2))
                cuts = sorted(rng.sample(range(1, n), k - 1))
                sizes = [b - a for a, b in zip([0] + cuts, cuts + [n])]
                most = int(4e10 / (4 * Hq * D * n))  # no dearer than the largest listed case
                pre = [min(_log_int(rng, page, max(page, far)), most) // page * page for _ in sizes]
                own_rows = [rng.randint(0, _log_int(rng, 1, 1024)) for _ in lens]
                lens = [p + own_rows[i] for i, p in enumerate(p for p, m in zip(pre, sizes) for _ in range(m))]
                groups, shared = _text(sizes), _text(pre)
            if rng.random() < 0.3:
                lens[rng.randrange(n)] = -1
        cap = int(5e8 / (4 * Hkv * D))  # rows: at most 0.5 GB of 16-bit keys and values
        own_total = sum(lens) - (sum(p * (m - 1) for p, m in zip(_ints(shared), _ints(groups))) if groups else 0)
        if own_total > cap and not groups:
            lens = [x * cap // own_total if x > 0 else x for x in lens]
        if op == "attn":
            c = _case("", "attn", lens, page, heads, dtype, groups=groups, shared=shared, gate=rng.random() < 0.5)
        else:
            n_sel = _log_int(rng, 4, 4096 // page)
            c = _case("", "sparse", lens, page, heads, dtype, n_sel=n_sel, first=rng.randint(0, 1),
                      last=rng.randint(1, 3))
    del c["name"]
    return c


def _dt(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt, op = _dt(case), case["op"]
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]

    def rand(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)

    lens = _ints(case["lens"])
    N = len(lens)
    rows = _ints(case["rows"]) if case.get("rows") else [1 if L >= 0 else 0 for L in lens]
    s = {"case": case, "lens": lens, "rows": rows, "dt": dt, "N": N, "max_len": max(max(lens), 0)}
    # a page table: pages of the pool in a random order, shared ones listed by every member; -1 where there is none
    cols = -(-(s["max_len"] + max(max(rows), 1)) // page)
    table = [[-1] * cols for _ in lens]
    used = 0
    # (appending touches the last pages alone: earlier ones need not be there)
    keep = [max(L, 0) // page if op in ("append", "bounds") else 0 for L in lens]
    shared_pages = [0] * N
    first = 0
    if case.get("groups"):
        for m, p in zip(_ints(case["groups"]), _ints(case["shared"])):
            for i in range(first, first + m):
                shared_pages[i] = p // page
                table[i][:p // page] = range(used, used + p // page)
            used += p // page
            first += m
    for i, (L, n) in enumerate(zip(lens, rows)):
        if L < 0:
            continue
        for j in range(max(keep[i], shared_pages[i]), -(-(L + max(n, 1)) // page)):
            table[i][j] = used
            used += 1
    n_pages = max(used, 1) + 3
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed))
    t = torch.tensor(table, dtype=torch.int32)
    s["table_host"] = torch.where(t >= 0, order[t.clamp(min=0).long()].int(), t)
    s["table"] = s["table_host"].to(DEV)
    s["len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["n_pages"], s["scale"] = n_pages, D ** -0.5
    n = sum(rows) if case.get("rows") else N
    if op == "append":
        # projections as they come: rows of unequal size
        s["q_raw"], s["k_raw"], s["v"] = rand(n, Hq, D) * 3, rand(n, Hkv, D) * 0.5, rand(n, Hkv, D)
        s["q_norm"], s["k_norm"] = (1 + 0.1 * rand(D, dtype=torch.float32) for _ in range(2))
        s["q"] = torch.zeros(n, Hq, D, dtype=dt, device=DEV)
        s["K"], s["V"] = (torch.zeros(n_pages, Hkv, page, D, dtype=dt, device=DEV) for _ in range(2))
        return s
    s["K"] = rand(n_pages, Hkv, page, D)
    if op != "attn":  # pages differ: what a page's keys have in common is about as large as what they have not
        s["K"] += rand(n_pages, Hkv, 1, D)
    if op == "bounds":
        s["code"] = torch.zeros(n_pages, Hkv, 2, D, dtype=torch.int8, device=DEV)
        s["exp"] = torch.zeros(n_pages, Hkv, dtype=torch.int32, device=DEV)
        return s
    s["V"] = rand(n_pages, Hkv, page, D)
    s["q"] = rand(n, Hq, D)
    s["gate"] = rand(n, Hq, D) if case.get("gate") else None
    s["out"] = torch.zeros(n, Hq, D, dtype=dt, device=DEV)
    if op == "sparse":  # the bounds that a program has kept up to the step before
        s["code"], s["exp"] = _bounds(s["K"])
        s["sel"] = torch.zeros(N, Hkv, case["n_sel"], dtype=torch.int32, device=DEV)
        s["count"] = torch.zeros(N, Hkv, dtype=torch.int32, device=DEV)
        for i, L in enumerate(lens):
            j = L // page
            s["code"][int(s["table_host"][i, j])] = 0
            s["exp"][int(s["table_host"][i, j])] = 0
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _handles(s)
    return s


def _handles(s):
    """The descriptors and workspaces that a user's program keeps beside a model."""
    from speculative_tree_verify_masked_gb300 import binding as B

    c = s["case"]
    s["B"] = B
    s["layer"] = B.PagedLayer(s["K"], s["V"] if "V" in s else s["K"], c["Hq"])
    s["batch"] = B.PagedBatch(s["table"], s["len"], s["max_len"])
    s["span"] = B.PagedRows(s["rows"], device=DEV) if c.get("rows") else None

    def space(need):
        return torch.empty(max(16, need), dtype=torch.uint8, device=DEV)

    if c["op"] == "attn":
        s["groups"] = B.PagedGroups(_ints(c["groups"]), _ints(c["shared"]), device=DEV) if c["groups"] else None
        s["ws"] = space(B.tv_paged_attn_workspace_bytes(s["layer"], s["batch"], s["groups"]))
    if c["op"] == "sparse":
        s["ws"] = space(max(B.tv_paged_select_workspace_bytes(s["layer"], s["batch"]),
                            B.tv_paged_attn_selected_workspace_bytes(s["layer"], s["batch"], c["n_sel"])))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    c, B = s["case"], s["B"]
    if c["op"] == "append":
        B.tv_paged_append(s["layer"], s["batch"], s["span"], s["q_norm"], s["k_norm"], EPS, c["rot"], THETA, s["q_raw"],
                          s["k_raw"], s["v"], s["q"])
        return {"q": s["q"], "K": s["K"], "V": s["V"]}
    if c["op"] == "bounds":
        B.tv_paged_bounds(s["layer"], s["batch"], s["span"], s["code"], s["exp"])
        return {"code": s["code"], "exp": s["exp"]}
    if c["op"] == "attn":
        B.tv_paged_attn(s["layer"], s["batch"], s["groups"], s["q"], s["gate"], s["out"], s["scale"], s["ws"])
        return s["out"]
    B.tv_paged_bounds(s["layer"], s["batch"], None, s["code"], s["exp"])
    B.tv_paged_select(s["layer"], s["batch"], s["code"], s["exp"], c["first"], c["last"], s["q"], s["sel"], s["count"],
                      s["ws"])
    B.tv_paged_attn_selected(s["layer"], s["batch"], s["sel"], s["count"], s["q"], None, s["out"], s["scale"], s["ws"])
    return {x: s[x] for x in ("code", "exp", "sel", "count", "out")}


def _run_plain(s):
    return {"append": _plain_append, "bounds": _plain_bounds, "attn": _plain_attn, "sparse": _plain_sparse}[
        s["case"]["op"]](s)


def _places(s):
    """Sequence, position, page and row in it of every row of a span or step."""
    seq, pos = [], []
    for i, (L, n) in enumerate(zip(s["lens"], s["rows"])):
        seq += [i] * n
        pos += range(L, L + n)
    seq, pos = torch.tensor(seq, device=DEV), torch.tensor(pos, device=DEV)
    page = s["case"]["page"]
    return seq, pos, s["table"][seq, pos // page].long(), pos % page


def _norm_rope(x, w, pos, rot):
    """x [n, H, D] in 32 bits: each head over its RMS, times w, its first `rot` dimensions turned."""
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    h = rot // 2
    ang = pos.double()[:, None] * THETA ** (-2.0 * torch.arange(h, device=DEV, dtype=torch.float64) / rot)
    cs, sn = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    a, b = x[..., :h], x[..., h:rot]
    return torch.cat([a * cs - b * sn, b * cs + a * sn, x[..., rot:]], -1)


def _plain_append(s):
    c, dt = s["case"], s["dt"]
    seq, pos, pages, r = _places(s)
    at = torch.arange(len(seq), device=DEV) if c["rows"] else seq  # a step's row is its sequence's
    s["q"][at] = _norm_rope(s["q_raw"][at].float(), s["q_norm"], pos, c["rot"]).to(dt)
    s["K"][pages, :, r] = _norm_rope(s["k_raw"][at].float(), s["k_norm"], pos, c["rot"]).to(dt)
    s["V"][pages, :, r] = s["v"][at]
    return {"q": s["q"], "K": s["K"], "V": s["V"]}


def _pow2(e):
    """2^e in 64 bits, put together from its bits (a power function may be off by a step, and floors and
    ceilings of whole numbers would see it)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _bounds(K):
    """Codes [n, Hkv, 2, D] and exponents [n, Hkv] of whole pages K [n, Hkv, page, D]: the columns' least
    and largest values in steps of 2^e, rounded outward; e the least with every code within 127."""
    lo, hi = K.amin(2).double(), K.amax(2).double()
    m, x = torch.frexp(torch.maximum(lo.abs(), hi.abs()).amax(-1))
    e = (x - 7 + (m > 127 / 128).int()).clamp(min=-100)
    step = _pow2(e)[..., None]
    return torch.stack([torch.floor(lo / step), torch.ceil(hi / step)], 2).to(torch.int8), e.int()


def _completed(s):
    """The pages that a span or step completes."""
    page = s["case"]["page"]
    return [int(s["table_host"][i, j]) for i, (L, n) in enumerate(zip(s["lens"], s["rows"])) if L >= 0
            for j in range(L // page, (L + n) // page)]


def _plain_bounds(s):
    done = torch.tensor(_completed(s), dtype=torch.long, device=DEV)
    if len(done):
        s["code"][done], s["exp"][done] = _bounds(s["K"][done])
    return {"code": s["code"], "exp": s["exp"]}


def _attend(s, i, K, V, q):
    """K, V [Hkv, T, D] and q [Hkv, G, D] in 32 bits."""
    p = torch.matmul(q, K.transpose(1, 2)).mul_(s["scale"])
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    return (torch.matmul(p, V) / p.sum(-1, keepdim=True)).reshape(-1, K.shape[-1])


def _plain_attn(s):
    c = s["case"]
    Hkv, D, page = c["Hkv"], c["D"], c["page"]
    for i, L in enumerate(s["lens"]):
        if L < 0:
            continue
        pages = s["table"][i, :L // page + 1].long()
        K, V = (s[x][pages].float().transpose(0, 1).reshape(Hkv, -1, D)[:, :L + 1] for x in ("K", "V"))
        o = _attend(s, i, K, V, s["q"][i].float().view(Hkv, -1, D))
        if c["gate"]:
            o = o / (1 + torch.exp(-s["gate"][i].float()))
        s["out"][i] = o.to(s["dt"])
    return s["out"]


def _query_codes(q):
    """q [Hkv, G, D] in whole steps of one power of two a KV head, the least with every code within 127."""
    m, x = torch.frexp(q.abs().amax((1, 2)).double())
    e = x - 7 + (m > 127 / 128).int()
    return torch.round(q.double() / _pow2(e)[:, None, None])


def _plain_sparse(s):
    c = s["case"]
    Hkv, D, page, n_sel = c["Hkv"], c["D"], c["page"], c["n_sel"]
    _plain_bounds(s)
    s["sel"].fill_(-1)
    for i, L in enumerate(s["lens"]):
        nb = L // page + 1
        if nb <= n_sel:
            sel = torch.arange(nb, device=DEV).expand(Hkv, nb)
        else:
            a, b = min(c["first"], nb), nb - c["last"]
            pages = s["table"][i, a:b].long()
            u = _query_codes(s["q"][i].view(Hkv, -1, D)).float()
            lo, hi = s["code"][pages].float().permute(2, 1, 3, 0)  # [Hkv, D, pages]
            score = (torch.matmul(u.clamp(min=0), hi) + torch.matmul(u.clamp(max=0), lo)).amax(1)  # whole numbers under 2^24
            score = score.double() * _pow2(s["exp"][pages].T)
            best = torch.sort(score, stable=True, dim=-1, descending=True)[1][:, :n_sel - c["first"] - c["last"]] + a
            ends = torch.cat([torch.arange(a, device=DEV), torch.arange(b, nb, device=DEV)]).expand(Hkv, -1)
            sel = torch.sort(torch.cat([ends, best], 1), -1)[0]
        s["sel"][i, :, :sel.shape[1]] = sel.int()
        s["count"][i] = sel.shape[1]
        pages, heads = s["table"][i][sel].long(), torch.arange(Hkv, device=DEV)[:, None]
        seen = (sel.shape[1] - 1) * page + L % page + 1  # the row's own page is the last one
        K, V = (s[x][pages, heads].float().view(Hkv, -1, D)[:, :seen] for x in ("K", "V"))
        s["out"][i] = _attend(s, i, K, V, s["q"][i].float().view(Hkv, -1, D)).to(s["dt"])
    return {x: s[x] for x in ("code", "exp", "sel", "count", "out")}


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    lens, es = _ints(case["lens"]), 4 if case["dtype"] == "fp32" else 2
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    live = sum(L >= 0 for L in lens)
    rows = _ints(case["rows"]) if case.get("rows") else [int(L >= 0) for L in lens]
    if case["op"] == "append":
        return {"bytes": sum(rows) * 2 * (Hq + 2 * Hkv) * D * es + 8 * D, "flops": sum(rows) * (Hq + Hkv) * D * 6}
    if case["op"] == "bounds":
        done = sum((L + n) // page - L // page for L, n in zip(lens, rows) if L >= 0)
        return {"bytes": done * Hkv * (page * D * es + 2 * D + 4) + 8 * len(lens), "flops": done * Hkv * page * D * 2}
    io = live * Hq * D * es * (3 if case.get("gate") else 2)
    if case["op"] == "attn":
        seen = [L + 1 for L in lens]
        distinct = sum(seen)
        if case["groups"]:
            distinct -= sum(p * (m - 1) for p, m in zip(_ints(case["shared"]), _ints(case["groups"])))
        return {"bytes": io + max(distinct, 0) * 2 * Hkv * D * es, "flops": 4 * Hq * D * sum(seen)}
    nb = [L // page + 1 for L in lens]
    seen = sum(L + 1 if b <= case["n_sel"] else (case["n_sel"] - 1) * page + L % page + 1 for L, b in zip(lens, nb))
    scored = sum(b - case["first"] - case["last"] for b in nb if b > case["n_sel"])
    return {"bytes": io + seen * 2 * Hkv * D * es + scored * Hkv * (2 * D + 4),
            "flops": 4 * Hq * D * seen + 4 * Hq * D * scored}


def exact(case, seed):
    s = _inputs(case, seed)
    return {"append": _exact_append, "bounds": _exact_bounds, "attn": _exact_attn, "sparse": _exact_sparse}[
        case["op"]](s)


def _exact_append(s):
    c = s["case"]
    rot, page = c["rot"], c["page"]

    def turned(x, w, pos):
        x = x.double()
        x = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * w.double()
        freq = torch.exp(torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) * (-math.log(THETA) / rot))
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos[:, None] * freq)[:, None]
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
        return torch.cat([z.real, z.imag, x[..., rot:]], -1)

    q, K, V = s["q"].double(), s["K"].double(), s["V"].double()
    off = 0
    for i, (L, n) in enumerate(zip(s["lens"], s["rows"])):
        at = off if c["rows"] else i
        off += n
        if L < 0 or n == 0:
            continue
        pos = torch.arange(L, L + n, dtype=torch.float64, device=DEV)
        q[at:at + n] = turned(s["q_raw"][at:at + n], s["q_norm"], pos)
        k, v = turned(s["k_raw"][at:at + n], s["k_norm"], pos), s["v"][at:at + n].double()
        for j in range(L // page, (L + n - 1) // page + 1):  # page by page
            a, b = max(j * page, L), min((j + 1) * page, L + n)
            p = int(s["table_host"][i, j])
            K[p, :, a - j * page:b - j * page] = k[a - L:b - L].permute(1, 0, 2)
            V[p, :, a - j * page:b - j * page] = v[a - L:b - L].permute(1, 0, 2)
    return {"q": q, "K": K, "V": V}


def _exact_code(K):
    """Codes and exponent of one page's keys [Hkv, page, D] by trying exponents from the least up."""
    k = K.double()
    e = []
    for top in k.abs().flatten(1).amax(1).tolist():
        e.append(-100)
        while top > 127 * 2.0 ** e[-1]:
            e[-1] += 1
    step = torch.tensor([2.0 ** x for x in e], dtype=torch.float64, device=DEV)[:, None]
    e = torch.tensor(e, dtype=torch.int32, device=DEV)
    return torch.stack([(k.amin(1) / step).floor(), (k.amax(1) / step).ceil()], 1).to(torch.int8), e


def _exact_bounds(s):
    code, exp = s["code"].clone(), s["exp"].clone()
    for p in _completed(s):
        code[p], exp[p] = _exact_code(s["K"][p])
    return {"code": code, "exp": exp}


def _exact_attn(s):
    c = s["case"]
    Hq, G, D, page = c["Hq"], c["Hq"] // c["Hkv"], c["D"], c["page"]
    out = s["out"].double()
    for i, L in enumerate(s["lens"]):
        if L < 0:
            continue
        pages = [int(p) for p in s["table_host"][i, :L // page + 1]]
        for g in range(c["Hkv"]):
            key, val = (s[x][pages, g].reshape(-1, D)[:L + 1].double() for x in ("K", "V"))
            w = torch.softmax(s["q"][i, g * G:(g + 1) * G].double() @ key.T * s["scale"], -1)
            out[i, g * G:(g + 1) * G] = w @ val
    return out * torch.sigmoid(s["gate"].double()) if c["gate"] else out


def _exact_sparse(s):
    c = s["case"]
    Hkv, G, D, page, n_sel = c["Hkv"], c["Hq"] // c["Hkv"], c["D"], c["page"], c["n_sel"]
    res = _exact_bounds(s)
    sel, count, out = torch.full_like(s["sel"], -1), torch.zeros_like(s["count"]), torch.zeros_like(s["out"]).double()
    for i, L in enumerate(s["lens"]):
        nb = L // page + 1
        row = s["table_host"][i]
        for g in range(Hkv):
            q = s["q"][i, g * G:(g + 1) * G].double()
            chosen = list(range(nb))
            if nb > n_sel:
                middle = chosen[c["first"]:nb - c["last"]]
                top, e = q.abs().max(), 0
                while top > 127 * 2.0 ** e:
                    e += 1
                while top <= 127 * 2.0 ** (e - 1) and top > 0:
                    e -= 1
                u = (q / 2.0 ** e).round()
                pages = row[middle].long().to(DEV)
                lo, hi = res["code"][pages, g].double().unbind(1)
                best = torch.where(u[:, None] > 0, u[:, None] * hi, u[:, None] * lo).sum(-1).amax(0)
                best = [x * 2.0 ** n for x, n in zip(best.tolist(), res["exp"][pages, g].tolist())]
                ranked = sorted(range(len(middle)), key=lambda j: (-best[j], j))
                chosen = sorted(chosen[:c["first"]] + chosen[nb - c["last"]:] +
                                [middle[j] for j in ranked[:n_sel - c["first"] - c["last"]]])
            sel[i, g, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
            count[i, g] = len(chosen)
            pages = row[chosen].long().to(DEV)
            pos = (torch.tensor(chosen, device=DEV)[:, None] * page + torch.arange(page, device=DEV)).flatten()
            key, val = (s[x][pages, g].reshape(-1, D).double() for x in ("K", "V"))
            w = (q @ key.T * s["scale"]).masked_fill(pos > L, -math.inf)
            out[i, g * G:(g + 1) * G] = torch.softmax(w, -1) @ val
    return {**res, "sel": sel, "count": count, "out": out}
