"""Attention layers' caches in pages behind one table, for decode steps of many slots.

PagedCaches holds the pools of a model's attention layers, hands out their
pages and keeps the table and the lengths that the calls read.  A page id names
the same page of every layer's pools.  Slots may share their first pages: an
admitted slot can take over a prefix of another one, whose pages then count one
more user.  ("Parallel requests", "The shared KV pool": rows of several
sequences in one pool; "What a slot costs".)

One decode step of one layer is

  tv_paged_append, tv_paged_attn
  or, where only the pages of the highest bounds are looked at,
  tv_paged_append, tv_paged_bounds, tv_paged_select, tv_paged_attn_selected

and after the last layer tv_paged_advance.  Prompts run on contiguous caches
(PromptPass) or come from elsewhere; their raw rows go into the pages by append().

Pages are handed out on the host, between steps: grow() before a step makes
room for its rows, so the step itself only enqueues calls and can be captured.
"""
from __future__ import annotations

import torch

from . import binding as B


class PagedCaches:
    """Pools of n_layers layers, n_pages pages of `page` rows each, for n_slots slots of up to max_len rows.

    sparse: None, or (n_sel, first, last) as tv_paged_select takes them."""

    def __init__(self, n_layers: int, n_pages: int, page: int, Hq: int, Hkv: int, D: int, n_slots: int, max_len: int,
                 dtype=torch.bfloat16, device="cuda", sparse=None, rot_dims: int = 0, theta: float = 10000.0,
                 eps: float = 1e-6, norms=None):
        self.page, self.n_slots, self.max_len, self.sparse = page, n_slots, max_len, sparse
        self.rot_dims, self.theta, self.eps, self.scale = rot_dims, theta, eps, D ** -0.5
        self.norms = norms or [(None, None)] * n_layers
        shape = (n_pages, Hkv, page, D)
        self.K, self.V = ([torch.zeros(shape, dtype=dtype, device=device) for _ in range(n_layers)] for _ in range(2))
        self.table = torch.full((n_slots, max_len // page + 1), -1, dtype=torch.int32, device=device)
        self.len = torch.full((n_slots,), -1, dtype=torch.int32, device=device)
        self.layers = [B.PagedLayer(k, v, Hq) for k, v in zip(self.K, self.V)]
        self.batch = B.PagedBatch(self.table, self.len, max_len)
        self.q = torch.empty((n_slots, Hq, D), dtype=dtype, device=device)
        self.free = list(range(n_pages - 1, -1, -1))
        self.users = [0] * n_pages
        self.pages = [[] for _ in range(n_slots)]  # of each slot, in order
        self.lens = [-1] * n_slots                 # the lengths, as the host knows them
        self.ws, self.outgrown = None, []
        if sparse:
            n_sel = sparse[0]
            self.code = [torch.zeros((n_pages, Hkv, 2, D), dtype=torch.int8, device=device) for _ in range(n_layers)]
            self.exp = [torch.zeros((n_pages, Hkv), dtype=torch.int32, device=device) for _ in range(n_layers)]
            self.sel = torch.empty((n_slots, Hkv, n_sel), dtype=torch.int32, device=device)
            self.count = torch.empty((n_slots, Hkv), dtype=torch.int32, device=device)
            self._space(max(B.tv_paged_select_workspace_bytes(self.layers[0], self.batch),
                            B.tv_paged_attn_selected_workspace_bytes(self.layers[0], self.batch, n_sel)))
        else:
            self._space(B.tv_paged_attn_workspace_bytes(self.layers[0], self.batch))

    def _space(self, need: int):
        if self.ws is None or self.ws.numel() < need:
            if self.ws is not None:
                self.outgrown.append(self.ws)  # (steps that are captured already go on in it)
            self.ws = torch.empty(max(16, need), dtype=torch.uint8, device=self.table.device)

    def groups(self, sizes, shared) -> B.PagedGroups:
        """Groups for decode(); the workspace then holds what they need (make them before the capture of steps that take them)."""
        g = B.PagedGroups(sizes, shared, device=self.table.device)
        self._space(B.tv_paged_attn_workspace_bytes(self.layers[0], self.batch, g))
        return g

    # ---- slots and pages (host calls between steps; device writes in the order of `stream`)
    def admit(self, slot: int, like: int | None = None, rows: int = 0, stream=None):
        """Makes an idle slot active: empty, or with the first `rows` rows of slot `like` (whole pages, shared)."""
        self._one(slot)
        if like is not None:
            self._one(like)
        if self.lens[slot] >= 0:
            raise ValueError(f"slot {slot} is in use")
        if rows < 0 or rows % self.page or (like is None and rows) or (like is not None and rows > self.lens[like]):
            raise ValueError(f"{rows} rows of slot {like} are not whole pages that it holds")
        B._need_no_capture(self.table, stream)
        self.pages[slot] = list(self.pages[like][:rows // self.page]) if rows else []
        for p in self.pages[slot]:
            self.users[p] += 1
        self.lens[slot] = rows
        self._write(slot, stream)

    def retire(self, slot: int, stream=None):
        """Makes a slot idle and gives back the pages that no other one shares."""
        self._one(slot)
        B._need_no_capture(self.table, stream)
        for p in self.pages[slot]:
            self.users[p] -= 1
            if self.users[p] == 0:
                self.free.append(p)
        self.pages[slot], self.lens[slot] = [], -1
        self._write(slot, stream)

    def grow(self, rows=None, stream=None):
        """Pages for the next rows of each slot (None: one for each active one), before they are appended."""
        rows = self._rows(rows)
        if len(rows) != self.n_slots or any(n < 0 or (n and L < 0) for L, n in zip(self.lens, rows)):
            raise ValueError(f"rows {rows} are not of {self.n_slots} slots, or of idle ones")
        need = [max(0, -(-(L + n) // self.page) - len(p)) if n else 0 for L, n, p in zip(self.lens, rows, self.pages)]
        if any(n and L + n > self.max_len for L, n in zip(self.lens, rows)):
            raise ValueError(f"a slot would hold more than {self.max_len} rows")
        if sum(need) > len(self.free):
            raise MemoryError(f"{sum(need)} pages wanted, {len(self.free)} free")
        if any(need):
            B._need_no_capture(self.table, stream)
        for slot, n in enumerate(need):
            if n:
                for _ in range(n):
                    p = self.free.pop()
                    self.users[p] = 1
                    self.pages[slot].append(p)
                self._write(slot, stream, lengths=False)

    def _one(self, slot):
        if not 0 <= slot < self.n_slots:
            raise ValueError(f"slot {slot} of {self.n_slots}")

    def _rows(self, rows):
        return [int(L >= 0) for L in self.lens] if rows is None else list(rows)

    def _write(self, slot, stream, lengths=True):
        row = self.pages[slot] + [-1] * (self.table.shape[1] - len(self.pages[slot]))
        B._upload(self.table[slot], row, stream)
        if lengths:
            B._upload(self.len[slot:slot + 1], [self.lens[slot]], stream)

    # ---- rows
    def append(self, li: int, rows: B.PagedRows, q_raw, k_raw, v, q, stream=None):
        """Prompts' rows of one layer into the pages (and their bounds); queries to q."""
        B.tv_paged_append(self.layers[li], self.batch, rows, *self.norms[li], self.eps, self.rot_dims, self.theta, q_raw,
                          k_raw, v, q, stream)
        if self.sparse:
            B.tv_paged_bounds(self.layers[li], self.batch, rows, self.code[li], self.exp[li], stream)

    def layer(self, li: int, x: dict, groups: B.PagedGroups | None = None, stream=None):
        """One layer of a decode step: x holds q, k, v [n_slots, heads, D] raw, out and, for a gated layer, gate."""
        layer, batch, gate = self.layers[li], self.batch, x.get("gate")
        B.tv_paged_append(layer, batch, None, *self.norms[li], self.eps, self.rot_dims, self.theta, x["q"], x["k"], x["v"],
                          self.q, stream)
        if not self.sparse:
            B.tv_paged_attn(layer, batch, groups, self.q, gate, x["out"], self.scale, self.ws, stream)
            return
        n_sel, first, last = self.sparse
        B.tv_paged_bounds(layer, batch, None, self.code[li], self.exp[li], stream)
        B.tv_paged_select(layer, batch, self.code[li], self.exp[li], first, last, self.q, self.sel, self.count, self.ws, stream)
        B.tv_paged_attn_selected(layer, batch, self.sel, self.count, self.q, gate, x["out"], self.scale, self.ws, stream)

    def advance(self, rows: B.PagedRows | None = None, stream=None):
        """The device's lengths past a step's rows, after its last layer; advanced() tells the host."""
        B.tv_paged_advance(self.batch, rows, stream)

    def advanced(self, rows=None):
        """The host's lengths past the rows that a step has appended (after each replay of a captured one, too)."""
        self.lens = [L + n if L >= 0 else L for L, n in zip(self.lens, self._rows(rows))]

    def decode(self, inputs, groups: B.PagedGroups | None = None, stream=None):
        """One step through every layer, inputs by layer: room for its rows, the layers, the lengths.  (A captured step is
        layer() and advance(); grow() and advanced() go with each replay.)"""
        B._need_no_capture(self.table, stream)
        self.grow(stream=stream)
        for li, x in enumerate(inputs):
            self.layer(li, x, groups, stream)
        self.advance(stream=stream)
        self.advanced()

    def status(self) -> int:
        return self.batch.status_code()
