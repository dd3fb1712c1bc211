"""Thin ctypes binding of libtreeverify.so (include/tv.h): the same names as
the C ABI, argument marshalling only.  Every step of the verify round runs in
the library's CUDA kernels; there is no Python or CPU fallback, and loading
fails loudly when the library has not been built.

PyTorch provides the device memory and the stream; tensors are passed as raw
device pointers.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_float, c_int32, c_size_t, c_void_p

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtreeverify.so")

TV_MAX_SEQ = 8
TV_MAX_NODES = 64
TV_MAX_PATH = 16
TV_MAX_PAGED_SEQ = 1024
TV_F32, TV_BF16 = 0, 1

STATUS_NAMES = {0: "TV_OK", 1: "TV_ERR_ARG", 2: "TV_ERR_SHAPE", 3: "TV_ERR_DTYPE", 4: "TV_ERR_ALIGN",
                5: "TV_ERR_TREE", 6: "TV_ERR_CAPACITY", 7: "TV_ERR_CUDA", 8: "TV_ERR_WORKSPACE",
                9: "TV_ERR_TIMEOUT", 10: "TV_ERR_LEN", 11: "TV_ERR_SCRATCH", 12: "TV_ERR_ROWS", 13: "TV_ERR_PAGE"}


class TvError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)} ({tv_status_string(code)})")


class tv_tree(ctypes.Structure):
    _fields_ = [("n_seq", c_int32), ("n_total", c_int32), ("n_max", c_int32), ("node_off", c_void_p),
                ("parent", c_void_p), ("meta", c_void_p), ("status", c_void_p), ("flags", c_int32)]


TV_TREE_OVERLAP = 1


class tv_attn_layer(ctypes.Structure):
    _fields_ = [("dtype", c_int32), ("Hq", c_int32), ("Hkv", c_int32), ("D", c_int32), ("cap", c_int32),
                ("K", POINTER(c_void_p)), ("V", POINTER(c_void_p))]


class tv_gdn_layer(ctypes.Structure):
    _fields_ = [("dtype", c_int32), ("Hk", c_int32), ("Hv", c_int32), ("dk", c_int32), ("dv", c_int32),
                ("S", POINTER(c_void_p))]


class tv_gdn_front_layer(ctypes.Structure):
    _fields_ = [("dtype", c_int32), ("Hk", c_int32), ("Hv", c_int32), ("dk", c_int32), ("dv", c_int32),
                ("width", c_int32), ("wconv", c_void_p), ("tail", POINTER(c_void_p))]


class tv_plan(ctypes.Structure):
    _fields_ = [("split", c_int32)]


class tv_prompt(ctypes.Structure):
    _fields_ = [("n_seq", c_int32), ("n_total", c_int32), ("n_max", c_int32), ("row_off", c_void_p),
                ("status", c_void_p)]


class tv_paged_layer(ctypes.Structure):
    _fields_ = [("dtype", c_int32), ("Hq", c_int32), ("Hkv", c_int32), ("D", c_int32), ("page", c_int32),
                ("n_pages", c_int32), ("K", c_void_p), ("V", c_void_p)]


class tv_paged(ctypes.Structure):
    _fields_ = [("n_seq", c_int32), ("cols", c_int32), ("max_len", c_int32), ("table", c_void_p), ("len", c_void_p),
                ("status", c_void_p)]


class tv_paged_rows(ctypes.Structure):
    _fields_ = [("n_total", c_int32), ("n_max", c_int32), ("row_off", c_void_p)]


class tv_paged_groups(ctypes.Structure):
    _fields_ = [("n_group", c_int32), ("group_off", c_void_p), ("shared", c_void_p)]


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with speculative_tree_verify_masked_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        T, A, G, P = POINTER(tv_tree), POINTER(tv_attn_layer), POINTER(tv_gdn_layer), POINTER(tv_plan)
        vp = c_void_p
        L.tv_status_string.restype = ctypes.c_char_p
        L.tv_status_string.argtypes = [c_int32]
        L.tv_version.restype = ctypes.c_char_p
        L.tv_version.argtypes = []
        L.tv_tree_meta_bytes.restype = c_size_t
        L.tv_tree_meta_bytes.argtypes = [c_int32, c_int32]
        L.tv_tree_prepare.restype = c_int32
        L.tv_tree_prepare.argtypes = [T, vp]
        L.tv_attn_workspace_bytes.restype = c_size_t
        L.tv_attn_workspace_bytes.argtypes = [P, A, c_int32, c_int32, c_int32]
        L.tv_attn_tree_verify.restype = c_int32
        L.tv_attn_tree_verify.argtypes = [P, A, T, vp, c_int32, vp, vp, vp, vp, c_float, vp, c_size_t, vp]
        L.tv_gdn_tree_verify.restype = c_int32
        L.tv_gdn_tree_verify.argtypes = [G, T, vp, vp, vp, vp, vp, vp, c_float, vp]
        L.tv_accept_path.restype = c_int32
        L.tv_accept_path.argtypes = [T, vp, vp, vp, vp, vp, vp]
        L.tv_commit_path.restype = c_int32
        L.tv_commit_path.argtypes = [T, vp, vp, c_int32, A, POINTER(vp), POINTER(vp), c_int32, G, POINTER(vp),
                                     POINTER(vp), POINTER(vp), POINTER(vp), vp, vp]
        L.tv_decode_step.restype = c_int32
        L.tv_decode_step.argtypes = [P, A, G, c_int32, vp, c_int32, vp, vp, vp, vp, vp, vp, c_float, vp, c_size_t,
                                     vp, vp]
        L.tv_len_advance.restype = c_int32
        L.tv_len_advance.argtypes = [vp, vp, c_int32, c_int32, vp]
        L.tv_attn_static_scratch_bytes.restype = c_size_t
        L.tv_attn_static_scratch_bytes.argtypes = []
        L.tv_attn_tree_verify_static.restype = c_int32
        L.tv_attn_tree_verify_static.argtypes = [P, A, T, vp, c_int32, vp, vp, vp, vp, c_float, vp]
        L.tv_attn_rope.restype = c_int32
        L.tv_attn_rope.argtypes = [A, T, c_int32, vp, c_int32, c_int32, c_float, vp, vp, vp, vp, vp, vp]
        L.tv_attn_tree_verify_gated.restype = c_int32
        L.tv_attn_tree_verify_gated.argtypes = [P, A, T, vp, c_int32, vp, vp, vp, vp, vp, c_float, vp, c_size_t, vp]
        L.tv_attn_decode_gated.restype = c_int32
        L.tv_attn_decode_gated.argtypes = [P, A, c_int32, vp, c_int32, vp, vp, vp, vp, vp, c_float, vp, c_size_t, vp,
                                           vp]
        F = POINTER(tv_gdn_front_layer)
        L.tv_gdn_front.restype = c_int32
        L.tv_gdn_front.argtypes = [F, T, c_int32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.tv_gdn_out_norm.restype = c_int32
        L.tv_gdn_out_norm.argtypes = [F, c_int32, vp, vp, vp, vp, vp]
        L.tv_gdn_tree_verify_fused.restype = c_int32
        L.tv_gdn_tree_verify_fused.argtypes = [G, F, T, vp, vp, vp, vp, vp, vp, c_float, vp]
        L.tv_gdn_decode_fused.restype = c_int32
        L.tv_gdn_decode_fused.argtypes = [G, F, c_int32, vp, vp, vp, vp, vp, vp, c_float, vp, vp]
        L.tv_gdn_conv_commit.restype = c_int32
        L.tv_gdn_conv_commit.argtypes = [F, T, c_int32, vp, vp, vp, vp, vp]
        L.tv_kvpool_page_bytes.restype = c_size_t
        L.tv_kvpool_page_bytes.argtypes = [c_int32, c_size_t]
        L.tv_kvpool_create.restype = c_int32
        L.tv_kvpool_create.argtypes = [c_int32, c_size_t, POINTER(vp)]
        L.tv_kvpool_reserve.restype = c_int32
        L.tv_kvpool_reserve.argtypes = [vp, c_size_t, POINTER(vp)]
        L.tv_kvpool_commit_rows.restype = c_int32
        L.tv_kvpool_commit_rows.argtypes = [vp, vp, c_int32, c_size_t, c_size_t, ctypes.c_int64, vp]
        L.tv_kvpool_release_rows.restype = c_int32
        L.tv_kvpool_release_rows.argtypes = [vp, vp, c_int32, c_size_t, c_size_t, ctypes.c_int64]
        L.tv_kvpool_committed_bytes.restype = c_size_t
        L.tv_kvpool_committed_bytes.argtypes = [vp]
        L.tv_kvpool_reserved_bytes.restype = c_size_t
        L.tv_kvpool_reserved_bytes.argtypes = [vp]
        L.tv_kvpool_destroy.restype = c_int32
        L.tv_kvpool_destroy.argtypes = [vp]
        R = POINTER(tv_prompt)
        L.tv_prompt_check.restype = c_int32
        L.tv_prompt_check.argtypes = [R, vp, c_int32, c_int32, vp]
        L.tv_prompt_advance.restype = c_int32
        L.tv_prompt_advance.argtypes = [R, vp, vp]
        L.tv_attn_norm_rope.restype = c_int32
        L.tv_attn_norm_rope.argtypes = [A, T, c_int32, vp, c_int32, vp, vp, c_float, c_int32, c_float, vp, vp, vp, vp,
                                        vp, vp]
        L.tv_attn_prompt_front.restype = c_int32
        L.tv_attn_prompt_front.argtypes = [A, R, vp, c_int32, vp, vp, c_float, c_int32, c_float, vp, vp, vp, vp, vp]
        L.tv_attn_prompt_workspace_bytes.restype = c_size_t
        L.tv_attn_prompt_workspace_bytes.argtypes = [A, R, c_int32]
        L.tv_attn_prompt.restype = c_int32
        L.tv_attn_prompt.argtypes = [A, R, vp, c_int32, vp, vp, vp, c_float, vp, c_size_t, vp]
        L.tv_gdn_prompt_workspace_bytes.restype = c_size_t
        L.tv_gdn_prompt_workspace_bytes.argtypes = [G, R]
        L.tv_gdn_prompt.restype = c_int32
        L.tv_gdn_prompt.argtypes = [G, R, vp, vp, vp, vp, vp, vp, c_float, vp, c_size_t, vp]
        L.tv_gdn_prompt_front.restype = c_int32
        L.tv_gdn_prompt_front.argtypes = [F, R, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        PL, PB, PR, PG = POINTER(tv_paged_layer), POINTER(tv_paged), POINTER(tv_paged_rows), POINTER(tv_paged_groups)
        L.tv_paged_append.restype = c_int32
        L.tv_paged_append.argtypes = [PL, PB, PR, vp, vp, c_float, c_int32, c_float, vp, vp, vp, vp, vp]
        L.tv_paged_advance.restype = c_int32
        L.tv_paged_advance.argtypes = [PB, PR, vp, vp]
        L.tv_paged_attn_workspace_bytes.restype = c_size_t
        L.tv_paged_attn_workspace_bytes.argtypes = [PL, PB, PG]
        L.tv_paged_attn.restype = c_int32
        L.tv_paged_attn.argtypes = [PL, PB, PG, vp, vp, vp, c_float, vp, c_size_t, vp]
        L.tv_paged_bounds.restype = c_int32
        L.tv_paged_bounds.argtypes = [PL, PB, PR, vp, vp, vp]
        L.tv_paged_select_workspace_bytes.restype = c_size_t
        L.tv_paged_select_workspace_bytes.argtypes = [PL, PB]
        L.tv_paged_select.restype = c_int32
        L.tv_paged_select.argtypes = [PL, PB, vp, vp, c_int32, c_int32, c_int32, vp, vp, vp, vp, c_size_t, vp]
        L.tv_paged_attn_selected_workspace_bytes.restype = c_size_t
        L.tv_paged_attn_selected_workspace_bytes.argtypes = [PL, PB, c_int32]
        L.tv_paged_attn_selected.restype = c_int32
        L.tv_paged_attn_selected.argtypes = [PL, PB, vp, vp, c_int32, vp, vp, vp, c_float, vp, c_size_t, vp]
        L.tv_wait_selftest.restype = c_int32
        L.tv_wait_selftest.argtypes = [vp, vp, ctypes.c_int64, vp]
        _lib = L
    return _lib


EXPORTED = ["tv_status_string", "tv_version", "tv_tree_meta_bytes", "tv_tree_prepare", "tv_attn_workspace_bytes",
            "tv_attn_tree_verify", "tv_gdn_tree_verify", "tv_accept_path", "tv_commit_path", "tv_decode_step",
            "tv_len_advance", "tv_attn_static_scratch_bytes", "tv_attn_tree_verify_static", "tv_kvpool_page_bytes",
            "tv_kvpool_create", "tv_kvpool_reserve", "tv_kvpool_commit_rows", "tv_kvpool_release_rows",
            "tv_kvpool_committed_bytes", "tv_kvpool_reserved_bytes", "tv_kvpool_destroy", "tv_attn_rope",
            "tv_attn_tree_verify_gated", "tv_attn_decode_gated", "tv_gdn_front", "tv_gdn_out_norm",
            "tv_gdn_conv_commit", "tv_gdn_tree_verify_fused", "tv_gdn_decode_fused", "tv_wait_selftest",
            "tv_prompt_check", "tv_prompt_advance", "tv_attn_norm_rope", "tv_attn_prompt_front", "tv_attn_prompt_workspace_bytes", "tv_attn_prompt",
            "tv_gdn_prompt_workspace_bytes", "tv_gdn_prompt", "tv_gdn_prompt_front", "tv_paged_append", "tv_paged_advance",
            "tv_paged_attn_workspace_bytes", "tv_paged_attn", "tv_paged_bounds", "tv_paged_select_workspace_bytes",
            "tv_paged_select", "tv_paged_attn_selected_workspace_bytes", "tv_paged_attn_selected"]


def _check(code: int, where: str):
    if code != 0:
        raise TvError(code, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _current_gpu() -> int:
    return torch._C._cuda_getDevice()


def _stream(stream):
    if stream is None:
        # the current stream's handle without building a Stream object (a small call's largest host cost)
        return torch._C._cuda_getCurrentRawStream(_current_gpu())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _torch_stream(stream):
    """The torch stream of a call's stream argument."""
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()


def _need_no_capture(dst, stream):
    """Raises inside a graph's capture: what the host writes to a device buffer goes before a replay."""
    if dst.is_cuda:
        with torch.cuda.stream(_torch_stream(stream)):
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("rows are written from the host: before a graph's replay, not inside its capture")


def _upload(dst, values, stream):
    """Writes a few int32 to a device buffer in the stream's order: without
    waiting for it, or, on the current stream (None), until they are there."""
    src = torch.tensor(values, dtype=torch.int32)
    if not dst.is_cuda:
        dst.copy_(src)
        return
    _need_no_capture(dst, stream)
    with torch.cuda.stream(_torch_stream(stream)):
        if stream is None:
            dst.copy_(src)
        else:
            dst.copy_(src.pin_memory(), non_blocking=True)  # (the memory is not reused before the copy has run)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return TV_BF16
    if dt == torch.float32:
        return TV_F32
    raise TypeError(f"unsupported dtype {dt}")


def _alike(tensors, shape, dtype) -> bool:
    """Whether each of a descriptor's tensors is contiguous memory of one GPU, of this shape and dtype."""
    gpu = tensors[0].get_device() if tensors else 0
    return gpu >= 0 and all(tuple(t.shape) == tuple(shape) and t.dtype is dtype and t.is_contiguous() and
                            t.get_device() == gpu for t in tensors)


def _ptr_array(tensors):
    arr = (c_void_p * max(1, len(tensors)))()
    for i, t in enumerate(tensors):
        arr[i] = t.data_ptr()
    return arr


# ---------------------------------------------------------------------------
# descriptors (own the device buffers / pointer arrays they point to)
# ---------------------------------------------------------------------------
class Tree:
    """Device buffers of a tv_tree for a list of per-sequence parent arrays."""

    def __init__(self, parents, device="cuda", n_max=None, overlap: bool = False):
        sizes = [len(p) for p in parents]
        off = [0]
        for n in sizes:
            off.append(off[-1] + n)
        flat = [int(x) for p in parents for x in p]
        self.n_seq = len(parents)
        self.n_total = off[-1]
        self.n_max = n_max if n_max is not None else max(sizes)
        self.node_off = torch.tensor(off, dtype=torch.int32, device=device)
        self.parent = torch.tensor(flat, dtype=torch.int32, device=device)
        self.meta = torch.zeros(max(16, tv_tree_meta_bytes(self.n_seq, self.n_total)), dtype=torch.uint8,
                                device=device)
        self.status = torch.zeros(4, dtype=torch.int32, device=device)
        self.c = tv_tree(self.n_seq, self.n_total, self.n_max, self.node_off.data_ptr(), self.parent.data_ptr(),
                         self.meta.data_ptr(), self.status.data_ptr(), TV_TREE_OVERLAP if overlap else 0)

    def status_code(self) -> int:
        return int(self.status[0].item())


class AttnLayer:
    """tv_attn_layer over per-sequence caches K[s], V[s] of shape [Hkv, cap, D]."""

    def __init__(self, K, V, Hq: int):
        self.K, self.V = list(K), list(V)
        Hkv, cap, D = self.K[0].shape
        self._k, self._v = _ptr_array(self.K), _ptr_array(self.V)
        self.n_seq = min(len(self.K), len(self.V))
        self.sound = _alike(self.K + self.V, self.K[0].shape, self.K[0].dtype)
        self.gpu = self.K[0].get_device()
        self.c = tv_attn_layer(_dtype_code(self.K[0].dtype), Hq, Hkv, D, cap, self._k, self._v)


class GdnLayer:
    """tv_gdn_layer over per-sequence fp32 states S[s] of shape [Hv, dv, dk]."""

    def __init__(self, S, Hk: int, dtype: torch.dtype):
        self.S = list(S)
        Hv, dv, dk = self.S[0].shape
        self._s = _ptr_array(self.S)
        self.n_seq, self.sound = len(self.S), _alike(self.S, self.S[0].shape, torch.float32)
        self.gpu = self.S[0].get_device()
        self.c = tv_gdn_layer(_dtype_code(dtype), Hk, Hv, dk, dv, self._s)


def plan(split: int) -> tv_plan:
    return tv_plan(split)


class Prompt:
    """Device buffers of a tv_prompt for the given rows per sequence.
    n_total and n_max may be larger than the rows need (padding behind the
    last sequence, a graph's bounds); set_rows writes another batch's offsets
    into the same buffer: with `stream`, the calls' one, behind what it holds
    (calls enqueued there before keep their rows) and without waiting; without,
    on the current stream, whose calls before it are waited for."""

    def __init__(self, rows, device="cuda", n_total: int | None = None, n_max: int | None = None):
        off = self._offsets(rows)
        self.n_seq = len(rows)
        self.n_total = off[-1] if n_total is None else n_total
        self.n_max = max(rows) if n_max is None else n_max
        self.row_off = torch.tensor(off, dtype=torch.int32, device=device)
        self.status = torch.zeros(4, dtype=torch.int32, device=device)
        self.c = tv_prompt(self.n_seq, self.n_total, self.n_max, self.row_off.data_ptr(), self.status.data_ptr())

    @staticmethod
    def _offsets(rows):
        off = [0]
        for n in rows:
            off.append(off[-1] + int(n))
        return off

    def set_rows(self, rows, stream=None):
        off = self._offsets(rows)
        if len(rows) != self.n_seq or off[-1] > self.n_total or (rows and max(rows) > self.n_max):
            raise ValueError(f"rows {rows} do not fit {self.n_seq} sequences, {self.n_total} rows, {self.n_max} each")
        _upload(self.row_off, off, stream)

    def counts(self) -> torch.Tensor:
        """Rows of each sequence, on the device (tv_len_advance's `by`)."""
        return (self.row_off[1:] - self.row_off[:-1]).contiguous()

    def status_code(self) -> int:
        return int(self.status[0].item())


class PagedLayer:
    """tv_paged_layer over pools K, V of shape [n_pages, Hkv, page, D]."""

    def __init__(self, K, V, Hq: int):
        self.K, self.V = K, V
        n_pages, Hkv, page, D = K.shape
        self.sound = _alike([K, V], K.shape, K.dtype)
        self.gpu = K.get_device()
        self.c = tv_paged_layer(_dtype_code(K.dtype), Hq, Hkv, D, page, n_pages, K.data_ptr(), V.data_ptr())
        # what a call needs of them, at hand (a small call's time is the host's)
        self.ref, self.dtype = ctypes.byref(self.c), K.dtype
        self.Hkv, self.q_row, self.kv_row, self.D, self.heads = Hkv, Hq * D, Hkv * D, D, n_pages * Hkv


class PagedBatch:
    """tv_paged over a page table [n_seq, cols] and lengths [n_seq] (int32, on
    the GPU; written to by the caller between steps), lengths up to max_len."""

    def __init__(self, table, len_, max_len: int):
        self.table, self.len, self.max_len = table, len_, max_len
        self.n_seq, self.cols = table.shape
        self.sound = _alike([table], (self.n_seq, self.cols), torch.int32) and _alike([len_], (self.n_seq,), torch.int32) \
            and table.get_device() == len_.get_device()
        self.gpu = table.get_device()
        self.status = torch.zeros(4, dtype=torch.int32, device=table.device)
        self.c = tv_paged(self.n_seq, self.cols, max_len, table.data_ptr(), len_.data_ptr(), self.status.data_ptr())
        self.ref = ctypes.byref(self.c)

    def status_code(self) -> int:
        return int(self.status[0].item())


class PagedRows:
    """tv_paged_rows for the given rows per slot; n_total, n_max and set_rows as in Prompt."""

    def __init__(self, rows, device="cuda", n_total: int | None = None, n_max: int | None = None):
        off = Prompt._offsets(rows)
        self.n_seq = len(rows)
        self.n_total = off[-1] if n_total is None else n_total
        self.n_max = max(rows) if n_max is None else n_max
        self.row_off = torch.tensor(off, dtype=torch.int32, device=device)
        self.c = tv_paged_rows(self.n_total, self.n_max, self.row_off.data_ptr())
        self.ref, self.gpu = ctypes.byref(self.c), self.row_off.get_device()

    _offsets = staticmethod(Prompt._offsets)
    set_rows, counts = Prompt.set_rows, Prompt.counts


class PagedGroups:
    """tv_paged_groups: consecutive groups of `sizes` slots (n_seq together) whose first shared[g] rows are the same pages."""

    def __init__(self, sizes, shared, device="cuda"):
        if len(sizes) != len(shared) or not len(sizes):
            raise ValueError("a shared length for each group, one group at least")
        off = Prompt._offsets(sizes)
        self.n_group, self.n_seq = len(sizes), off[-1]
        self.group_off = torch.tensor(off, dtype=torch.int32, device=device)
        self.shared = torch.tensor(list(shared), dtype=torch.int32, device=device)
        self.c = tv_paged_groups(self.n_group, self.group_off.data_ptr(), self.shared.data_ptr())
        self.ref, self.gpu = ctypes.byref(self.c), self.group_off.get_device()

    def set_groups(self, sizes, shared, stream=None):
        """Other groups in the same buffers (as many), in the stream's order as Prompt.set_rows."""
        off = Prompt._offsets(sizes)
        if len(sizes) != self.n_group or len(shared) != self.n_group or off[-1] != self.n_seq:
            raise ValueError(f"groups {sizes} are not {self.n_group} over {self.n_seq} slots")
        _upload(self.group_off, off, stream)
        _upload(self.shared, list(shared), stream)


# ---------------------------------------------------------------------------
# the C ABI, one wrapper per entry point
# ---------------------------------------------------------------------------
def tv_status_string(code: int) -> str:
    return lib().tv_status_string(code).decode()


def tv_version() -> str:
    return lib().tv_version().decode()


def tv_tree_meta_bytes(n_seq: int, n_total: int) -> int:
    return int(lib().tv_tree_meta_bytes(n_seq, n_total))


def tv_tree_prepare(tree: Tree, stream=None):
    _check(lib().tv_tree_prepare(ctypes.byref(tree.c), _stream(stream)), "tv_tree_prepare")


def tv_attn_workspace_bytes(pl: tv_plan, layer: AttnLayer, n_seq: int, n_max: int, max_len: int) -> int:
    return int(lib().tv_attn_workspace_bytes(ctypes.byref(pl), ctypes.byref(layer.c), n_seq, n_max, max_len))


def tv_attn_tree_verify(pl, layer: AttnLayer, tree: Tree, len_, max_len, q, k_t, v_t, out, scale, ws, stream=None):
    _check(lib().tv_attn_tree_verify(ctypes.byref(pl) if pl is not None else None, ctypes.byref(layer.c),
                                     ctypes.byref(tree.c), _ptr(len_), max_len, _ptr(q), _ptr(k_t), _ptr(v_t),
                                     _ptr(out), scale, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                     _stream(stream)), "tv_attn_tree_verify")


def tv_attn_rope(layer: AttnLayer, tree: Tree | None, n_seq, len_, max_len, rot_dims, theta, q_raw, k_raw, q, k,
                 status=None, stream=None):
    """Rotary embedding of one layer's query and key rows at each row's
    logical position (tree: L + depth; tree None: one decode token per
    sequence at L)."""
    _check(lib().tv_attn_rope(ctypes.byref(layer.c), ctypes.byref(tree.c) if tree is not None else None, n_seq,
                              _ptr(len_), max_len, rot_dims, theta, _ptr(q_raw), _ptr(k_raw), _ptr(q), _ptr(k),
                              _ptr(status), _stream(stream)), "tv_attn_rope")


def tv_attn_tree_verify_gated(pl, layer: AttnLayer, tree: Tree, len_, max_len, q, k_t, v_t, gate, out, scale, ws,
                              stream=None):
    _check(lib().tv_attn_tree_verify_gated(ctypes.byref(pl) if pl is not None else None, ctypes.byref(layer.c),
                                           ctypes.byref(tree.c), _ptr(len_), max_len, _ptr(q), _ptr(k_t), _ptr(v_t),
                                           _ptr(gate), _ptr(out), scale, _ptr(ws),
                                           0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
           "tv_attn_tree_verify_gated")


def tv_attn_decode_gated(pl, attn: AttnLayer, n_seq, len_, max_len, q, k, v, gate, out, scale, ws, status,
                         stream=None):
    _check(lib().tv_attn_decode_gated(ctypes.byref(pl) if pl is not None else None, ctypes.byref(attn.c), n_seq,
                                      _ptr(len_), max_len, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(out), scale,
                                      _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _ptr(status),
                                      _stream(stream)), "tv_attn_decode_gated")


class GdnFrontLayer:
    """A tv_gdn_front_layer over torch tensors: wconv [C][W] fp32, one tail
    [W-1][C] per sequence."""

    def __init__(self, Hk: int, Hv: int, dk: int, dv: int, wconv, tails, dtype: torch.dtype):
        self.wconv, self.tails = wconv, list(tails)
        self._tail = _ptr_array(self.tails)
        C, W = 2 * Hk * dk + Hv * dv, wconv.shape[1]
        self.n_seq = len(self.tails)
        self.gpu = wconv.get_device()
        self.sound = _alike([wconv], (C, W), torch.float32) and _alike(self.tails, (W - 1, C), dtype) and all(
            t.get_device() == self.gpu for t in self.tails)
        self.c = tv_gdn_front_layer(_dtype_code(dtype), Hk, Hv, dk, dv, wconv.shape[1], _ptr(wconv), self._tail)


def tv_gdn_front(layer: GdnFrontLayer, tree: Tree | None, n_seq, x, a_raw, b_raw, q, k, v, alpha, beta, status=None,
                 stream=None):
    _check(lib().tv_gdn_front(ctypes.byref(layer.c), ctypes.byref(tree.c) if tree is not None else None, n_seq,
                              _ptr(x), _ptr(a_raw), _ptr(b_raw), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                              _ptr(status), _stream(stream)), "tv_gdn_front")


def tv_gdn_out_norm(layer: GdnFrontLayer, rows, o, z, w_norm, out, stream=None):
    _check(lib().tv_gdn_out_norm(ctypes.byref(layer.c), rows, _ptr(o), _ptr(z), _ptr(w_norm), _ptr(out),
                                 _stream(stream)), "tv_gdn_out_norm")


def tv_gdn_conv_commit(layer: GdnFrontLayer, tree: Tree | None, n_seq, x, path=None, acc_len=None, status=None,
                       stream=None):
    _check(lib().tv_gdn_conv_commit(ctypes.byref(layer.c), ctypes.byref(tree.c) if tree is not None else None, n_seq,
                                    _ptr(x), _ptr(path), _ptr(acc_len), _ptr(status), _stream(stream)),
           "tv_gdn_conv_commit")


def tv_attn_static_scratch_bytes() -> int:
    return int(lib().tv_attn_static_scratch_bytes())


def tv_attn_tree_verify_static(pl, layer: AttnLayer, tree: Tree, len_, max_len, q, k_t, v_t, out, scale,
                               stream=None):
    _check(lib().tv_attn_tree_verify_static(ctypes.byref(pl) if pl is not None else None, ctypes.byref(layer.c),
                                            ctypes.byref(tree.c), _ptr(len_), max_len, _ptr(q), _ptr(k_t),
                                            _ptr(v_t), _ptr(out), scale, _stream(stream)),
           "tv_attn_tree_verify_static")


def tv_gdn_tree_verify(layer: GdnLayer, tree: Tree, q, k, v, alpha, beta, out, scale, stream=None):
    _check(lib().tv_gdn_tree_verify(ctypes.byref(layer.c), ctypes.byref(tree.c), _ptr(q), _ptr(k), _ptr(v),
                                    _ptr(alpha), _ptr(beta), _ptr(out), scale, _stream(stream)),
           "tv_gdn_tree_verify")


def tv_gdn_tree_verify_fused(layer: GdnLayer, front: GdnFrontLayer, tree: Tree, x, a_raw, b_raw, z, w_norm, out,
                             scale, stream=None):
    _check(lib().tv_gdn_tree_verify_fused(ctypes.byref(layer.c), ctypes.byref(front.c), ctypes.byref(tree.c), _ptr(x),
                                          _ptr(a_raw), _ptr(b_raw), _ptr(z), _ptr(w_norm), _ptr(out), scale,
                                          _stream(stream)), "tv_gdn_tree_verify_fused")


def tv_gdn_decode_fused(layer: GdnLayer, front: GdnFrontLayer, n_seq, x, a_raw, b_raw, z, w_norm, out, scale, status,
                        stream=None):
    _check(lib().tv_gdn_decode_fused(ctypes.byref(layer.c), ctypes.byref(front.c), n_seq, _ptr(x), _ptr(a_raw),
                                     _ptr(b_raw), _ptr(z), _ptr(w_norm), _ptr(out), scale, _ptr(status),
                                     _stream(stream)), "tv_gdn_decode_fused")


def tv_accept_path(tree: Tree, tok, greedy, path, acc_len, bonus, stream=None):
    _check(lib().tv_accept_path(ctypes.byref(tree.c), _ptr(tok), _ptr(greedy), _ptr(path), _ptr(acc_len),
                                _ptr(bonus), _stream(stream)), "tv_accept_path")


class CommitArgs:
    """Marshalled argument block of tv_commit_path for fixed layer lists."""

    def __init__(self, attn_layers, k_t, v_t, gdn_layers, k, v, alpha, beta):
        self.n_attn, self.n_gdn = len(attn_layers), len(gdn_layers)
        self.attn = (tv_attn_layer * max(1, self.n_attn))(*[l.c for l in attn_layers])
        self.gdn = (tv_gdn_layer * max(1, self.n_gdn))(*[l.c for l in gdn_layers])
        self.keep = (attn_layers, gdn_layers, k_t, v_t, k, v, alpha, beta)
        self.k_t, self.v_t = _ptr_array(k_t), _ptr_array(v_t)
        self.k, self.v = _ptr_array(k), _ptr_array(v)
        self.alpha, self.beta = _ptr_array(alpha), _ptr_array(beta)


def tv_commit_path(tree: Tree, path, acc_len, args: CommitArgs, len_, stream=None):
    _check(lib().tv_commit_path(ctypes.byref(tree.c), _ptr(path), _ptr(acc_len), args.n_attn, args.attn, args.k_t,
                                args.v_t, args.n_gdn, args.gdn, args.k, args.v, args.alpha, args.beta, _ptr(len_),
                                _stream(stream)), "tv_commit_path")


def tv_decode_step(pl, attn: AttnLayer | None, gdn: GdnLayer | None, n_seq, len_, max_len, q, k, v, alpha, beta,
                   out, scale, ws, status, stream=None):
    _check(lib().tv_decode_step(ctypes.byref(pl) if pl is not None else None,
                                ctypes.byref(attn.c) if attn is not None else None,
                                ctypes.byref(gdn.c) if gdn is not None else None, n_seq, _ptr(len_), max_len,
                                _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(out), scale, _ptr(ws),
                                0 if ws is None else ws.numel() * ws.element_size(), _ptr(status), _stream(stream)),
           "tv_decode_step")


def tv_len_advance(len_, by, inc: int, n_seq: int, stream=None):
    _check(lib().tv_len_advance(_ptr(len_), _ptr(by), inc, n_seq, _stream(stream)), "tv_len_advance")


# ---------------------------------------------------------------------------
# prompts
# ---------------------------------------------------------------------------
def _need(where: str, **tensors):
    """Raises where a buffer is not what the C side will take it for: each
    value is (tensor, dtype, elements); the memory must be contiguous, on the
    current GPU (where the call's kernels run), and hold at least that many
    elements."""
    here = -1
    for name, (t, dtype, n) in tensors.items():
        if t is None:
            continue
        gpu = t.get_device()  # (-1: host memory)
        if t.dtype is not dtype or not t.is_contiguous() or gpu < 0 or t.numel() < n:
            raise ValueError(f"{where}: {name} must be a contiguous {dtype} GPU tensor of at least {n} elements, got "
                             f"{tuple(t.shape)} {t.dtype} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")
        if gpu != here:
            here = _current_gpu()
            if gpu != here:
                raise ValueError(f"{where}: {name} is on GPU {gpu}, the current one is {here}")


def _need_layer(where: str, layer, prompt):
    """Raises where a layer's caches, states or tails are fewer than the call's
    sequences (the C side would read past its pointers), not alike, or not on
    the current GPU, or the prompt's rows are not there."""
    if layer.n_seq < prompt.n_seq:
        raise ValueError(f"{where}: {prompt.n_seq} sequences, but the layer holds {layer.n_seq}")
    if not layer.sound:
        raise ValueError(f"{where}: the layer's tensors must be contiguous memory of one GPU, of one shape and dtype each")
    here = _current_gpu()
    if layer.gpu != here or prompt.row_off.get_device() != here:
        raise ValueError(f"{where}: the layer is on GPU {layer.gpu}, the rows are on {prompt.row_off.device}, the current "
                         f"GPU is {here}")


def _ws_bytes(ws) -> int:
    if ws is None:
        return 0
    if not ws.is_cuda or not ws.is_contiguous() or ws.get_device() != _current_gpu():
        raise ValueError("the workspace must be contiguous memory of the current GPU")
    return ws.numel() * ws.element_size()


def tv_prompt_check(prompt: Prompt, len_, max_len: int, cap: int, stream=None):
    """The checks of a span, before its first layer."""
    _need("tv_prompt_check", len=(len_, torch.int32, prompt.n_seq))
    _check(lib().tv_prompt_check(ctypes.byref(prompt.c), _ptr(len_), max_len, cap, _stream(stream)), "tv_prompt_check")


def tv_prompt_advance(prompt: Prompt, len_, stream=None):
    """The lengths past the span, after its last layer; not past a refused one."""
    _need("tv_prompt_advance", len=(len_, torch.int32, prompt.n_seq))
    _check(lib().tv_prompt_advance(ctypes.byref(prompt.c), _ptr(len_), _stream(stream)), "tv_prompt_advance")


def tv_attn_norm_rope(layer: AttnLayer, tree: Tree | None, n_seq, len_, max_len, q_norm, k_norm, eps, rot_dims, theta,
                      q_raw, k_raw, q, k, status=None, stream=None):
    """Head norms and rotation of one layer's query and key rows (positions as in tv_attn_rope)."""
    c, dt = layer.c, layer.K[0].dtype
    n = tree.n_total if tree is not None else n_seq
    nq, nk = n * c.Hq * c.D, n * c.Hkv * c.D
    _need("tv_attn_norm_rope", len=(len_, torch.int32, tree.n_seq if tree is not None else n_seq),
          q_norm=(q_norm, torch.float32, c.D), k_norm=(k_norm, torch.float32, c.D), q_raw=(q_raw, dt, nq),
          k_raw=(k_raw, dt, nk), q=(q, dt, nq), k=(k, dt, nk))
    _check(lib().tv_attn_norm_rope(ctypes.byref(c), ctypes.byref(tree.c) if tree is not None else None, n_seq,
                                   _ptr(len_), max_len, _ptr(q_norm), _ptr(k_norm), eps, rot_dims, theta, _ptr(q_raw),
                                   _ptr(k_raw), _ptr(q), _ptr(k), _ptr(status), _stream(stream)), "tv_attn_norm_rope")


def tv_attn_prompt_front(layer: AttnLayer, prompt: Prompt, len_, max_len, q_norm, k_norm, eps, rot_dims, theta, q_raw,
                         k_raw, v, q, stream=None):
    """Head norms and rotation of a prompt's rows; keys and values go into the caches."""
    _need_layer("tv_attn_prompt_front", layer, prompt)
    c, dt, n = layer.c, layer.K[0].dtype, prompt.n_total
    nq, nk = n * c.Hq * c.D, n * c.Hkv * c.D
    _need("tv_attn_prompt_front", len=(len_, torch.int32, prompt.n_seq), q_norm=(q_norm, torch.float32, c.D),
          k_norm=(k_norm, torch.float32, c.D), q_raw=(q_raw, dt, nq), k_raw=(k_raw, dt, nk), v=(v, dt, nk),
          q=(q, dt, nq))
    _check(lib().tv_attn_prompt_front(ctypes.byref(c), ctypes.byref(prompt.c), _ptr(len_), max_len, _ptr(q_norm),
                                      _ptr(k_norm), eps, rot_dims, theta, _ptr(q_raw), _ptr(k_raw), _ptr(v), _ptr(q),
                                      _stream(stream)), "tv_attn_prompt_front")


def tv_attn_prompt_workspace_bytes(layer: AttnLayer, prompt: Prompt, max_len: int) -> int:
    return int(lib().tv_attn_prompt_workspace_bytes(ctypes.byref(layer.c), ctypes.byref(prompt.c), max_len))


def tv_attn_prompt(layer: AttnLayer, prompt: Prompt, len_, max_len, q, gate, out, scale, ws, stream=None):
    """Causal attention of a prompt's rows over the caches that hold them."""
    _need_layer("tv_attn_prompt", layer, prompt)
    c, dt = layer.c, layer.K[0].dtype
    nq = prompt.n_total * c.Hq * c.D
    _need("tv_attn_prompt", len=(len_, torch.int32, prompt.n_seq), q=(q, dt, nq), gate=(gate, dt, nq),
          out=(out, dt, nq))
    _check(lib().tv_attn_prompt(ctypes.byref(c), ctypes.byref(prompt.c), _ptr(len_), max_len, _ptr(q), _ptr(gate),
                                _ptr(out), scale, _ptr(ws), _ws_bytes(ws), _stream(stream)), "tv_attn_prompt")


def tv_gdn_prompt_workspace_bytes(layer: GdnLayer, prompt: Prompt) -> int:
    return int(lib().tv_gdn_prompt_workspace_bytes(ctypes.byref(layer.c), ctypes.byref(prompt.c)))


def tv_gdn_prompt(layer: GdnLayer, prompt: Prompt, q, k, v, alpha, beta, out, scale, ws, stream=None):
    """The gated delta rule over a prompt's rows; the states advance in place."""
    _need_layer("tv_gdn_prompt", layer, prompt)
    c, n = layer.c, prompt.n_total
    dt = torch.bfloat16 if c.dtype == TV_BF16 else torch.float32
    nk, nv, nh = n * c.Hk * c.dk, n * c.Hv * c.dv, n * c.Hv
    _need("tv_gdn_prompt", q=(q, dt, nk), k=(k, dt, nk), v=(v, dt, nv), alpha=(alpha, torch.float32, nh),
          beta=(beta, torch.float32, nh), out=(out, dt, nv))
    _check(lib().tv_gdn_prompt(ctypes.byref(c), ctypes.byref(prompt.c), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                               _ptr(beta), _ptr(out), scale, _ptr(ws), _ws_bytes(ws), _stream(stream)),
           "tv_gdn_prompt")


def tv_gdn_prompt_front(layer: GdnFrontLayer, prompt: Prompt, x, a_raw, b_raw, q, k, v, alpha, beta, stream=None):
    """The GDN front end over a prompt's rows; the convolution tails advance."""
    _need_layer("tv_gdn_prompt_front", layer, prompt)
    c, n = layer.c, prompt.n_total
    dt = torch.bfloat16 if c.dtype == TV_BF16 else torch.float32
    nk, nv, nh = n * c.Hk * c.dk, n * c.Hv * c.dv, n * c.Hv
    _need("tv_gdn_prompt_front", x=(x, dt, 2 * nk + nv), a_raw=(a_raw, torch.float32, nh),
          b_raw=(b_raw, torch.float32, nh), q=(q, dt, nk), k=(k, dt, nk), v=(v, dt, nv),
          alpha=(alpha, torch.float32, nh), beta=(beta, torch.float32, nh))
    _check(lib().tv_gdn_prompt_front(ctypes.byref(c), ctypes.byref(prompt.c), _ptr(x), _ptr(a_raw), _ptr(b_raw),
                                     _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _stream(stream)),
           "tv_gdn_prompt_front")


# ---------------------------------------------------------------------------
# caches in pages
# ---------------------------------------------------------------------------
def _need_paged(where: str, layer, batch, extra, here):
    """Raises where a paged call's descriptors are not memory of the current GPU
    of the shapes they say, or its rows or groups are for another number of slots."""
    if not layer.sound or not batch.sound:
        raise ValueError(f"{where}: pools, table and lengths must be contiguous memory of one GPU, the pools alike, the others int32")
    if layer.gpu != here or batch.gpu != here:
        raise ValueError(f"{where}: the pools are on GPU {layer.gpu}, the batch is on {batch.gpu}, the current GPU is {here}")
    if extra is not None and (extra.n_seq != batch.n_seq or extra.gpu != here):
        raise ValueError(f"{where}: rows or groups for {extra.n_seq} slots, {batch.n_seq} in the batch, or of another GPU than {here}")


def _paged(where: str, layer, batch, extra, stream):
    """What every paged call begins with: its descriptors checked; the current GPU and the stream."""
    here = _current_gpu()
    if not (layer.sound and batch.sound and layer.gpu == here and batch.gpu == here and
            (extra is None or (extra.n_seq == batch.n_seq and extra.gpu == here))):
        _need_paged(where, layer, batch, extra, here)
    return here, torch._C._cuda_getCurrentRawStream(here) if stream is None else _stream(stream)


def _fits(t, dtype, n, here):
    """Whether a buffer is what the C side will take it for (None: not given); _need says what is not."""
    return t is None or (t.dtype is dtype and t.get_device() == here and t.is_contiguous() and t.numel() >= n)


def _space(ws, here) -> int:
    """Bytes of a workspace, which must be contiguous memory of the current GPU."""
    if ws is None:
        return 0
    return ws.nbytes if ws.get_device() == here and ws.is_contiguous() else _ws_bytes(ws)


def _ref(x):
    return None if x is None else x.ref


def tv_paged_append(layer: PagedLayer, batch: PagedBatch, rows: PagedRows | None, q_norm, k_norm, eps, rot_dims, theta,
                    q_raw, k_raw, v, q, stream=None):
    """Head norms and rotation of a step's rows (rows None: one a slot) or of
    prompts' rows; queries to q, keys and values into the slots' pages."""
    here, st = _paged("tv_paged_append", layer, batch, rows, stream)
    n, dt, f32 = batch.n_seq if rows is None else rows.n_total, layer.dtype, torch.float32
    nq, nk = n * layer.q_row, n * layer.kv_row
    # (_fits written out: its calls were a tenth of a small call's time)
    if not (q_raw.dtype is dt and q_raw.get_device() == here and q_raw.is_contiguous() and q_raw.numel() >= nq and
            k_raw.dtype is dt and k_raw.get_device() == here and k_raw.is_contiguous() and k_raw.numel() >= nk and
            v.dtype is dt and v.get_device() == here and v.is_contiguous() and v.numel() >= nk and
            q.dtype is dt and q.get_device() == here and q.is_contiguous() and q.numel() >= nq and
            _fits(q_norm, f32, layer.D, here) and _fits(k_norm, f32, layer.D, here)):
        _need("tv_paged_append", q_norm=(q_norm, f32, layer.D), k_norm=(k_norm, f32, layer.D), q_raw=(q_raw, dt, nq),
              k_raw=(k_raw, dt, nk), v=(v, dt, nk), q=(q, dt, nq))
    code = lib().tv_paged_append(layer.ref, batch.ref, None if rows is None else rows.ref, _ptr(q_norm), _ptr(k_norm), eps,
                                 rot_dims, theta, q_raw.data_ptr(), k_raw.data_ptr(), v.data_ptr(), q.data_ptr(), st)
    if code:
        _check(code, "tv_paged_append")


def tv_paged_advance(batch: PagedBatch, rows: PagedRows | None = None, stream=None):
    """The batch's lengths past a step's rows, after its last layer."""
    here, st = _paged("tv_paged_advance", batch, batch, rows, stream)
    _check(lib().tv_paged_advance(batch.ref, _ref(rows), _ptr(batch.len), st), "tv_paged_advance")


def tv_paged_attn_workspace_bytes(layer: PagedLayer, batch: PagedBatch, groups: PagedGroups | None = None) -> int:
    return int(lib().tv_paged_attn_workspace_bytes(layer.ref, batch.ref, _ref(groups)))


def tv_paged_attn(layer: PagedLayer, batch: PagedBatch, groups: PagedGroups | None, q, gate, out, scale, ws, stream=None):
    """Decode attention over pages; the prefixes that groups share are read once."""
    here, st = _paged("tv_paged_attn", layer, batch, groups, stream)
    dt, nq = layer.dtype, batch.n_seq * layer.q_row
    if not (_fits(q, dt, nq, here) and _fits(gate, dt, nq, here) and _fits(out, dt, nq, here)):
        _need("tv_paged_attn", q=(q, dt, nq), gate=(gate, dt, nq), out=(out, dt, nq))
    code = lib().tv_paged_attn(layer.ref, batch.ref, _ref(groups), _ptr(q), _ptr(gate), _ptr(out), scale, _ptr(ws),
                               _space(ws, here), st)
    if code:
        _check(code, "tv_paged_attn")


def tv_paged_bounds(layer: PagedLayer, batch: PagedBatch, rows: PagedRows | None, code, exp, stream=None):
    """Bounds of the pages that a step's rows complete: code int8 [n_pages, Hkv, 2, D], exp int32 [n_pages, Hkv]."""
    here, st = _paged("tv_paged_bounds", layer, batch, rows, stream)
    nc = layer.heads * 2 * layer.D
    if not (_fits(code, torch.int8, nc, here) and _fits(exp, torch.int32, layer.heads, here)):
        _need("tv_paged_bounds", code=(code, torch.int8, nc), exp=(exp, torch.int32, layer.heads))
    status = lib().tv_paged_bounds(layer.ref, batch.ref, _ref(rows), _ptr(code), _ptr(exp), st)
    if status:
        _check(status, "tv_paged_bounds")


def tv_paged_select_workspace_bytes(layer: PagedLayer, batch: PagedBatch) -> int:
    return int(lib().tv_paged_select_workspace_bytes(layer.ref, batch.ref))


def tv_paged_select(layer: PagedLayer, batch: PagedBatch, code, exp, first: int, last: int, q, sel, count, ws=None, stream=None):
    """The pages that each slot's queries look at: sel int32 [n_seq, Hkv, n_sel], count int32 [n_seq, Hkv]."""
    here, st = _paged("tv_paged_select", layer, batch, None, stream)
    n_sel, units, i32 = sel.shape[-1], batch.n_seq * layer.Hkv, torch.int32
    nc, nq = layer.heads * 2 * layer.D, batch.n_seq * layer.q_row
    if not (code.dtype is torch.int8 and code.get_device() == here and code.is_contiguous() and code.numel() >= nc and
            exp.dtype is i32 and exp.get_device() == here and exp.is_contiguous() and exp.numel() >= layer.heads and
            q.dtype is layer.dtype and q.get_device() == here and q.is_contiguous() and q.numel() >= nq and
            sel.dtype is i32 and sel.get_device() == here and sel.is_contiguous() and sel.numel() >= units * n_sel and
            count.dtype is i32 and count.get_device() == here and count.is_contiguous() and count.numel() >= units):
        _need("tv_paged_select", code=(code, torch.int8, nc), exp=(exp, i32, layer.heads), q=(q, layer.dtype, nq),
              sel=(sel, i32, units * n_sel), count=(count, i32, units))
    status = lib().tv_paged_select(layer.ref, batch.ref, code.data_ptr(), exp.data_ptr(), first, last, n_sel, q.data_ptr(),
                                   sel.data_ptr(), count.data_ptr(), _ptr(ws), _space(ws, here), st)
    if status:
        _check(status, "tv_paged_select")


def tv_paged_attn_selected_workspace_bytes(layer: PagedLayer, batch: PagedBatch, n_sel: int) -> int:
    return int(lib().tv_paged_attn_selected_workspace_bytes(layer.ref, batch.ref, n_sel))


def tv_paged_attn_selected(layer: PagedLayer, batch: PagedBatch, sel, count, q, gate, out, scale, ws, stream=None):
    """Decode attention over the listed pages alone."""
    here, st = _paged("tv_paged_attn_selected", layer, batch, None, stream)
    n_sel, units, dt, i32 = sel.shape[-1], batch.n_seq * layer.Hkv, layer.dtype, torch.int32
    nq = batch.n_seq * layer.q_row
    if not (_fits(sel, i32, units * n_sel, here) and _fits(count, i32, units, here) and _fits(q, dt, nq, here) and
            _fits(gate, dt, nq, here) and _fits(out, dt, nq, here)):
        _need("tv_paged_attn_selected", sel=(sel, i32, units * n_sel), count=(count, i32, units), q=(q, dt, nq),
              gate=(gate, dt, nq), out=(out, dt, nq))
    code = lib().tv_paged_attn_selected(layer.ref, batch.ref, _ptr(sel), _ptr(count), n_sel, _ptr(q), _ptr(gate), _ptr(out),
                                        scale, _ptr(ws), _space(ws, here), st)
    if code:
        _check(code, "tv_paged_attn_selected")


# ---------------------------------------------------------------------------
# KV pool
# ---------------------------------------------------------------------------
def tv_wait_selftest(status, result, limit_cycles: int, stream=None):
    _check(lib().tv_wait_selftest(_ptr(status), _ptr(result), int(limit_cycles), _stream(stream)), "tv_wait_selftest")


def tv_kvpool_page_bytes(device: int, page_bytes: int = 0) -> int:
    return int(lib().tv_kvpool_page_bytes(device, page_bytes))


def tv_kvpool_create(device: int, page_bytes: int = 0) -> c_void_p:
    h = c_void_p()
    _check(lib().tv_kvpool_create(device, page_bytes, ctypes.byref(h)), "tv_kvpool_create")
    return h


def tv_kvpool_reserve(pool, nbytes: int) -> int:
    base = c_void_p()
    _check(lib().tv_kvpool_reserve(pool, nbytes, ctypes.byref(base)), "tv_kvpool_reserve")
    return int(base.value)


def tv_kvpool_commit_rows(pool, base: int, n_heads: int, head_stride: int, row_bytes: int, rows: int, stream=None):
    _check(lib().tv_kvpool_commit_rows(pool, c_void_p(base), n_heads, head_stride, row_bytes, rows, _stream(stream)),
           "tv_kvpool_commit_rows")


def tv_kvpool_release_rows(pool, base: int, n_heads: int, head_stride: int, row_bytes: int, keep_rows: int):
    _check(lib().tv_kvpool_release_rows(pool, c_void_p(base), n_heads, head_stride, row_bytes, keep_rows),
           "tv_kvpool_release_rows")


def tv_kvpool_committed_bytes(pool) -> int:
    return int(lib().tv_kvpool_committed_bytes(pool))


def tv_kvpool_reserved_bytes(pool) -> int:
    return int(lib().tv_kvpool_reserved_bytes(pool))


def tv_kvpool_destroy(pool):
    _check(lib().tv_kvpool_destroy(pool), "tv_kvpool_destroy")


class _DeviceRange:
    """A device address range presented to torch through the CUDA array
    interface (torch keeps this object alive with the tensor)."""

    def __init__(self, ptr: int, numel: int, typestr: str, pool):
        self.pool = pool
        self.__cuda_array_interface__ = {"shape": (numel,), "typestr": typestr, "data": (ptr, False),
                                         "version": 3, "strides": None, "stream": None}


class KVPool:
    """Caches [H][cap][D] whose address space is reserved whole and whose
    pages are committed as rows are written (tv_kvpool_*)."""

    _TYPESTR = {torch.float32: "<f4", torch.bfloat16: "<i2", torch.float16: "<f2"}

    def __init__(self, device: int = 0, page_bytes: int = 0):
        self.device = device
        self.h = tv_kvpool_create(device, page_bytes)
        self.page_bytes = tv_kvpool_page_bytes(device, page_bytes)

    def cache(self, heads: int, cap: int, dim: int, dtype: torch.dtype) -> torch.Tensor:
        """A [heads, cap, dim] tensor over a fresh reservation; row 0 of every
        head is committed (zeroed), nothing else."""
        esize = torch.empty((), dtype=dtype).element_size()
        numel = heads * cap * dim
        base = tv_kvpool_reserve(self.h, numel * esize)
        tv_kvpool_commit_rows(self.h, base, heads, cap * dim * esize, dim * esize, 1)
        t = torch.as_tensor(_DeviceRange(base, numel, self._TYPESTR[dtype], self), device=f"cuda:{self.device}")
        return t.view(dtype).view(heads, cap, dim)

    @staticmethod
    def _geom(t: torch.Tensor):
        heads, cap, dim = t.shape
        es = t.element_size()
        return t.data_ptr(), heads, cap * dim * es, dim * es

    def commit_rows(self, t: torch.Tensor, rows: int, stream=None):
        base, heads, hs, rb = self._geom(t)
        tv_kvpool_commit_rows(self.h, base, heads, hs, rb, rows, stream)

    def release_rows(self, t: torch.Tensor, keep_rows: int):
        base, heads, hs, rb = self._geom(t)
        tv_kvpool_release_rows(self.h, base, heads, hs, rb, keep_rows)

    @property
    def committed_bytes(self) -> int:
        return tv_kvpool_committed_bytes(self.h)

    @property
    def reserved_bytes(self) -> int:
        return tv_kvpool_reserved_bytes(self.h)

    def close(self):
        """Frees every page and reservation: tensors from cache() must not be
        used afterwards."""
        if self.h is not None:
            tv_kvpool_destroy(self.h)
            self.h = None
