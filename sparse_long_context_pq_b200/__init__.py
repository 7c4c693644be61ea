"""PQ-HSA sparse decode attention for B200 (sm_100a): Python binding of libpqhsa.so.

Every step of the decode path runs in the library's CUDA kernels; this module only
marshals torch tensors (device memory) and the current CUDA stream into the C ABI
declared in include/pqhsa.h. There is no CPU fallback: importing works without a
GPU, but every compute call needs the built library and a CUDA device.

Method: rit.work "pq-hsa-long-context-attention" (PQ-HSA).
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

from . import build as _build

__all__ = [
    "PagedKV", "PQIndex", "HSAError", "load_library", "hsa_decode", "hsa_decode_host", "dense_decode",
    "hsa_build_from_codes", "hsa_append_encode", "hsa_decode_workspace_bytes", "hsa_decode_host_workspace_bytes",
    "dense_decode_workspace_bytes", "hsa_index_workspace_bytes", "hsa_read_error", "hsa_strerror",
    "selected_counts", "DecodeStep", "HSA_DEVERR_PAGE", "HSA_DEVERR_CLUSTER", "HSA_DEVERR_TIMEOUT",
    "HSA_DEVERR_SELECT",
    "HSA_DEVERR_LIMIT", "KV4Cache", "KV4_TILE_BYTES", "hsa_kv4_workspace_bytes", "hsa_kv4_write", "hsa_kv4_read", "dense_decode_kv4",
    "dense_prefill_kv4",
]

HSA_DEVERR_PAGE, HSA_DEVERR_CLUSTER, HSA_DEVERR_TIMEOUT, HSA_DEVERR_SELECT = 1, 2, 4, 8
HSA_DEVERR_LIMIT = 32
M_SUB, DSUB, NCODE, HEAD_DIM = 16, 8, 256, 128
KV4_TILE_TOKENS, KV4_TILE_BYTES = 16, 2304


class _KV(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("seq_lens_host", ctypes.c_void_p),
                ("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("num_pages", ctypes.c_int32)]


class _Index(ctypes.Structure):
    _fields_ = [("centroids", ctypes.c_void_p), ("codebooks", ctypes.c_void_p), ("codes", ctypes.c_void_p),
                ("ids", ctypes.c_void_p), ("sum_v", ctypes.c_void_p), ("mean_v", ctypes.c_void_p),
                ("count", ctypes.c_void_p), ("n_indexed", ctypes.c_void_p), ("n_indexed_host", ctypes.c_void_p),
                ("list_codes", ctypes.c_void_p), ("list_slot", ctypes.c_void_p),
                ("chunk_cluster", ctypes.c_void_p), ("list_meta", ctypes.c_void_p),
                ("C", ctypes.c_int32), ("M", ctypes.c_int32), ("dsub", ctypes.c_int32),
                ("ncode", ctypes.c_int32), ("cap", ctypes.c_int32), ("n_sink", ctypes.c_int32),
                ("list_slots", ctypes.c_int32)]


class _KV4(ctypes.Structure):
    _fields_ = [("cache", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("seq_lens_host", ctypes.c_void_p),
                ("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("D", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("num_pages", ctypes.c_int32)]


class _KV4Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


def index_list_slots(cap: int, C: int) -> int:
    """List slots per unit the cluster-ordered code lists need: 32 * (ceil(cap / 32) + C)."""
    return 32 * ((cap + 31) // 32 + C)


class _Params(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("budget", ctypes.c_double), ("k_override", ctypes.c_int32),
                ("background", ctypes.c_int32)]


class _Debug(ctypes.Structure):
    _fields_ = [("approx_logits", ctypes.c_void_p), ("selected", ctypes.c_void_p),
                ("n_selected", ctypes.c_void_p), ("stage_events", ctypes.c_void_p)]


NUM_STAGES = 4
STAGE_NAMES = ("tables", "scan_select", "attend", "merge")


EXPORTS = ("hsa_decode", "hsa_decode_host", "hsa_decode_step_create", "hsa_decode_step_run",
           "hsa_decode_step_destroy", "dense_decode", "hsa_build_from_codes", "hsa_append_encode",
           "hsa_index_list_slots", "hsa_decode_workspace_bytes", "hsa_decode_host_workspace_bytes",
           "dense_decode_workspace_bytes", "hsa_index_workspace_bytes",
           "hsa_read_error", "hsa_strerror", "hsa_abi_sizes", "hsa_kv4_workspace_bytes", "hsa_kv4_write",
           "hsa_kv4_read", "dense_decode_kv4", "dense_prefill_kv4", "hsa_kv4_abi_sizes")

_lib = None


class HSAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {hsa_strerror(status)} (status {status})")
        self.status = status


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libpqhsa.so (built in-tree by sparse_long_context_pq_b200.build). Raises if missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or os.environ.get("PQHSA_LIB", _build.LIB_PATH)
    if not os.path.exists(path):
        raise RuntimeError(f"libpqhsa.so not found at {path}; build it with "
                           f"`python -m sparse_long_context_pq_b200.build`")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.hsa_decode.argtypes = [P(_KV), P(_Index), vp, vp, P(_Params), P(_Debug), vp, sz, vp]
    lib.hsa_decode_host.argtypes = [P(_KV), P(_Index), vp, vp, P(_Params), vp, sz, vp]
    lib.hsa_decode_host_workspace_bytes.argtypes = [P(_KV), P(_Index)]
    lib.hsa_decode_step_create.argtypes = [P(_KV), P(_Index), P(_Params), vp, sz, P(vp)]
    lib.hsa_decode_step_run.argtypes = [vp, vp, vp, vp]
    lib.hsa_decode_step_destroy.argtypes = [vp]
    lib.hsa_decode_step_destroy.restype = None
    lib.dense_decode.argtypes = [P(_KV), vp, vp, ctypes.c_float, vp, sz, vp]
    lib.hsa_build_from_codes.argtypes = [P(_KV), P(_Index), vp, sz, vp]
    lib.hsa_append_encode.argtypes = [P(_KV), P(_Index), i32, vp, sz, vp]
    lib.hsa_train_workspace_bytes.argtypes = [P(_KV), P(_Index), i32]
    lib.hsa_train_index.argtypes = [P(_KV), P(_Index), i32, vp, i32, i32, vp, vp, sz, vp]
    lib.hsa_decode_workspace_bytes.argtypes = [P(_KV), P(_Index)]
    lib.dense_decode_workspace_bytes.argtypes = [P(_KV)]
    lib.hsa_index_workspace_bytes.argtypes = [P(_KV), P(_Index), i32]
    lib.hsa_read_error.argtypes = [vp, P(i32), vp]
    lib.hsa_strerror.argtypes = [ctypes.c_int]
    lib.hsa_abi_sizes.argtypes = [P(ctypes.c_int64)] * 4
    i64, f32 = ctypes.c_int64, ctypes.c_float
    lib.hsa_kv4_workspace_bytes.argtypes = [P(_KV4)]
    lib.hsa_kv4_workspace_bytes.restype = sz
    lib.hsa_kv4_write.argtypes = [P(_KV4), P(_KV4Rows), P(_KV4Rows), i32, vp, vp, vp, sz, vp]
    lib.hsa_kv4_read.argtypes = [P(_KV4), P(_KV4Rows), P(_KV4Rows), i32, vp, vp, vp, vp, vp, sz, vp]
    lib.dense_decode_kv4.argtypes = [P(_KV4), vp, vp, vp, i32, f32, i32, vp, sz, vp]
    lib.dense_prefill_kv4.argtypes = [P(_KV4), vp, i64, vp, vp, i32, vp, vp, f32, i32, i32, vp, sz, vp]
    lib.hsa_kv4_abi_sizes.argtypes = [P(ctypes.c_int64)] * 2
    lib.hsa_kv4_abi_sizes.restype = None
    for f in ("hsa_kv4_write", "hsa_kv4_read", "dense_decode_kv4", "dense_prefill_kv4"):
        getattr(lib, f).restype = ctypes.c_int
    for f in ("hsa_decode", "hsa_decode_host", "hsa_decode_step_create", "hsa_decode_step_run", "dense_decode",
              "hsa_build_from_codes", "hsa_append_encode", "hsa_read_error", "hsa_train_index"):
        getattr(lib, f).restype = ctypes.c_int
    for f in ("hsa_decode_workspace_bytes", "hsa_decode_host_workspace_bytes", "dense_decode_workspace_bytes",
              "hsa_index_workspace_bytes", "hsa_train_workspace_bytes"):
        getattr(lib, f).restype = sz
    lib.hsa_strerror.restype = ctypes.c_char_p
    lib.hsa_abi_sizes.restype = None
    sizes = [ctypes.c_int64() for _ in range(4)]
    lib.hsa_abi_sizes(*[ctypes.byref(s) for s in sizes])
    mine = [ctypes.sizeof(t) for t in (_KV, _Index, _Params, _Debug)]
    if [s.value for s in sizes] != mine:
        raise RuntimeError(f"ABI struct size mismatch: library {[s.value for s in sizes]} vs binding {mine}")
    lib.hsa_kv4_abi_sizes(ctypes.byref(sizes[0]), ctypes.byref(sizes[1]))
    if [s.value for s in sizes[:2]] != [ctypes.sizeof(_KV4), ctypes.sizeof(_KV4Rows)]:
        raise RuntimeError(f"ABI struct size mismatch of the kv4 structs: library {[s.value for s in sizes[:2]]}")
    if path == _build.LIB_PATH or "PQHSA_LIB" in os.environ:
        _lib = lib
    return lib


def hsa_strerror(status: int) -> str:
    return load_library().hsa_strerror(int(status)).decode()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _on_gpu(*ts: Optional[torch.Tensor]) -> None:
    """The library dereferences these on the device: a host tensor here would be a bad address."""
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("expected a CUDA tensor, got one on " + str(t.device))


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn: str, status: int):
    if status != 0:
        raise HSAError(fn, status)


@dataclass
class PagedKV:
    """Paged bf16 KV cache [num_pages][Hkv][page_size][D] plus the block table and lengths."""

    k_cache: torch.Tensor
    v_cache: torch.Tensor
    block_table: torch.Tensor      # int32 [B, max_pages] (device)
    seq_lens: torch.Tensor         # int32 [B] (device)
    seq_lens_host: torch.Tensor    # int32 [B] (cpu)
    Hq: int

    def struct(self) -> _KV:
        P, Hkv, ps, D = self.k_cache.shape
        B, maxp = self.block_table.shape
        assert self.k_cache.dtype == torch.bfloat16 and self.v_cache.dtype == torch.bfloat16
        assert self.block_table.dtype == torch.int32 and self.seq_lens.dtype == torch.int32
        assert self.seq_lens_host.dtype == torch.int32 and self.seq_lens_host.device.type == "cpu"
        assert self.k_cache.is_contiguous() and self.v_cache.is_contiguous() and self.block_table.is_contiguous()
        _on_gpu(self.k_cache, self.v_cache, self.block_table, self.seq_lens)
        return _KV(_ptr(self.k_cache), _ptr(self.v_cache), _ptr(self.block_table), _ptr(self.seq_lens),
                   _ptr(self.seq_lens_host), B, self.Hq, Hkv, D, ps, maxp, P)

    @property
    def B(self) -> int:
        return self.block_table.shape[0]

    @property
    def Hkv(self) -> int:
        return self.k_cache.shape[1]


@dataclass
class PQIndex:
    """Per-(sequence, KV head) IVF-PQ index storage (caller-owned device tensors)."""

    centroids: torch.Tensor        # fp32 [B, Hkv, C, D]
    codebooks: torch.Tensor        # fp32 [B, Hkv, M, 256, 8]
    codes: torch.Tensor            # uint8 [B, Hkv, cap, M]
    ids: torch.Tensor              # int16 storage of u16 cluster ids [B, Hkv, cap]
    sum_v: torch.Tensor            # fp32 [B, Hkv, C, D]
    mean_v: torch.Tensor           # fp32 [B, Hkv, C, D]
    count: torch.Tensor            # int32 [B, Hkv, C]
    n_indexed: torch.Tensor        # int32 [B] (device)
    n_indexed_host: torch.Tensor   # int32 [B] (cpu)
    n_sink: int
    list_codes: Optional[torch.Tensor] = None     # uint8 [B, Hkv, list_slots, M]  (library-maintained)
    list_slot: Optional[torch.Tensor] = None      # int32 [B, Hkv, list_slots]
    chunk_cluster: Optional[torch.Tensor] = None  # int16 storage of u16 [B, Hkv, list_slots / 32]
    list_meta: Optional[torch.Tensor] = None      # int32 [B, Hkv, 2 + 2C]

    def __post_init__(self):
        if self.list_codes is None:
            B, Hkv, cap, _ = self.codes.shape
            C = self.centroids.shape[2]
            ls = index_list_slots(cap, C)
            dev = self.codes.device
            self.list_codes = torch.zeros(B, Hkv, ls, M_SUB, device=dev, dtype=torch.uint8)
            self.list_slot = torch.full((B, Hkv, ls), -1, device=dev, dtype=torch.int32)
            self.chunk_cluster = torch.zeros(B, Hkv, ls // 32, device=dev, dtype=torch.int16)
            self.list_meta = torch.zeros(B, Hkv, 2 + 2 * C, device=dev, dtype=torch.int32)

    @staticmethod
    def allocate(B: int, Hkv: int, C: int, cap: int, n_sink: int, device) -> "PQIndex":
        f = dict(device=device, dtype=torch.float32)
        return PQIndex(
            centroids=torch.zeros(B, Hkv, C, HEAD_DIM, **f),
            codebooks=torch.zeros(B, Hkv, M_SUB, NCODE, DSUB, **f),
            codes=torch.zeros(B, Hkv, cap, M_SUB, device=device, dtype=torch.uint8),
            ids=torch.zeros(B, Hkv, cap, device=device, dtype=torch.int16),
            sum_v=torch.zeros(B, Hkv, C, HEAD_DIM, **f),
            mean_v=torch.zeros(B, Hkv, C, HEAD_DIM, **f),
            count=torch.zeros(B, Hkv, C, device=device, dtype=torch.int32),
            n_indexed=torch.zeros(B, device=device, dtype=torch.int32),
            n_indexed_host=torch.zeros(B, dtype=torch.int32),
            n_sink=n_sink,
        )

    @property
    def C(self) -> int:
        return self.centroids.shape[2]

    @property
    def cap(self) -> int:
        return self.codes.shape[2]

    def struct(self) -> _Index:
        for t in (self.centroids, self.codebooks, self.codes, self.ids, self.sum_v, self.mean_v, self.count,
                  self.list_codes, self.list_slot, self.chunk_cluster, self.list_meta):
            assert t.is_contiguous()
        assert self.n_indexed_host.device.type == "cpu" and self.n_indexed_host.dtype == torch.int32
        _on_gpu(self.centroids, self.codebooks, self.codes, self.ids, self.sum_v, self.mean_v, self.count,
                self.n_indexed, self.list_codes, self.list_slot, self.chunk_cluster, self.list_meta)
        return _Index(_ptr(self.centroids), _ptr(self.codebooks), _ptr(self.codes), _ptr(self.ids),
                      _ptr(self.sum_v), _ptr(self.mean_v), _ptr(self.count), _ptr(self.n_indexed),
                      _ptr(self.n_indexed_host), _ptr(self.list_codes), _ptr(self.list_slot),
                      _ptr(self.chunk_cluster), _ptr(self.list_meta), self.C, M_SUB, DSUB, NCODE, self.cap,
                      self.n_sink, self.list_codes.shape[2])


def hsa_decode_workspace_bytes(kv: PagedKV, index: PQIndex) -> int:
    kvs, ixs = kv.struct(), index.struct()
    n = load_library().hsa_decode_workspace_bytes(ctypes.byref(kvs), ctypes.byref(ixs))
    if n == 0:
        raise HSAError("hsa_decode_workspace_bytes", 1)
    return int(n)


def hsa_decode_host_workspace_bytes(kv: PagedKV, index: PQIndex) -> int:
    kvs, ixs = kv.struct(), index.struct()
    n = load_library().hsa_decode_host_workspace_bytes(ctypes.byref(kvs), ctypes.byref(ixs))
    if n == 0:
        raise HSAError("hsa_decode_host_workspace_bytes", 1)
    return int(n)


def _check_host_io(t: torch.Tensor, shape, name: str) -> None:
    """hsa_decode_host reads and writes these on the host (pinned memory keeps the copies
    asynchronous)."""
    if t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected a contiguous fp32 host tensor {list(shape)}")


def dense_decode_workspace_bytes(kv: PagedKV) -> int:
    kvs = kv.struct()
    n = load_library().dense_decode_workspace_bytes(ctypes.byref(kvs))
    if n == 0:
        raise HSAError("dense_decode_workspace_bytes", 1)
    return int(n)


def hsa_index_workspace_bytes(kv: PagedKV, index: PQIndex, n_new: int = 0) -> int:
    """Workspace of hsa_append_encode(kv, index, n_new) (n_new = 0: of hsa_build_from_codes)."""
    kvs, ixs = kv.struct(), index.struct()
    return int(load_library().hsa_index_workspace_bytes(ctypes.byref(kvs), ctypes.byref(ixs), int(n_new)))


def workspace(nbytes: int, device) -> torch.Tensor:
    """A zeroed workspace buffer (torch allocations are 256-byte aligned)."""
    return torch.zeros(max(256, (nbytes + 255) // 256 * 256), dtype=torch.uint8, device=device)


def hsa_decode(kv: PagedKV, index: PQIndex, q: torch.Tensor, out: Optional[torch.Tensor] = None, *,
               scale: float, budget: float = 0.01, k_override: int = -1, background: bool = True,
               approx_logits: Optional[torch.Tensor] = None, selected: Optional[torch.Tensor] = None,
               n_selected: Optional[torch.Tensor] = None, workspace_buf: Optional[torch.Tensor] = None,
               stage_events=None, stream=None) -> torch.Tensor:
    """One PQ-HSA decode step (see hsa_decode in include/pqhsa.h). q, out: fp32 [B, Hq, D]."""
    assert q.dtype == torch.float32 and q.is_contiguous()
    if out is None:
        out = torch.empty_like(q)
    kvs, ixs = kv.struct(), index.struct()
    lib = load_library()
    if workspace_buf is None:
        workspace_buf = workspace(hsa_decode_workspace_bytes(kv, index), q.device)
    prm = _Params(float(scale), float(budget), int(k_override), 1 if background else 0)
    ev_arr = None
    if stage_events is not None:
        assert len(stage_events) == NUM_STAGES + 1
        ev_arr = (ctypes.c_void_p * (NUM_STAGES + 1))(*[e.cuda_event for e in stage_events])
    _on_gpu(q, out, approx_logits, selected, n_selected, workspace_buf)
    dbg = _Debug(_ptr(approx_logits), _ptr(selected), _ptr(n_selected),
                 ctypes.cast(ev_arr, ctypes.c_void_p) if ev_arr is not None else None)
    st = lib.hsa_decode(ctypes.byref(kvs), ctypes.byref(ixs), q.data_ptr(), out.data_ptr(), ctypes.byref(prm),
                        ctypes.byref(dbg), workspace_buf.data_ptr(), workspace_buf.numel(), _stream(stream))
    _check("hsa_decode", st)
    return out


class DecodeStep:
    """hsa_decode prepared for one cache, index and workspace, for a decode loop: the C-ABI
    views of the cache and the index, the parameters and the workspace are checked and
    marshalled once here, and each call passes only q, out and the stream (the library still
    validates every call, lengths included). The tensors must keep their storage while the
    step is in use; their contents (lengths, appended tokens, lists) may change between calls.
    Calling the step runs it on device q / out: by default as one hsa_decode call, or with
    graph=True as the library's prepared step (hsa_decode_step_run: one CUDA graph launch per
    call while the split plan and the buffers stay the same - worth it when a loop reuses
    the same q and out tensors). .host() runs it on page-locked host q / out: by default as
    the prepared step, or with graph=False as one hsa_decode_host call. The workspace is
    sized for all of them.
    """

    def __init__(self, kv: PagedKV, index: PQIndex, *, scale: float, budget: float = 0.01, k_override: int = -1,
                 background: bool = True, workspace_buf: Optional[torch.Tensor] = None):
        self.kv, self.index = kv, index          # keep the tensors behind the views alive
        self._kvs, self._ixs = kv.struct(), index.struct()
        if workspace_buf is None:
            workspace_buf = workspace(hsa_decode_host_workspace_bytes(kv, index), kv.k_cache.device)
        _on_gpu(workspace_buf)
        self.workspace_buf = workspace_buf
        self._prm = _Params(float(scale), float(budget), int(k_override), 1 if background else 0)
        self._shape = (kv.B, kv.Hq, kv.k_cache.shape[3])
        self._device = kv.k_cache.device
        self._fn = load_library().hsa_decode
        self._fn_host = load_library().hsa_decode_host
        self._kv_ref, self._ix_ref = ctypes.byref(self._kvs), ctypes.byref(self._ixs)
        self._prm_ref = ctypes.byref(self._prm)
        self._ws_ptr, self._ws_len = workspace_buf.data_ptr(), workspace_buf.numel()
        self._lib = load_library()
        self._handle = ctypes.c_void_p(None)
        self._host_ok = None   # (q_host, out_host, their data pointers) last checked

    def _check_io(self, t: torch.Tensor, name: str) -> None:
        if (t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != self._shape
                or t.device != self._device):
            raise ValueError(f"{name}: expected a contiguous fp32 tensor {list(self._shape)} on {self._device}")

    def __call__(self, q: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None,
                 graph: bool = False) -> torch.Tensor:
        self._check_io(q, "q")
        if out is None:
            out = torch.empty_like(q)
        else:
            self._check_io(out, "out")
        if graph:
            self._run_step(q, out, stream)
            return out
        st = self._fn(self._kv_ref, self._ix_ref, q.data_ptr(), out.data_ptr(), self._prm_ref, None, self._ws_ptr,
                      self._ws_len, _stream(stream))
        _check("hsa_decode", st)
        return out

    def _run_step(self, q: torch.Tensor, out: torch.Tensor, stream) -> None:
        if not self._handle.value:
            _check("hsa_decode_step_create",
                   self._lib.hsa_decode_step_create(self._kv_ref, self._ix_ref, self._prm_ref, self._ws_ptr,
                                                    self._ws_len, ctypes.byref(self._handle)))
        _check("hsa_decode_step_run",
               self._lib.hsa_decode_step_run(self._handle, q.data_ptr(), out.data_ptr(), _stream(stream)))

    def host(self, q_host: torch.Tensor, out_host: torch.Tensor, stream=None, graph: bool = True) -> torch.Tensor:
        """q in from and out back to host memory, queued on the stream (out_host holds the result
        once the stream has reached it). A decode loop passes the same two buffers every step:
        they are checked once, and again whenever another tensor or storage comes in."""
        ok = self._host_ok
        if (ok is None or ok[0] is not q_host or ok[1] is not out_host or ok[2] != q_host.data_ptr()
                or ok[3] != out_host.data_ptr()):
            _check_host_io(q_host, self._shape, "q_host")
            _check_host_io(out_host, self._shape, "out_host")
            self._host_ok = (q_host, out_host, q_host.data_ptr(), out_host.data_ptr())
        if not graph:
            st = self._fn_host(self._kv_ref, self._ix_ref, q_host.data_ptr(), out_host.data_ptr(), self._prm_ref,
                               self._ws_ptr, self._ws_len, _stream(stream))
            _check("hsa_decode_host", st)
            return out_host
        self._run_step(q_host, out_host, stream)
        return out_host

    def close(self) -> None:
        """Release the library's prepared step (after its queued work has finished)."""
        if getattr(self, "_handle", None) is not None and self._handle.value:
            self._lib.hsa_decode_step_destroy(self._handle)
            self._handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def hsa_decode_host(kv: PagedKV, index: PQIndex, q_host: torch.Tensor, out_host: torch.Tensor, *, scale: float,
                    budget: float = 0.01, k_override: int = -1, background: bool = True,
                    workspace_buf: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """hsa_decode with q and out in host memory (see hsa_decode_host in include/pqhsa.h).
    Queued on the stream: out_host holds the result once the stream has reached it."""
    shape = (kv.B, kv.Hq, kv.k_cache.shape[3])
    _check_host_io(q_host, shape, "q_host")
    _check_host_io(out_host, shape, "out_host")
    kvs, ixs = kv.struct(), index.struct()
    if workspace_buf is None:
        workspace_buf = workspace(hsa_decode_host_workspace_bytes(kv, index), kv.k_cache.device)
    _on_gpu(workspace_buf)
    prm = _Params(float(scale), float(budget), int(k_override), 1 if background else 0)
    st = load_library().hsa_decode_host(ctypes.byref(kvs), ctypes.byref(ixs), q_host.data_ptr(), out_host.data_ptr(),
                                        ctypes.byref(prm), workspace_buf.data_ptr(), workspace_buf.numel(),
                                        _stream(stream))
    _check("hsa_decode_host", st)
    return out_host


def selected_counts(kv: PagedKV, index: PQIndex, q: torch.Tensor, *, scale: float, budget: float = 0.01,
                    k_override: int = -1, background: bool = True,
                    workspace_buf: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Selected tokens per (sequence, KV head) as hsa_decode reports them: int32 [B, Hkv] on the
    host, from one decode step with the n_selected debug output (synchronises the stream)."""
    n_sel = torch.full((kv.B, kv.Hkv), -1, dtype=torch.int32, device=q.device)
    hsa_decode(kv, index, q, scale=scale, budget=budget, k_override=k_override, background=background,
               n_selected=n_sel, workspace_buf=workspace_buf)
    return n_sel.cpu()


def dense_decode(kv: PagedKV, q: torch.Tensor, out: Optional[torch.Tensor] = None, *, scale: float,
                 workspace_buf: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Dense split-K GQA decode over every token (see dense_decode in include/pqhsa.h)."""
    assert q.dtype == torch.float32 and q.is_contiguous()
    if out is None:
        out = torch.empty_like(q)
    kvs = kv.struct()
    if workspace_buf is None:
        workspace_buf = workspace(dense_decode_workspace_bytes(kv), q.device)
    _on_gpu(q, out, workspace_buf)
    st = load_library().dense_decode(ctypes.byref(kvs), q.data_ptr(), out.data_ptr(), ctypes.c_float(scale),
                                     workspace_buf.data_ptr(), workspace_buf.numel(), _stream(stream))
    _check("dense_decode", st)
    return out


def hsa_build_from_codes(kv: PagedKV, index: PQIndex, workspace_buf: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """count / sum_v / mean_v of every cluster from the caller's codes and ids."""
    kvs, ixs = kv.struct(), index.struct()
    if workspace_buf is None:
        workspace_buf = workspace(hsa_index_workspace_bytes(kv, index), index.centroids.device)
    _on_gpu(workspace_buf)
    st = load_library().hsa_build_from_codes(ctypes.byref(kvs), ctypes.byref(ixs), workspace_buf.data_ptr(),
                                             workspace_buf.numel(), _stream(stream))
    _check("hsa_build_from_codes", st)


def hsa_append_encode(kv: PagedKV, index: PQIndex, n_new: int, workspace_buf: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    """Encode the next n_new tokens of every sequence into the index (advances n_indexed)."""
    kvs, ixs = kv.struct(), index.struct()
    if workspace_buf is None:
        workspace_buf = workspace(hsa_index_workspace_bytes(kv, index, n_new), index.centroids.device)
    _on_gpu(workspace_buf)
    st = load_library().hsa_append_encode(ctypes.byref(kvs), ctypes.byref(ixs), int(n_new),
                                          workspace_buf.data_ptr(), workspace_buf.numel(), _stream(stream))
    _check("hsa_append_encode", st)


def hsa_train_workspace_bytes(kv: PagedKV, index: PQIndex, n_train: int) -> int:
    kvs, ixs = kv.struct(), index.struct()
    n = load_library().hsa_train_workspace_bytes(ctypes.byref(kvs), ctypes.byref(ixs), int(n_train))
    if n == 0:
        raise HSAError("hsa_train_workspace_bytes", 1)
    return int(n)


def hsa_train_index(kv: PagedKV, index: PQIndex, n_train: int, init_slots: torch.Tensor, *,
                    coarse_iters: int = 8, pq_iters: int = 8, assign_out: Optional[torch.Tensor] = None,
                    workspace_buf: Optional[torch.Tensor] = None, stream=None) -> None:
    """Train index.centroids / index.codebooks by Lloyd k-means on the keys at positions
    [n_sink, n_sink + n_train) (see hsa_train_index in include/pqhsa.h).
    init_slots: int32 [B, Hkv, C + 16 * 256] training slots seeding the centroids, then the codewords."""
    assert init_slots.dtype == torch.int32 and init_slots.is_contiguous()
    if assign_out is not None:
        assert assign_out.dtype == torch.int32 and assign_out.is_contiguous()
    kvs, ixs = kv.struct(), index.struct()
    if workspace_buf is None:
        workspace_buf = workspace(hsa_train_workspace_bytes(kv, index, n_train), index.centroids.device)
    _on_gpu(init_slots, assign_out, workspace_buf)
    st = load_library().hsa_train_index(ctypes.byref(kvs), ctypes.byref(ixs), int(n_train), init_slots.data_ptr(),
                                        int(coarse_iters), int(pq_iters), _ptr(assign_out),
                                        workspace_buf.data_ptr(), workspace_buf.numel(), _stream(stream))
    _check("hsa_train_index", st)


def hsa_read_error(workspace_buf: torch.Tensor, stream=None) -> int:
    """Read and clear the device error word of a workspace (synchronises the stream)."""
    v = ctypes.c_int32(0)
    _on_gpu(workspace_buf)
    st = load_library().hsa_read_error(workspace_buf.data_ptr(), ctypes.byref(v), _stream(stream))
    _check("hsa_read_error", st)
    return int(v.value)


def dense_decode_static(kv: PagedKV, q: torch.Tensor, out: Optional[torch.Tensor] = None, *, scale: float,
                        stream=None) -> torch.Tensor:
    """dense_decode with the library's static scratch array: no workspace, no allocation in the
    library (see dense_decode_static in include/pqhsa.h for its limit and its sharing rules)."""
    assert q.dtype == torch.float32 and q.is_contiguous()
    if out is None:
        out = torch.empty_like(q)
    lib = load_library()
    fn = lib.dense_decode_static
    fn.argtypes = [ctypes.POINTER(_KV), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p]
    fn.restype = ctypes.c_int
    kvs = kv.struct()
    _on_gpu(q, out)
    _check("dense_decode_static", fn(ctypes.byref(kvs), q.data_ptr(), out.data_ptr(), ctypes.c_float(scale),
                                     _stream(stream)))
    return out


# ---- 4-bit KV cache ------------------------------------------------------------------------

_KV4_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


@dataclass(frozen=True, eq=False)
class KV4Cache:
    """Paged KV cache held in 4 bits (number format and tile layout: include/pqhsa.h), with the block
    table and lengths: 144 bytes a token and KV head. The views are checked and marshalled once,
    here, as DecodeStep does it; the tensors' contents (lengths too) may change between calls.
    KV4Cache.empty() allocates the pages."""

    cache: torch.Tensor            # uint8 [num_pages, Hkv, page_size / 16, KV4_TILE_BYTES] (device)
    block_table: torch.Tensor      # int32 [B, max_pages] (device)
    seq_lens: torch.Tensor         # int32 [B] (device)
    seq_lens_host: torch.Tensor    # int32 [B] (cpu)
    Hq: int

    def __post_init__(self):
        c, bt = self.cache, self.block_table
        _need(c.dtype == torch.uint8 and c.dim() == 4 and c.is_contiguous() and c.shape[3] == KV4_TILE_BYTES,
              f"cache: expected a contiguous uint8 tensor [pages, Hkv, page_size / 16, {KV4_TILE_BYTES}]")
        _need(bt.dtype == torch.int32 and bt.dim() == 2 and bt.is_contiguous(),
              "block_table: expected a contiguous int32 tensor [B, max_pages]")
        B = bt.shape[0]
        for t, name in ((self.seq_lens, "seq_lens"), (self.seq_lens_host, "seq_lens_host")):
            _need(t.dtype == torch.int32 and t.is_contiguous() and tuple(t.shape) == (B,),
                  f"{name}: expected a contiguous int32 tensor [{B}]")
        _need(self.seq_lens_host.device.type == "cpu", "seq_lens_host: expected a host tensor")
        _on_gpu(c, bt, self.seq_lens)
        _need(bt.device == c.device and self.seq_lens.device == c.device, "the cache's tensors are on different devices")
        s = _KV4(_ptr(c), _ptr(bt), _ptr(self.seq_lens), _ptr(self.seq_lens_host), B, self.Hq, c.shape[1], HEAD_DIM,
                 c.shape[2] * KV4_TILE_TOKENS, bt.shape[1], c.shape[0])
        object.__setattr__(self, "_struct", s)
        object.__setattr__(self, "_ref", ctypes.byref(s))
        object.__setattr__(self, "_index", c.device.index)
        object.__setattr__(self, "_row_shape", (c.shape[1], HEAD_DIM))
        object.__setattr__(self, "_per_seq", (B,))
        object.__setattr__(self, "_offsets", (B + 1,))

    @staticmethod
    def empty(num_pages: int, Hkv: int, page_size: int, device) -> torch.Tensor:
        """Pages for the `cache` field; their contents need no initialisation."""
        _need(page_size % KV4_TILE_TOKENS == 0, f"page_size: a multiple of {KV4_TILE_TOKENS}")
        return torch.empty(num_pages, Hkv, page_size // KV4_TILE_TOKENS, KV4_TILE_BYTES, dtype=torch.uint8,
                           device=device)

    @property
    def B(self) -> int:
        return self.block_table.shape[0]

    @property
    def Hkv(self) -> int:
        return self.cache.shape[1]

    @property
    def page_size(self) -> int:
        return self.cache.shape[2] * KV4_TILE_TOKENS

    def struct(self) -> _KV4:
        return self._struct


def hsa_kv4_workspace_bytes(kv: KV4Cache) -> int:
    """Workspace of any kv4 call on this cache."""
    n = load_library().hsa_kv4_workspace_bytes(kv._ref)
    if n == 0:
        raise HSAError("hsa_kv4_workspace_bytes", 1)
    return int(n)


def _kv4_on(kv: KV4Cache, *ts) -> None:
    for t in ts:
        if t is not None and t.device != kv.cache.device:
            raise ValueError(f"expected a tensor on {kv.cache.device}, got one on {t.device}")


def _kv4_new(kv: KV4Cache, stream, make):
    """make() with its allocation (and whatever fills it) on the device and stream of the call."""
    if stream is None:
        return make()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=kv.cache.device)
    with torch.cuda.stream(stream):
        return make()


def _kv4_workspace(kv: KV4Cache, workspace_buf, stream) -> torch.Tensor:
    if workspace_buf is None:
        n = hsa_kv4_workspace_bytes(kv)
        return _kv4_new(kv, stream, lambda: workspace(n, kv.cache.device))
    _kv4_on(kv, workspace_buf)
    _need(workspace_buf.is_contiguous(), "workspace_buf: expected a contiguous tensor")
    return workspace_buf


def _kv4_call(kv: KV4Cache, name: str, args, workspace_buf, stream) -> None:
    """One library call on the cache's device (the current one or not) and the given or current stream."""
    if torch.cuda.current_device() != kv._index:
        with torch.cuda.device(kv._index):
            return _kv4_call(kv, name, args, workspace_buf, stream)
    ws = _kv4_workspace(kv, workspace_buf, stream)
    # the current stream as a handle: building the Stream object takes longer than the rest of a short call
    raw = torch._C._cuda_getCurrentRawStream(kv._index) if stream is None else _stream(stream)
    st = getattr(load_library(), name)(kv._ref, *args, ws.data_ptr(), ws.numel() * ws.element_size(), raw)
    if st != 0:
        raise HSAError(name, st)


def _kv4_rows(kv: KV4Cache, t: torch.Tensor, name: str, n: int) -> _KV4Rows:
    strides = t.stride()
    if t.shape != (n,) + kv._row_shape or strides[2] != 1:
        raise ValueError(f"{name}: expected [{n}, {kv.Hkv}, {HEAD_DIM}] with contiguous rows")
    # between the rows of a dim of one: anything
    return _KV4Rows(t.data_ptr(), strides[0] if n > 1 else 0, strides[1] if kv._row_shape[0] > 1 else 0)


def _kv4_ints(kv: KV4Cache, t: torch.Tensor, host: torch.Tensor, shape, name: str) -> None:
    if (t.dtype != torch.int32 or host.dtype != torch.int32 or t.shape != shape or host.shape != shape
            or not t.is_contiguous() or not host.is_contiguous() or not host.is_cpu):
        raise ValueError(f"{name}: expected contiguous int32 tensors {list(shape)} on the device and on the host")
    _kv4_on(kv, t)


def _kv4_cu(kv: KV4Cache, cu: torch.Tensor, cu_host: torch.Tensor, name: str) -> int:
    """Checks the row offsets of the sequences; returns the rows of the call."""
    _kv4_ints(kv, cu, cu_host, kv._offsets, name)
    return ctypes.c_int32.from_address(cu_host.data_ptr() + 4 * (kv._offsets[0] - 1)).value


def _kv4_type(a: torch.Tensor, b: torch.Tensor) -> int:
    code = _KV4_TYPES.get(a.dtype)
    if code is None or b.dtype != a.dtype:
        raise ValueError("expected tensors of one type: float32, bfloat16 or float16")
    return code


def hsa_kv4_write(kv: KV4Cache, k: torch.Tensor, v: torch.Tensor, cu_new: torch.Tensor, cu_new_host: torch.Tensor, *,
                  workspace_buf: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantise new tokens into the cache (see hsa_kv4_write in include/pqhsa.h): sequence b's last tokens are
    rows [cu_new[b], cu_new[b + 1]) of k and v [rows, Hkv, 128], of any token and head strides (views of a
    fused projection need no copy). Set seq_lens and seq_lens_host to the lengths with them first."""
    n = _kv4_cu(kv, cu_new, cu_new_host, "cu_new")
    _kv4_on(kv, k, v)
    code = _kv4_type(k, v)
    if n == 0:
        return
    kr, vr = _kv4_rows(kv, k, "k", n), _kv4_rows(kv, v, "v", n)
    _kv4_call(kv, "hsa_kv4_write", (ctypes.byref(kr), ctypes.byref(vr), code, cu_new.data_ptr(),
                                    cu_new_host.data_ptr()), workspace_buf, stream)


def hsa_kv4_read(kv: KV4Cache, start: torch.Tensor, start_host: torch.Tensor, cu: torch.Tensor,
                 cu_host: torch.Tensor, *, dtype: torch.dtype = torch.bfloat16,
                 k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                 workspace_buf: Optional[torch.Tensor] = None, stream=None):
    """Read positions [start[b], start[b] + n_b) of every sequence back (see hsa_kv4_read in include/pqhsa.h) as
    rows [cu[b], cu[b + 1]) of two tensors [rows, Hkv, 128], new ones of `dtype` or the given ones."""
    n = _kv4_cu(kv, cu, cu_host, "cu")
    _kv4_ints(kv, start, start_host, kv._per_seq, "start")
    new = lambda: torch.empty(n, kv.Hkv, HEAD_DIM, dtype=dtype, device=kv.cache.device)  # noqa: E731
    if k_out is None:
        k_out = _kv4_new(kv, stream, new)
    if v_out is None:
        v_out = _kv4_new(kv, stream, new)
    _kv4_on(kv, k_out, v_out)
    code = _kv4_type(k_out, v_out)
    if n == 0:
        return k_out, v_out
    kr, vr = _kv4_rows(kv, k_out, "k_out", n), _kv4_rows(kv, v_out, "v_out", n)
    _kv4_call(kv, "hsa_kv4_read", (ctypes.byref(kr), ctypes.byref(vr), code, start.data_ptr(), start_host.data_ptr(),
                                   cu.data_ptr(), cu_host.data_ptr()), workspace_buf, stream)
    return k_out, v_out


def _kv4_window(window: int) -> int:
    """As an int32: more than any sequence has is all the same."""
    return max(-1, min(window, (1 << 31) - 1))


def _kv4_out(kv: KV4Cache, q: torch.Tensor, out: Optional[torch.Tensor], lse: Optional[torch.Tensor], stream):
    shape = q.shape
    if out is None:
        out = _kv4_new(kv, stream, lambda: torch.empty(shape, dtype=q.dtype, device=q.device))
    elif out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out: expected a contiguous tensor {list(shape)}")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != shape[:2] or not lse.is_contiguous()):
        raise ValueError(f"lse: expected a contiguous float32 tensor {list(shape[:2])}")
    _kv4_on(kv, q, out, lse)
    return out


def dense_decode_kv4(kv: KV4Cache, q: torch.Tensor, out: Optional[torch.Tensor] = None, *, scale: float,
                     window: int = 0, lse: Optional[torch.Tensor] = None,
                     workspace_buf: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of one query token a sequence over a 4-bit cache (see dense_decode_kv4 in include/pqhsa.h).
    q, out: [B, Hq, 128] in float32, bfloat16 or float16; lse: float32 [B, Hq], filled if given."""
    if tuple(q.shape) != (kv.B, kv.Hq, HEAD_DIM) or not q.is_contiguous():
        raise ValueError(f"q: expected a contiguous tensor [{kv.B}, {kv.Hq}, {HEAD_DIM}]")
    out = _kv4_out(kv, q, out, lse, stream)
    _kv4_call(kv, "dense_decode_kv4", (q.data_ptr(), out.data_ptr(), _ptr(lse), _kv4_type(q, out), scale,
                                       _kv4_window(window)),
              workspace_buf, stream)
    return out


def dense_prefill_kv4(kv: KV4Cache, q: torch.Tensor, cu_q: torch.Tensor, cu_q_host: torch.Tensor,
                      out: Optional[torch.Tensor] = None, *, scale: float, causal: bool = True, window: int = 0,
                      lse: Optional[torch.Tensor] = None, workspace_buf: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Attention of the last tokens of every sequence over a 4-bit cache that holds them already (see
    dense_prefill_kv4 in include/pqhsa.h): chunks of prompts, drafted tokens to verify. q: [rows, Hq, 128] of any
    token stride, rows [cu_q[b], cu_q[b + 1]) of sequence b; out: the same shape, contiguous."""
    n = _kv4_cu(kv, cu_q, cu_q_host, "cu_q")
    if tuple(q.shape) != (n, kv.Hq, HEAD_DIM) or (n and (q.stride(2) != 1 or (kv.Hq > 1 and q.stride(1) != HEAD_DIM))):
        raise ValueError(f"q: expected [{n}, {kv.Hq}, {HEAD_DIM}] with contiguous heads")
    out = _kv4_out(kv, q, out, lse, stream)
    code = _kv4_type(q, out)
    if n == 0:
        return out
    stride = q.stride(0) if n > 1 else kv.Hq * HEAD_DIM    # of a single row: anything
    _kv4_call(kv, "dense_prefill_kv4", (q.data_ptr(), stride, out.data_ptr(), _ptr(lse), code, cu_q.data_ptr(),
                                        cu_q_host.data_ptr(), scale, 1 if causal else 0, _kv4_window(window)),
              workspace_buf, stream)
    return out
