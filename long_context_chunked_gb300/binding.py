"""ctypes binding of ``libcpattn.so`` (declared in include/cpattn.h).

Argument marshalling only: every step of the hot path runs in the CUDA
kernels of the library.  There is no fallback -- if the library is missing
or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
# CPATTN_LIBRARY overrides the library path (e.g. an instrumented build).
LIB_PATH = os.environ.get("CPATTN_LIBRARY") or os.path.join(_PKG, "libcpattn.so")

OK, E_INVALID, E_UNSUPPORTED, E_CUDA, E_NOMEM, E_TIMEOUT, E_RANGE, E_PAGE = range(8)
MAX_SEQS = 128
MAX_ROW_BLOCKS = 2048
MAX_PAGED_SEQS = 4096
PAGE_SIZES = (16, 32, 64, 128, 256)
PAGES_BF16, PAGES_E4M3, PAGES_E2M1 = 0, 1, 4  # CPATTN_PAGES_*
GROUP4 = 32  # values of an e2m1 row that share a scale

# Every symbol include/cpattn.h declares.
EXPORTS = ("cpattn_create", "cpattn_write_kv", "cpattn_prefill", "cpattn_sync_status",
           "cpattn_set_fault_injection", "cpattn_cache_walk", "cpattn_destroy",
           "cpattn_status_string", "cpattn_last_error", "cpattn_prefill_noalloc",
           "cpattn_two_launch_workspace", "cpattn_prefill_two_launch", "cpattn_set_splitkv",
           "cpattn_splitkv_workspace", "cpattn_cache_walk_from", "cpattn_prefill_write_kv",
           "cpattn_set_barrier_counts", "cpattn_set_v_staging", "cpattn_v_staging_bytes",
           "cpattn_prefill_packed", "cpattn_prefill_packed_workspace", "cpattn_paged_write_kv",
           "cpattn_paged_read_kv", "cpattn_paged_decode", "cpattn_paged_decode_workspace",
           "cpattn_paged_write_planned_kv", "cpattn_paged_plan", "cpattn_paged_trim", "cpattn_rope_steps", "cpattn_norm_rope",
           "cpattn_norm_rope_write_kv")

# cpattn_config.pairing values, by name.
PAIRING = {"mma2": 0, "none": 1, "pingpong": 2}
COUNT_BARS = 40      # CPATTN_COUNT_BARS
COUNT_RECORD = 200   # CPATTN_COUNT_RECORD: uint32 per CTA


class CpattnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"cpattn status {status}: {msg}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("num_shards", ctypes.c_int32),
                ("shard_capacity", ctypes.c_int32), ("chunk_size", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("fast_p", ctypes.c_int32),
                ("v_cache_f16", ctypes.c_int32), ("pairing", ctypes.c_int32),
                ("gqa_packing", ctypes.c_int32)]


class Pages(ctypes.Structure):
    """cpattn_pages."""
    _fields_ = [("format", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("table_stride", ctypes.c_int64), ("k_pages", ctypes.c_void_p),
                ("v_pages", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("block_table", ctypes.c_void_p)]


class PagedKV:
    """A paged KV cache: pools [num_pages, NKV, page_size, HD] of bf16, or of
    torch.float8_e4m3fn with fp32 scales [num_pages, NKV, page_size], or 4-bit
    pools [num_pages, NKV, page_size, HD // 2] of uint8 (two e2m1 values each)
    with uint8 scale records [num_pages, NKV, page_size, 4 + HD // 32]; and the
    int32 block table [num_seqs, max_pages] (its rows may be a slice of a wider
    table).  Holds references to the tensors and checks them once; their
    contents are read by the kernels of each call."""

    def __init__(self, k_pages, v_pages, block_table, k_scales=None, v_scales=None):
        import torch
        formats = {torch.bfloat16: PAGES_BF16, torch.float8_e4m3fn: PAGES_E4M3, torch.uint8: PAGES_E2M1}
        if k_pages.dtype not in formats:
            raise ValueError(f"pages must be bfloat16, float8_e4m3fn or uint8 (e2m1), got {k_pages.dtype}")
        if k_pages.dim() != 4 or v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype:
            raise ValueError("k_pages and v_pages must be alike, [num_pages, NKV, page_size, HD]")
        fmt = formats[k_pages.dtype]
        if (k_scales is None) != (fmt == PAGES_BF16) or (v_scales is None) != (fmt == PAGES_BF16):
            raise ValueError("e4m3 and e2m1 pages need k_scales and v_scales, bf16 pages take none")
        dense = [k_pages, v_pages] + ([] if fmt == PAGES_BF16 else [k_scales, v_scales])
        hd = k_pages.shape[3] * (2 if fmt == PAGES_E2M1 else 1)
        for t in dense[2:]:
            if fmt == PAGES_E4M3 and (t.dtype != torch.float32 or t.shape != k_pages.shape[:3]):
                raise ValueError("scales must be float32 [num_pages, NKV, page_size]")
            if fmt == PAGES_E2M1 and (t.dtype != torch.uint8 or
                                      t.shape != (*k_pages.shape[:3], 4 + hd // GROUP4)):
                raise ValueError("scales must be uint8 [num_pages, NKV, page_size, 4 + HD // 32]")
        if block_table.dim() != 2 or block_table.dtype != torch.int32 or (
                block_table.shape[1] > 1 and block_table.stride(1) != 1) or (
                block_table.shape[0] > 1 and block_table.stride(0) < block_table.shape[1]):
            raise ValueError("block_table must be int32 [num_seqs, max_pages] with dense rows")
        if any(not t.is_contiguous() for t in dense):
            raise ValueError("pages and scales must be contiguous")
        if any(not t.is_cuda or t.device != k_pages.device for t in dense + [block_table]):
            raise ValueError("pages, scales and block_table must be on one CUDA device")
        self.k_pages, self.v_pages, self.block_table = k_pages, v_pages, block_table
        self.k_scales, self.v_scales = k_scales, v_scales
        self.device, self.i32 = k_pages.get_device(), torch.int32
        self.num_seqs, cols = block_table.shape
        self.num_kv_heads, self.head_dim = k_pages.shape[1], hd
        self.c = Pages(fmt, k_pages.shape[2], k_pages.shape[0], cols,
                       max(block_table.stride(0), cols), _ptr(k_pages), _ptr(v_pages),
                       _ptr(k_scales), _ptr(v_scales), _ptr(block_table))
        self.ref = ctypes.byref(self.c)


class NormRopeDesc(ctypes.Structure):
    """cpattn_norm_rope_desc."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("rope_steps", ctypes.c_void_p), ("weight_f32", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("eps", ctypes.c_float), ("rope_scale", ctypes.c_float)]


class NormRope:
    """Norm weights and rotation of a layer's query and key heads: inv_freq, the
    rotary_dim / 2 angles per position (host values, taken as float64; empty: no
    rotation), q_weight and k_weight [HD] of bf16 or fp32 on the GPU (None: no
    norm).  interleaved: pairs (2i, 2i + 1) instead of (i, i + rotary_dim / 2);
    scale: a factor of the rotated values.  Holds the tensors; a context's calls
    read them."""

    def __init__(self, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, scale: float = 1.0, device=None):
        import torch
        freq = np.ascontiguousarray(np.asarray(inv_freq, dtype=np.float64))
        if freq.ndim != 1 or freq.size % 4:
            raise ValueError("inv_freq must be a vector of rotary_dim / 2 values, rotary_dim a multiple of 8")
        steps = np.zeros(freq.size, dtype=np.uint64)
        if load().cpattn_rope_steps(freq.ctypes.data, freq.size, steps.ctypes.data) != OK:
            raise ValueError("inv_freq must be finite and within 2^20")
        weights = [w for w in (q_weight, k_weight) if w is not None]
        for w in weights:
            if w.dtype not in (torch.bfloat16, torch.float32) or w.dtype != weights[0].dtype or \
                    w.dim() != 1 or w.shape != weights[0].shape or not w.is_cuda or \
                    not w.is_contiguous() or w.device != weights[0].device:
                raise ValueError("weights must be alike, contiguous bfloat16 or float32 [HD] on one CUDA device")
        if device is None or torch.device(device) == torch.device("cuda"):
            device = weights[0].device if weights else torch.device("cuda", torch.cuda.current_device())
        self.steps = torch.from_numpy(steps.view(np.int64)).to(device) if freq.size else None
        self.q_weight, self.k_weight, self.rotary_dim = q_weight, k_weight, 2 * freq.size
        held = weights + ([self.steps] if freq.size else [])
        if any(w.device != held[0].device for w in held):
            raise ValueError("weights and device must be the same CUDA device")
        self.device = held[0].get_device() if held else torch.device(device).index
        self.head_dim = weights[0].numel() if weights else None
        self.types = torch.bfloat16, torch.int32  # of heads and of positions
        f32 = bool(weights) and weights[0].dtype is torch.float32
        self.c = NormRopeDesc(_ptr(q_weight), _ptr(k_weight), _ptr(self.steps), int(f32),
                              self.rotary_dim, int(bool(interleaved)), float(eps), float(scale))
        self.ref = ctypes.byref(self.c)


_libs = {}


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load a build of the library (once per path).  Raises if it has not
    been built."""
    if path in _libs:
        return _libs[path]
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library {path} is missing: build it with "
                           "long_context_chunked_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P, I32, U32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32
    I32P = ctypes.POINTER(ctypes.c_int32)
    lib.cpattn_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(P)]
    lib.cpattn_create.restype = I32
    lib.cpattn_write_kv.argtypes = [P, I32, I32P, I32P, P, P, P, P, P]
    lib.cpattn_write_kv.restype = I32
    lib.cpattn_prefill.argtypes = [P, I32, I32P, I32P, P, P, P, P, P, P, P, P]
    lib.cpattn_prefill.restype = I32
    lib.cpattn_sync_status.argtypes = [P, P]
    lib.cpattn_sync_status.restype = I32
    lib.cpattn_set_fault_injection.argtypes = [P, I32, I32]
    lib.cpattn_set_fault_injection.restype = I32
    lib.cpattn_cache_walk.argtypes = [P, I32, I32P, ctypes.POINTER(U32), I32, I32P]
    lib.cpattn_cache_walk.restype = I32
    lib.cpattn_destroy.argtypes = [P]
    lib.cpattn_destroy.restype = None
    lib.cpattn_status_string.argtypes = [I32]
    lib.cpattn_status_string.restype = ctypes.c_char_p
    lib.cpattn_last_error.argtypes = [P]
    lib.cpattn_last_error.restype = ctypes.c_char_p
    lib.cpattn_prefill_noalloc.argtypes = [ctypes.POINTER(Config), I32, I32P, I32P] + [P] * 8
    lib.cpattn_prefill_noalloc.restype = I32
    lib.cpattn_two_launch_workspace.argtypes = [P, I32, ctypes.POINTER(ctypes.c_uint64)]
    lib.cpattn_two_launch_workspace.restype = I32
    lib.cpattn_prefill_two_launch.argtypes = [P, I32, I32P, I32P] + [P] * 8 + [ctypes.c_uint64, P]
    lib.cpattn_prefill_two_launch.restype = I32
    lib.cpattn_set_splitkv.argtypes = [P, P, ctypes.c_uint64, I32]
    lib.cpattn_set_splitkv.restype = I32
    lib.cpattn_splitkv_workspace.argtypes = [P, I32, I32P, I32P, I32,
                                             ctypes.POINTER(ctypes.c_uint64), I32P]
    lib.cpattn_splitkv_workspace.restype = I32
    lib.cpattn_cache_walk_from.argtypes = [P, I32, I32, I32P, ctypes.POINTER(U32), I32, I32P]
    lib.cpattn_cache_walk_from.restype = I32
    lib.cpattn_prefill_write_kv.argtypes = [P, I32, I32P, I32P, P, P, P, P, P, P, P, P]
    lib.cpattn_prefill_write_kv.restype = I32
    lib.cpattn_set_barrier_counts.argtypes = [P, P, ctypes.c_uint64]
    lib.cpattn_set_barrier_counts.restype = I32
    if hasattr(lib, "cpattn_set_v_staging"):  # absent from older builds (A/B timing only)
        lib.cpattn_set_v_staging.argtypes = [P, P, ctypes.c_uint64]
        lib.cpattn_set_v_staging.restype = I32
        lib.cpattn_v_staging_bytes.argtypes = [P, I32, ctypes.POINTER(ctypes.c_uint64)]
        lib.cpattn_v_staging_bytes.restype = I32
    if hasattr(lib, "cpattn_paged_decode"):  # absent from older builds (A/B timing only)
        U64, PAGES = ctypes.c_uint64, ctypes.POINTER(Pages)
        for name, args in (
                ("cpattn_prefill_packed_workspace", [P, I32, I32P, ctypes.POINTER(U64)]),
                ("cpattn_prefill_packed", [P, I32, I32P, P, P, P, P, P, P, U64, P]),
                ("cpattn_paged_write_kv", [P, PAGES, I32, I32, P, P, P, P, P]),
                ("cpattn_paged_read_kv", [P, PAGES, I32, P, P, P, P, P]),
                ("cpattn_paged_decode_workspace", [P, I32, ctypes.POINTER(U64)]),
                ("cpattn_paged_decode", [P, PAGES, I32, P, P, P, P, P, U64, P])):
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = I32
    if hasattr(lib, "cpattn_paged_write_planned_kv"):
        lib.cpattn_paged_write_planned_kv.argtypes = [P, PAGES, I32, I32] + [P] * 6
        lib.cpattn_paged_write_planned_kv.restype = I32
    if hasattr(lib, "cpattn_paged_plan"):
        I64, NR = ctypes.c_int64, ctypes.POINTER(NormRopeDesc)
        for name, args in (
                ("cpattn_paged_plan", [P, PAGES, I32, I32] + [P] * 9),
                ("cpattn_paged_trim", [P, PAGES, I32] + [P] * 5),
                ("cpattn_rope_steps", [P, I32, P]),
                ("cpattn_norm_rope", [P, NR, I32, P] + [P, I64] * 4 + [P]),
                ("cpattn_norm_rope_write_kv", [P, NR, PAGES, I32, P, P] + [P, I64] * 4 + [P])):
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = I32
    _libs[path] = lib
    return lib


def _i32(values: Sequence[int]):
    arr = np.ascontiguousarray(np.asarray(values, dtype=np.int32))
    return arr, arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


def _ptr(t) -> int:
    """Device pointer of a tensor, or an int passed through; None -> NULL."""
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _want(name, t, dtype, shape, device: int):
    """A contiguous CUDA tensor of this dtype and shape, on CUDA device `device`."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or device < 0 \
            or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {list(shape)} on CUDA device "
                         f"{device}, got {t.dtype} {list(t.shape)} on {t.device}")


def _i32_ptrs(i32, names, device: int, *tensors_and_sizes):
    """Device pointers of contiguous int32 vectors on CUDA device `device`: tensor,
    size, tensor, size .. (each of `names`).  i32: torch.int32."""
    out = []
    sizes = iter(tensors_and_sizes)
    for t in sizes:
        n = next(sizes)
        if t.dtype is not i32 or t.numel() != n or t.dim() != 1 or t.get_device() != device \
                or not t.is_contiguous():
            _want(names.split()[len(out)], t, i32, (n,), device)
        out.append(t.data_ptr())
    return out


def _want_rows(name, t, rows: int, heads: int, hd: int, device: int, bf16) -> int:
    """The row stride of a bf16 CUDA tensor [rows, heads, hd] whose rows are dense."""
    if t.dtype is bf16 and t.shape == (rows, heads, hd) and t.get_device() == device >= 0:
        at, head, value = t.stride()
        if value == 1 and (head == hd or heads == 1) or rows == 0:
            return at if rows > 1 else heads * hd
    raise ValueError(f"{name}: expected a bfloat16 tensor [{rows}, {heads}, {hd}] with dense rows on "
                     f"CUDA device {device}, got {t.dtype} {list(t.shape)} on {t.device}")


def _workspace_bytes(workspace, device: int) -> int:
    if workspace.get_device() != device or device < 0 or not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous CUDA tensor on the inputs' device")
    return workspace.numel() * workspace.element_size()


def _stream_on(stream, device: int) -> int:
    """`stream`, or the current stream of CUDA device `device`."""
    if stream is None:
        import torch
        # (What torch.cuda.current_stream wraps in an object, at a tenth of the time.)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(device) if raw is not None else torch.cuda.current_stream(device).cuda_stream
    return _stream(stream)


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Context:
    """One attention-layer shape: NQ, NKV, HD, shard count P, shard capacity S, chunk C.
    pairing: "mma2" (default), "none" or "pingpong"; gqa_packing: False turns
    the packed short-chunk form off; library: the path of another build of the
    library (e.g. the barrier-count build) to run this context on."""

    def __init__(self, num_q_heads: int, num_kv_heads: int, head_dim: int, num_shards: int,
                 shard_capacity: int, chunk_size: int, softmax_scale: float = 0.0,
                 fast_p: bool = False, v_cache_f16: bool = False, pairing: str = "mma2",
                 gqa_packing: bool = True, library: Optional[str] = None):
        self.lib = load(library or LIB_PATH)
        self.cfg = Config(num_q_heads, num_kv_heads, head_dim, num_shards, shard_capacity,
                          chunk_size, softmax_scale, int(bool(fast_p)), int(bool(v_cache_f16)),
                          PAIRING[pairing], 0 if gqa_packing else 1)
        self.v_cache_f16 = bool(v_cache_f16)
        self.dims = (int(num_q_heads), int(num_kv_heads), int(head_dim))
        h = ctypes.c_void_p()
        st = self.lib.cpattn_create(ctypes.byref(self.cfg), ctypes.byref(h))
        if st != OK:
            raise CpattnError(st, self.lib.cpattn_status_string(st).decode())
        self._h = h

    @classmethod
    def for_workload(cls, w, fast_p: bool = False, v_cache_f16: bool = False,
                     pairing: str = "mma2", gqa_packing: bool = True,
                     library: Optional[str] = None) -> "Context":
        return cls(w.num_q_heads, w.num_kv_heads, w.head_dim, w.shards, w.shard_capacity,
                   w.chunk, w.scale, fast_p, v_cache_f16, pairing, gqa_packing, library)

    # -- status --------------------------------------------------------
    def _check(self, st: int):
        if st != OK:
            msg = self.lib.cpattn_last_error(self._h).decode() or \
                self.lib.cpattn_status_string(st).decode()
            raise CpattnError(st, msg)

    def status(self, st: int) -> int:
        return st

    # -- entry points --------------------------------------------------
    def write_kv_raw(self, cache_lens, chunk_lens, k_new, v_new, k_cache, v_cache, stream=None) -> int:
        cl, clp = _i32(cache_lens)
        ch, chp = _i32(chunk_lens)
        return self.lib.cpattn_write_kv(self._h, len(cl), clp, chp, _ptr(k_new), _ptr(v_new),
                                        _ptr(k_cache), _ptr(v_cache), _stream(stream))

    def write_kv(self, cache_lens, chunk_lens, k_new, v_new, k_cache, v_cache, stream=None):
        self._check_tensors((k_new, v_new, k_cache), v_cache)
        self._check(self.write_kv_raw(cache_lens, chunk_lens, k_new, v_new, k_cache, v_cache,
                                      stream))

    def prefill_raw(self, cache_lens, chunk_lens, q, k_new, v_new, k_cache, v_cache, out,
                    lse=None, stream=None) -> int:
        cl, clp = _i32(cache_lens)
        ch, chp = _i32(chunk_lens)
        return self.lib.cpattn_prefill(self._h, len(cl), clp, chp, _ptr(q), _ptr(k_new),
                                       _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(out),
                                       _ptr(lse), _stream(stream))

    def prefill(self, cache_lens, chunk_lens, q, k_new, v_new, k_cache, v_cache, out, lse=None,
                stream=None):
        self._check_tensors((q, k_new, v_new, k_cache, out), v_cache)
        self._check(self.prefill_raw(cache_lens, chunk_lens, q, k_new, v_new, k_cache, v_cache,
                                     out, lse, stream))

    def prefill_write_kv_raw(self, cache_lens, chunk_lens, q, k_new, v_new, k_cache, v_cache,
                             out, lse=None, stream=None) -> int:
        cl, clp = _i32(cache_lens)
        ch, chp = _i32(chunk_lens)
        return self.lib.cpattn_prefill_write_kv(
            self._h, len(cl), clp, chp, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
            _ptr(v_cache), _ptr(out), _ptr(lse), _stream(stream))

    def prefill_write_kv(self, cache_lens, chunk_lens, q, k_new, v_new, k_cache, v_cache, out,
                         lse=None, stream=None):
        """Prefill and the chunk's KV-cache write in one launch."""
        self._check_tensors((q, k_new, v_new, k_cache, out), v_cache)
        self._check(self.prefill_write_kv_raw(cache_lens, chunk_lens, q, k_new, v_new, k_cache,
                                              v_cache, out, lse, stream))

    def two_launch_workspace(self, num_seqs: int) -> int:
        n = ctypes.c_uint64()
        self._check(self.lib.cpattn_two_launch_workspace(self._h, num_seqs, ctypes.byref(n)))
        return n.value

    def prefill_two_launch(self, cache_lens, chunk_lens, q, k_new, v_new, k_cache, v_cache, out,
                           workspace, lse=None, stream=None):
        """The removed two-launch variant (cache-only + current-only + LSE merge)."""
        self._check_tensors((q, k_new, v_new, k_cache, out), v_cache)
        cl, clp = _i32(cache_lens)
        ch, chp = _i32(chunk_lens)
        nbytes = workspace.numel() * workspace.element_size()
        self._check(self.lib.cpattn_prefill_two_launch(
            self._h, len(cl), clp, chp, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
            _ptr(v_cache), _ptr(out), _ptr(lse), _ptr(workspace), nbytes, _stream(stream)))

    def set_splitkv(self, workspace=None, max_split_tiles: int = 0):
        """Register a device workspace (a CUDA tensor, 256-byte aligned) for
        split-KV, or None to turn it off; max_split_tiles 0 = automatic."""
        nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        self._check(self.lib.cpattn_set_splitkv(self._h, _ptr(workspace), nbytes,
                                                max_split_tiles))

    def splitkv_workspace(self, cache_lens, chunk_lens, max_split_tiles: int = 0):
        """(workspace bytes, work blocks) of this batch's split-KV plan."""
        cl, clp = _i32(cache_lens)
        ch, chp = _i32(chunk_lens)
        n = ctypes.c_uint64()
        blocks = ctypes.c_int32()
        self._check(self.lib.cpattn_splitkv_workspace(self._h, len(cl), clp, chp, max_split_tiles,
                                                      ctypes.byref(n), ctypes.byref(blocks)))
        return n.value, blocks.value

    def set_v_staging(self, buffer=None):
        """fp16 V cache: register a device buffer (a CUDA tensor, 16-byte
        aligned, v_staging_bytes(num_seqs) bytes for the largest batch) in
        which the prefill calls stage the chunk's V in fp16, or None to stop
        staging."""
        nbytes = 0 if buffer is None else buffer.numel() * buffer.element_size()
        self._check(self.lib.cpattn_set_v_staging(self._h, _ptr(buffer), nbytes))

    def v_staging_bytes(self, num_seqs: int) -> int:
        """Bytes of the V staging buffer for a batch of num_seqs sequences."""
        n = ctypes.c_uint64()
        self._check(self.lib.cpattn_v_staging_bytes(self._h, num_seqs, ctypes.byref(n)))
        return n.value

    # -- packed prompts and the paged cache ------------------------------
    def prefill_packed_workspace(self, seq_lens) -> int:
        """Workspace bytes of prefill_packed for these prompt lengths."""
        sl, slp = _i32(seq_lens)
        n = ctypes.c_uint64()
        self._check(self.lib.cpattn_prefill_packed_workspace(self._h, len(sl), slp,
                                                             ctypes.byref(n)))
        return n.value

    def prefill_packed(self, seq_lens, q, k, v, out, workspace, lse=None, stream=None):
        """Causal attention over whole prompts packed one behind the other:
        q, out [sum(seq_lens), NQ, HD], k, v [sum(seq_lens), NKV, HD], bf16.  A
        context made with v_cache_f16 takes V in fp16, with one P.V product
        instead of two."""
        import torch
        n = len(seq_lens)
        sl = (ctypes.c_int32 * n)(*[int(x) for x in seq_lens])
        rows, dev = sum(sl), q.get_device()
        nq, nkv, hd = self.dims
        _want("q", q, torch.bfloat16, (rows, nq, hd), dev)
        _want("k", k, torch.bfloat16, (rows, nkv, hd), dev)
        _want("v", v, torch.bfloat16, (rows, nkv, hd), dev)
        _want("out", out, torch.bfloat16, (rows, nq, hd), dev)
        if lse is not None:
            _want("lse", lse, torch.float32, (rows, nq), dev)
        self._check(self.lib.cpattn_prefill_packed(
            self._h, n, sl, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _ptr(lse),
            workspace.data_ptr(), _workspace_bytes(workspace, dev), _stream_on(stream, dev)))

    def paged_write_kv(self, pages: PagedKV, cache_lens, k_new, v_new, row_starts=None,
                       stream=None, lens=None):
        """Write (for e4m3 and e2m1 pages: quantise) new tokens into their pages: rows
        row_starts[b] .. row_starts[b + 1] - 1 of k_new and v_new [rows, NKV, HD]
        are the tokens of sequence b from cache_lens[b] on; row_starts None: one
        token per sequence.  lens: tokens from lens[b] on are left out -- after
        paged_plan give it the plan's lens (another tensor than cache_lens then), or
        sequences that the plan did not serve are written through whatever their rows
        of the table hold.  cache_lens, row_starts and lens: int32 CUDA tensors."""
        import torch
        self._check_pages(pages)
        b, dev, rows = pages.num_seqs, pages.device, k_new.shape[0]
        shape = (rows, pages.num_kv_heads, pages.head_dim)
        _want("k_new", k_new, torch.bfloat16, shape, dev)
        _want("v_new", v_new, torch.bfloat16, shape, dev)
        _want("cache_lens", cache_lens, torch.int32, (b,), dev)
        if row_starts is not None:
            _want("row_starts", row_starts, torch.int32, (b + 1,), dev)
        given = _ptr(row_starts), k_new.data_ptr(), v_new.data_ptr(), _stream_on(stream, dev)
        if lens is None:
            self._check(self.lib.cpattn_paged_write_kv(self._h, pages.ref, b, rows, cache_lens.data_ptr(), *given))
        else:
            _want("lens", lens, torch.int32, (b,), dev)
            self._check(self.lib.cpattn_paged_write_planned_kv(self._h, pages.ref, b, rows, cache_lens.data_ptr(),
                                                               lens.data_ptr(), *given))

    def paged_read_kv(self, pages: PagedKV, lens, k_cache, v_cache, first=None, stream=None):
        """Read tokens first[b] (None: 0) .. lens[b] - 1 back into the striped
        caches [num_seqs, NKV, P, S, HD] of the chunked prefill."""
        import torch
        self._check_pages(pages)
        c, b, dev = self.cfg, pages.num_seqs, pages.device
        shape = (b, pages.num_kv_heads, c.num_shards, c.shard_capacity, pages.head_dim)
        _want("k_cache", k_cache, torch.bfloat16, shape, dev)
        _want("v_cache", v_cache, torch.float16 if self.v_cache_f16 else torch.bfloat16, shape, dev)
        _want("lens", lens, torch.int32, (b,), dev)
        if first is not None:
            _want("first", first, torch.int32, (b,), dev)
        self._check(self.lib.cpattn_paged_read_kv(
            self._h, pages.ref, b, _ptr(first), lens.data_ptr(), k_cache.data_ptr(),
            v_cache.data_ptr(), _stream_on(stream, dev)))

    def paged_decode_workspace(self, num_seqs: int) -> int:
        """Workspace bytes of paged_decode for a batch of num_seqs sequences."""
        n = ctypes.c_uint64()
        self._check(self.lib.cpattn_paged_decode_workspace(self._h, num_seqs, ctypes.byref(n)))
        return n.value

    def paged_decode(self, pages: PagedKV, lens, q, out, workspace, lse=None, stream=None):
        """Attention of one new token per sequence, q [num_seqs, NQ, HD], over
        the first lens[b] (int32 CUDA tensor) tokens of its pages.  Row b of q is
        sequence b's: of the rows that paged_plan packed, q[row_starts[1:] - 1],
        unless every sequence has exactly one new token."""
        import torch
        self._check_pages(pages)
        b, nq, hd, dev = pages.num_seqs, self.dims[0], pages.head_dim, pages.device
        _want("q", q, torch.bfloat16, (b, nq, hd), dev)
        _want("out", out, torch.bfloat16, (b, nq, hd), dev)
        _want("lens", lens, torch.int32, (b,), dev)
        if lse is not None:
            _want("lse", lse, torch.float32, (b, nq), dev)
        self._check(self.lib.cpattn_paged_decode(
            self._h, pages.ref, b, lens.data_ptr(), q.data_ptr(), out.data_ptr(), _ptr(lse),
            workspace.data_ptr(), _workspace_bytes(workspace, dev), _stream_on(stream, dev)))

    # -- a serving step around the attention ------------------------------
    def paged_plan(self, pages: PagedKV, cache_lens, new_lens, free_pages, free_count, lens,
                   row_starts, positions, slots, stream=None):
        """Pages, places and positions of a step's new tokens, from the requests'
        lengths: new_lens[b] more for sequence b, which holds cache_lens[b] (< 0: an
        empty place).  Takes pages off the stack free_pages [num_pages] (free_count
        [1]: how many are free), extends pages.block_table and fills lens [num_seqs],
        row_starts [num_seqs + 1] and each row's positions and slots [rows].  All int32
        CUDA tensors; lens may be cache_lens.  What does not fit is not served."""
        b, dev, rows = pages.num_seqs, pages.device, positions.numel()
        self._check_pages(pages)
        have, new, free, count, out, starts, pos, at = _i32_ptrs(
            pages.i32, "cache_lens new_lens free_pages free_count lens row_starts positions slots", dev, cache_lens, b,
            new_lens, b, free_pages, pages.c.num_pages, free_count, 1, lens, b, row_starts, b + 1,
            positions, rows, slots, rows)
        self._check(self.lib.cpattn_paged_plan(self._h, pages.ref, b, rows, have, new, free, count, out,
                                               starts, pos, at, _stream_on(stream, dev)))

    def paged_trim(self, pages: PagedKV, lens, keep, free_pages, free_count, stream=None):
        """Give back to the list the pages of sequence b behind those of its first
        keep[b] tokens, of the lens[b] it holds (0: all of them; < 0: none)."""
        b, dev = pages.num_seqs, pages.device
        self._check_pages(pages)
        have, left, free, count = _i32_ptrs(pages.i32, "lens keep free_pages free_count", dev, lens, b,
                                            keep, b, free_pages, pages.c.num_pages, free_count, 1)
        self._check(self.lib.cpattn_paged_trim(self._h, pages.ref, b, have, left, free, count,
                                               _stream_on(stream, dev)))

    def norm_rope(self, nr: NormRope, positions, q, k, q_out, k_out, stream=None):
        """Per-head norm and rotation of q [rows, NQ, HD] and k [rows, NKV, HD] (bf16;
        rows may lie apart, as in a projection's output) into q_out and k_out, which
        may be q and k.  positions: int32 [rows]; < 0: the row is left alone."""
        rows, nq, nkv, hd, dev = self._check_norm_rope(nr, positions)
        bf16, _ = nr.types
        at = _want_rows("q", q, rows, nq, hd, dev, bf16), _want_rows("k", k, rows, nkv, hd, dev, bf16), \
            _want_rows("q_out", q_out, rows, nq, hd, dev, bf16), _want_rows("k_out", k_out, rows, nkv, hd, dev, bf16)
        if rows:
            self._check(self.lib.cpattn_norm_rope(
                self._h, nr.ref, rows, positions.data_ptr(), q.data_ptr(), at[0], k.data_ptr(), at[1],
                q_out.data_ptr(), at[2], k_out.data_ptr(), at[3], _stream_on(stream, dev)))

    def norm_rope_write_kv(self, nr: NormRope, pages: PagedKV, positions, slots, q, k, v, q_out,
                           stream=None):
        """The same, with K and V [rows, NKV, HD] going straight into their pages: row r
        to slots[r] = page * page_size + slot (int32, from paged_plan; < 0: not stored)."""
        rows, nq, nkv, hd, dev = self._check_norm_rope(nr, positions)
        bf16, i32 = nr.types
        self._check_pages(pages)
        _want("slots", slots, i32, (rows,), dev)
        if pages.device != dev:
            raise ValueError("pages and positions must be on one CUDA device")
        at = _want_rows("q", q, rows, nq, hd, dev, bf16), _want_rows("k", k, rows, nkv, hd, dev, bf16), \
            _want_rows("v", v, rows, nkv, hd, dev, bf16), _want_rows("q_out", q_out, rows, nq, hd, dev, bf16)
        if rows:
            self._check(self.lib.cpattn_norm_rope_write_kv(
                self._h, nr.ref, pages.ref, rows, positions.data_ptr(), slots.data_ptr(), q.data_ptr(), at[0],
                k.data_ptr(), at[1], v.data_ptr(), at[2], q_out.data_ptr(), at[3], _stream_on(stream, dev)))

    def _check_norm_rope(self, nr: NormRope, positions):
        nq, nkv, hd = self.dims
        rows, dev = positions.numel(), positions.get_device()
        _want("positions", positions, nr.types[1], (rows,), dev)
        if nr.device != dev:
            raise ValueError("the norm's weights and positions must be on one CUDA device")
        if nr.head_dim not in (None, hd):
            raise ValueError(f"norm weights of {nr.head_dim} values, the context's heads have {hd}")
        return rows, nq, nkv, hd, dev

    def _check_pages(self, pages: PagedKV):
        if pages.num_kv_heads != self.dims[1] or pages.head_dim != self.dims[2]:
            raise ValueError(f"pages hold {pages.num_kv_heads} kv heads of {pages.head_dim}, the "
                             f"context {self.dims[1]} of {self.dims[2]}")

    def sync_status(self, stream=None) -> int:
        """Synchronise and return the status code (E_TIMEOUT if a device wait expired)."""
        return self.lib.cpattn_sync_status(self._h, _stream(stream))

    def set_barrier_counts(self, records=None):
        """Register a zeroed device uint32 tensor of COUNT_RECORD entries per
        CTA (barrier-count build only), or None to stop counting."""
        nbytes = 0 if records is None else records.numel() * records.element_size()
        self._check(self.lib.cpattn_set_barrier_counts(self._h, _ptr(records), nbytes))

    def set_fault_injection(self, flags: int, timeout_ms: int = 0):
        self._check(self.lib.cpattn_set_fault_injection(self._h, flags, timeout_ms))

    def cache_walk(self, cache_len: int, first: int = 0):
        """(tiles int32 [n], masks uint32 [n, 4]) of the kernel's cache walk,
        from its tile `first` on (the start of a split-KV piece)."""
        n = ctypes.c_int32()
        fn = self.lib.cpattn_cache_walk_from
        self._check(fn(self._h, cache_len, first, None, None, 0, ctypes.byref(n)))
        tiles = np.zeros(max(n.value, 1), dtype=np.int32)
        masks = np.zeros((max(n.value, 1), 4), dtype=np.uint32)
        self._check(fn(self._h, cache_len, first,
                       tiles.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                       masks.ctypes.data_as(ctypes.POINTER(ctypes.c_uint32)), n.value,
                       ctypes.byref(n)))
        return tiles[:n.value], masks[:n.value]

    def last_error(self) -> str:
        return self.lib.cpattn_last_error(self._h).decode()

    def close(self):
        if getattr(self, "_h", None):
            self.lib.cpattn_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check_tensors(self, ts, v_cache):
        """bf16 tensors, and the V cache in the context's format (fp16 with
        v_cache_f16, else bf16); contiguous, on the GPU."""
        import torch
        want_v = torch.float16 if self.v_cache_f16 else torch.bfloat16
        for t, want in [(t, torch.bfloat16) for t in ts] + [(v_cache, want_v)]:
            if t is None or isinstance(t, int):
                continue
            if t.dtype != want or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"expected a contiguous {want} CUDA tensor, got {t.dtype}")


def prefill_noalloc(cfg: Config, cache_lens, chunk_lens, q, k_new, v_new, k_cache, v_cache, out,
                    lse=None, stream=None) -> int:
    """cpattn_prefill_noalloc: the fused prefill without a context and without
    any allocation, for callers that cannot allocate device memory.  Returns
    the status code."""
    fn = load().cpattn_prefill_noalloc
    cl, clp = _i32(cache_lens)
    ch, chp = _i32(chunk_lens)
    return fn(ctypes.byref(cfg), len(cl), clp, chp, _ptr(q), _ptr(k_new), _ptr(v_new),
              _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse), _stream(stream))
