"""Python binding over libpkv's C ABI (include/pkv.h).

Argument marshalling only: every step of the hot path runs in libpkv's CUDA
kernels. There is no CPU fallback; if the library is missing or a call fails,
these functions raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence

import torch

from . import build as _build

PKV_F32, PKV_F16, PKV_BF16, PKV_INT8, PKV_FP8_E4M3 = 0, 1, 2, 3, 4
CODE_DTYPES = {"int8": PKV_INT8, "fp8_e4m3": PKV_FP8_E4M3}
DTYPE_CODE = {torch.float32: PKV_F32, torch.float16: PKV_F16, torch.bfloat16: PKV_BF16}
CODE_DTYPE = {v: k for k, v in DTYPE_CODE.items()}

STATUS = {0: "PKV_OK", -1: "PKV_ERR_INVALID_ARG", -2: "PKV_ERR_UNSUPPORTED", -3: "PKV_ERR_CUDA",
          -4: "PKV_ERR_OUT_OF_RANGE", -5: "PKV_ERR_TIMEOUT", -6: "PKV_ERR_WORKSPACE"}
DEVERR_BLOCK_ID, DEVERR_CONTEXT, DEVERR_TIMEOUT, DEVERR_SLOT = 0x1, 0x2, 0x4, 0x8
DEVERR_NO_BLOCKS, DEVERR_TOKENS, DEVERR_TREE = 0x10, 0x20, 0x40


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class QCacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("code_dtype", ctypes.c_int32), ("act_dtype", ctypes.c_int32)]


class DecodeOptions(ctypes.Structure):
    _fields_ = [("num_ctas", ctypes.c_int32), ("consumer", ctypes.c_int32),
                ("timing_events", ctypes.c_void_p * 2), ("lse_out", ctypes.c_void_p),
                ("tables_ready", ctypes.c_int32), ("pending_tail", ctypes.c_int32)]


class PreparedBmStep:
    """pkv_bm_append_batch + pkv_bm_block_tables for a fixed batch of sequences,
    marshalled once: each call reuses the same host buffers, so what remains per
    step is the two native calls. The returned tensors are views of those
    buffers, overwritten by the next call."""

    def __init__(self, bm, seq_ids, num_tokens, max_blocks_per_seq: int):
        self._ids = torch.as_tensor(list(seq_ids), dtype=torch.int64).contiguous()
        self._nt = torch.as_tensor(list(num_tokens), dtype=torch.int32).contiguous()
        S = len(self._ids)
        self._total = int(self._nt.sum()) if S else 0
        self.slots = torch.empty(max(1, self._total), dtype=torch.int64)
        self.pairs = torch.empty(max(1, S), 2, dtype=torch.int64)
        self.tables = torch.empty(S, max_blocks_per_seq, dtype=torch.int32)
        self.lens = torch.empty(S, dtype=torch.int32)
        self._nc, self._nd = ctypes.c_int32(0), ctypes.c_int32(0)
        L, h = bm._L, bm._h
        self._bm = bm       # keeps the manager alive
        self._append = (L.pkv_bm_append_batch,
                        (h, self._ids.data_ptr(), self._nt.data_ptr(), S, self.slots.data_ptr(),
                         self.pairs.data_ptr(), S, ctypes.byref(self._nc),
                         ctypes.byref(self._nd)))
        self._tables = (L.pkv_bm_block_tables,
                        (h, self._ids.data_ptr(), S, max_blocks_per_seq, self.tables.data_ptr(),
                         self.lens.data_ptr()))
        self._slots_view = self.slots[:self._total]
        self._no_pairs = self.pairs[:0]

    def append(self):
        """(slots, copy pairs) of the step's new tokens."""
        fn, args = self._append
        _bm_check(fn(*args))
        nc = self._nc.value
        return self._slots_view, (self.pairs[:nc] if nc else self._no_pairs)

    def block_tables(self):
        """(block_tables [S][M], context_lens [S]) of the batch."""
        fn, args = self._tables
        _bm_check(fn(*args))
        return self.tables, self.lens


class AppendOptions(ctypes.Structure):
    _fields_ = [("inputs_ready", ctypes.c_int32)]


class PrefixGroups(ctypes.Structure):
    _fields_ = [("num_groups", ctypes.c_int32), ("group_of_seq", ctypes.c_void_p),
                ("group_prefix_blocks", ctypes.c_void_p)]


class PkvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None


def lib_path() -> str:
    return _build.LIB


def lib():
    """Load libpkv (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"libpkv is not built ({path}); run paged_kv_cache_47_gb300.build.build()")
        L = ctypes.CDLL(path)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        dp = ctypes.POINTER(CacheDesc)
        L.pkv_append.argtypes = [dp, vp, vp, vp, i32, vp, vp, vp]
        L.pkv_append.restype = i32
        L.pkv_append_ex.argtypes = [dp, vp, vp, vp, i32, vp, vp, vp,
                                    ctypes.POINTER(AppendOptions)]
        L.pkv_append_ex.restype = i32
        L.pkv_decode_workspace_bytes.argtypes = [dp, i32, i32, i32]
        L.pkv_decode_workspace_bytes.restype = sz
        L.pkv_decode_workspace_bytes_ex.argtypes = [dp, i32, i32]
        L.pkv_decode_workspace_bytes_ex.restype = sz
        dec = [dp, vp, i32, i32, vp, vp, vp, i32, vp, ctypes.c_float, vp, i32, vp, sz, vp]
        L.pkv_decode_attention.argtypes = dec
        L.pkv_decode_attention.restype = i32
        L.pkv_decode_attention_ex.argtypes = dec + [ctypes.POINTER(DecodeOptions)]
        L.pkv_decode_attention_ex.restype = i32
        L.pkv_append_decode_attention.argtypes = [dp, vp, i32, i32, vp, vp, vp, vp, vp, i32, vp,
                                                  ctypes.c_float, vp, i32, vp, sz, vp,
                                                  ctypes.POINTER(DecodeOptions)]
        L.pkv_append_decode_attention.restype = i32
        L.pkv_block_copy.argtypes = [dp, vp, i32, vp, vp, vp]
        L.pkv_block_copy.restype = i32
        qp = ctypes.POINTER(QCacheDesc)
        L.pkv_append_quant.argtypes = [qp, vp, vp, vp, i32, vp, vp, vp, vp, vp]
        L.pkv_append_quant.restype = i32
        L.pkv_append_quant_ex.argtypes = [qp, vp, vp, vp, i32, vp, vp, vp, vp, vp,
                                          ctypes.POINTER(AppendOptions)]
        L.pkv_append_quant_ex.restype = i32
        L.pkv_decode_quant_workspace_bytes.argtypes = [qp, i32, i32]
        L.pkv_decode_quant_workspace_bytes.restype = sz
        L.pkv_decode_attention_quant.argtypes = [qp, vp, i32, i32, vp, vp, vp, vp, vp, i32, vp,
                                                 ctypes.c_float, vp, i32, vp, sz, vp,
                                                 ctypes.POINTER(DecodeOptions)]
        L.pkv_decode_attention_quant.restype = i32
        L.pkv_append_decode_attention_quant.argtypes = [qp, vp, i32, i32, vp, vp, vp, vp, vp, vp,
                                                        vp, i32, vp, ctypes.c_float, vp, i32, vp,
                                                        sz, vp, ctypes.POINTER(DecodeOptions)]
        L.pkv_append_decode_attention_quant.restype = i32
        L.pkv_block_copy_quant.argtypes = [qp, vp, i32, vp, vp, vp, vp, vp]
        L.pkv_block_copy_quant.restype = i32
        L.pkv_decode_prefix_workspace_bytes.argtypes = [dp, i32, i32, i32,
                                                        ctypes.POINTER(PrefixGroups), i32]
        L.pkv_decode_prefix_workspace_bytes.restype = sz
        L.pkv_decode_attention_prefix.argtypes = [dp, vp, i32, i32, vp, vp, vp, i32, vp,
                                                  ctypes.c_float, ctypes.POINTER(PrefixGroups),
                                                  vp, i32, vp, sz, vp,
                                                  ctypes.POINTER(DecodeOptions)]
        L.pkv_decode_attention_prefix.restype = i32
        L.pkv_debug_set_wait_fault.argtypes = [ctypes.c_uint64, i32]
        L.pkv_debug_set_wait_fault.restype = i32
        L.pkv_get_error.argtypes = [ctypes.POINTER(ctypes.c_int32), vp]
        L.pkv_get_error.restype = i32
        L.pkv_status_string.argtypes = [i32]
        L.pkv_status_string.restype = ctypes.c_char_p
        L.pkv_last_error_message.argtypes = []
        L.pkv_last_error_message.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise PkvError(status, lib().pkv_last_error_message().decode())


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def cache_desc(k_pool: torch.Tensor) -> CacheDesc:
    """Descriptor of a pool tensor [NB][Hk][B][D]."""
    NB, Hk, B, D = k_pool.shape
    return CacheDesc(NB, B, Hk, D, DTYPE_CODE[k_pool.dtype])


def _pools(k_pool, v_pool):
    if k_pool.shape != v_pool.shape or k_pool.dtype != v_pool.dtype:
        raise ValueError("k_pool and v_pool differ in shape or dtype")
    if not (k_pool.is_contiguous() and v_pool.is_contiguous()):
        raise ValueError("pools must be contiguous")
    return cache_desc(k_pool)


def append(k_new, v_new, slot_mapping, k_pool, v_pool, stream=None,
           inputs_ready: bool = False) -> None:
    """Write k_new/v_new [N][Hk][D] into the pools at slot_mapping [N] (int64).
    inputs_ready: no kernel that may still be running writes the three inputs, so
    they are read before the wait on the preceding kernel (pkv_append_options)."""
    desc = _pools(k_pool, v_pool)
    k_new, v_new = k_new.contiguous(), v_new.contiguous()
    sm = slot_mapping.contiguous()
    assert sm.dtype == torch.int64 and k_new.dtype == k_pool.dtype
    opts = AppendOptions(int(inputs_ready))
    _check(lib().pkv_append_ex(ctypes.byref(desc), _ptr(k_new), _ptr(v_new), _ptr(sm),
                               sm.numel(), _ptr(k_pool), _ptr(v_pool), _stream(stream),
                               ctypes.byref(opts)))


def workspace_bytes(k_pool, num_q_heads: int, num_ctas: int = 0) -> int:
    desc = cache_desc(k_pool)
    return int(lib().pkv_decode_workspace_bytes_ex(ctypes.byref(desc), num_q_heads, num_ctas))


def alloc_workspace(k_pool, num_q_heads: int, num_ctas: int = 0) -> torch.Tensor:
    """Split-K workspace, zero-filled as the library requires before first use
    (its arrival counters; every call leaves them zero again)."""
    n = workspace_bytes(k_pool, num_q_heads, num_ctas)
    if n == 0:
        raise PkvError(-1, "workspace size query failed")
    return torch.zeros(n, dtype=torch.uint8, device=k_pool.device)


def decode_attention(q, k_pool, v_pool, block_tables, context_lens, scale: float,
                     out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                     workspace: Optional[torch.Tensor] = None, num_ctas: int = 0,
                     consumer: int = 0, timing_events: Optional[Sequence] = None,
                     stream=None, lse_out: Optional[torch.Tensor] = None,
                     tables_ready: bool = False, pending_tail: int = 0) -> torch.Tensor:
    """Paged decode attention: out[s][h] = softmax(scale q K^T) V over context_lens[s] tokens.
    tables_ready: the caller promises that no kernel that may still be running writes the
    tables or lengths (pkv_decode_options.tables_ready).
    pending_tail: n > 0 promises, besides, that no kernel that may still be running
    writes q or any row below the last n of each sequence
    (pkv_decode_options.pending_tail)."""
    desc = _pools(k_pool, v_pool)
    S, Hq, D = q.shape
    q = q.contiguous()
    bt = block_tables.contiguous()
    cl = context_lens.contiguous()
    assert bt.dtype == torch.int32 and cl.dtype == torch.int32 and q.dtype == k_pool.dtype
    if out is None:
        out = torch.empty(S, Hq, D, dtype=out_dtype or q.dtype, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(k_pool, Hq, num_ctas)
    opts = DecodeOptions()
    opts.num_ctas = num_ctas
    opts.consumer = consumer
    opts.tables_ready = int(tables_ready)
    opts.pending_tail = int(pending_tail)
    if timing_events is not None:
        for i, ev in enumerate(timing_events):
            opts.timing_events[i] = None if ev is None else ev.cuda_event
    if lse_out is not None:
        assert lse_out.dtype == torch.float32 and lse_out.shape == (S, Hq) and lse_out.is_contiguous()
        opts.lse_out = lse_out.data_ptr()
    _check(lib().pkv_decode_attention_ex(
        ctypes.byref(desc), _ptr(q), S, Hq, _ptr(k_pool), _ptr(v_pool), _ptr(bt), bt.shape[1],
        _ptr(cl), float(scale), _ptr(out), DTYPE_CODE[out.dtype], _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream), ctypes.byref(opts)))
    return out


class PreparedDecode:
    """A decode-attention call whose arguments are marshalled once.

    For repeated decode steps on stable buffers (the usual serving loop, and
    CUDA-graph capture): the tensors' addresses, shapes and the workspace are
    fixed at construction; each call only passes the stream. The caller keeps
    the tensors alive and rewrites their contents in place between steps.
    """

    def __init__(self, q, k_pool, v_pool, block_tables, context_lens, scale: float,
                 out: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                 num_ctas: int = 0, consumer: int = 0, tables_ready: bool = False,
                 pending_tail: int = 0):
        self._desc = _pools(k_pool, v_pool)
        for t in (q, block_tables, context_lens, out):
            if not t.is_contiguous():
                raise ValueError("prepared decode needs contiguous tensors")
        assert block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32
        assert q.dtype == k_pool.dtype
        S, Hq, D = q.shape
        if workspace is None:
            workspace = alloc_workspace(k_pool, Hq, num_ctas)
        self._keep = (q, k_pool, v_pool, block_tables, context_lens, out, workspace)
        self._opts = DecodeOptions()
        self._opts.num_ctas = num_ctas
        self._opts.consumer = consumer
        self._opts.tables_ready = int(tables_ready)
        self._opts.pending_tail = int(pending_tail)
        self._args = (ctypes.byref(self._desc), q.data_ptr(), S, Hq, k_pool.data_ptr(),
                      v_pool.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
                      context_lens.data_ptr(), float(scale), out.data_ptr(),
                      DTYPE_CODE[out.dtype], workspace.data_ptr(),
                      workspace.numel() * workspace.element_size())
        self._fn = lib().pkv_decode_attention_ex
        self.out = out

    def __call__(self, stream, timing_events: Optional[Sequence] = None) -> None:
        opts = self._opts
        for i in range(2):
            ev = timing_events[i] if timing_events is not None else None
            opts.timing_events[i] = None if ev is None else ev.cuda_event
        _check(self._fn(*self._args, _stream(stream), ctypes.byref(opts)))


def append_decode_attention(q, k_new, v_new, k_pool, v_pool, block_tables, context_lens,
                            scale: float, out: Optional[torch.Tensor] = None,
                            out_dtype: Optional[torch.dtype] = None,
                            workspace: Optional[torch.Tensor] = None, num_ctas: int = 0,
                            consumer: int = 0, stream=None, tables_ready: bool = False,
                            pending_tail: int = 0) -> torch.Tensor:
    """One decode step in one launch (pkv_append_decode_attention): each
    sequence's new row k_new[s] / v_new[s] [S][Hk][D] goes to position
    context_lens[s] - 1 (the slot its block table gives), and the attention
    runs over the context including it."""
    desc = _pools(k_pool, v_pool)
    S, Hq, D = q.shape
    q, k_new, v_new = q.contiguous(), k_new.contiguous(), v_new.contiguous()
    bt, cl = block_tables.contiguous(), context_lens.contiguous()
    assert bt.dtype == torch.int32 and cl.dtype == torch.int32
    assert q.dtype == k_pool.dtype == k_new.dtype == v_new.dtype
    if out is None:
        out = torch.empty(S, Hq, D, dtype=out_dtype or q.dtype, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(k_pool, Hq, num_ctas)
    opts = DecodeOptions()
    opts.num_ctas = num_ctas
    opts.consumer = consumer
    opts.tables_ready = int(tables_ready)
    opts.pending_tail = int(pending_tail)
    _check(lib().pkv_append_decode_attention(
        ctypes.byref(desc), _ptr(q), S, Hq, _ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool),
        _ptr(bt), bt.shape[1], _ptr(cl), float(scale), _ptr(out), DTYPE_CODE[out.dtype],
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream),
        ctypes.byref(opts)))
    return out


class PreparedAppendDecode(PreparedDecode):
    """A pkv_append_decode_attention call whose arguments are marshalled once
    (see PreparedDecode); k_new and v_new are rewritten in place each step."""

    def __init__(self, q, k_new, v_new, k_pool, v_pool, block_tables, context_lens,
                 scale: float, out: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                 num_ctas: int = 0, consumer: int = 0, tables_ready: bool = False,
                 pending_tail: int = 0):
        super().__init__(q, k_pool, v_pool, block_tables, context_lens, scale, out, workspace,
                         num_ctas, consumer, tables_ready, pending_tail)
        for t in (k_new, v_new):
            if not t.is_contiguous() or t.dtype != k_pool.dtype:
                raise ValueError("k_new / v_new must be contiguous, in the cache dtype")
        self._keep = self._keep + (k_new, v_new)
        a = self._args
        # q, S, Hq | k_new, v_new | pools, tables, ...
        self._args = a[:4] + (k_new.data_ptr(), v_new.data_ptr()) + a[4:]
        self._fn = lib().pkv_append_decode_attention


class PreparedAppend:
    """An append call whose arguments are marshalled once (see PreparedDecode)."""

    def __init__(self, k_new, v_new, slot_mapping, k_pool, v_pool, inputs_ready: bool = False):
        self._desc = _pools(k_pool, v_pool)
        for t in (k_new, v_new, slot_mapping):
            if not t.is_contiguous():
                raise ValueError("prepared append needs contiguous tensors")
        assert slot_mapping.dtype == torch.int64 and k_new.dtype == k_pool.dtype
        self._keep = (k_new, v_new, slot_mapping, k_pool, v_pool)
        self._opts = AppendOptions(int(inputs_ready))
        self._args = (ctypes.byref(self._desc), k_new.data_ptr(), v_new.data_ptr(),
                      slot_mapping.data_ptr(), slot_mapping.numel(), k_pool.data_ptr(),
                      v_pool.data_ptr())
        self._fn = lib().pkv_append_ex

    def __call__(self, stream) -> None:
        _check(self._fn(*self._args, _stream(stream), ctypes.byref(self._opts)))


def block_copy(pairs, k_pool, v_pool, stream=None) -> None:
    """Copy whole blocks src -> dst; pairs is host data [n][2] (list or CPU tensor)."""
    desc = _pools(k_pool, v_pool)
    p = torch.as_tensor(pairs, dtype=torch.int64).reshape(-1, 2).contiguous()
    assert p.device.type == "cpu", "block-copy pairs are host memory"
    _check(lib().pkv_block_copy(ctypes.byref(desc), _ptr(p), p.shape[0], _ptr(k_pool),
                                _ptr(v_pool), _stream(stream)))


def set_wait_fault(wait_limit_ns: int = 0, drop_arrivals: int = 0) -> None:
    """Test hook (pkv_debug_set_wait_fault): the wait limit of the next decode
    launches (0 = the default 2 s) and how many of them withhold one arrival
    so that a bounded wait runs out. (0, 0) restores normal operation."""
    _check(lib().pkv_debug_set_wait_fault(int(wait_limit_ns), int(drop_arrivals)))


def get_error_status(stream=None):
    """(status, word): pkv_get_error's return code and the device error word
    it read and cleared."""
    w = ctypes.c_int32(0)
    st = lib().pkv_get_error(ctypes.byref(w), _stream(stream))
    return int(st), int(w.value)


def get_error(stream=None) -> int:
    """Synchronise and read+clear the device error word (PKV_DEVERR_* bits)."""
    w = ctypes.c_int32(0)
    lib().pkv_get_error(ctypes.byref(w), _stream(stream))
    return int(w.value)


# ------------------------------------------------------------------ 8-bit caches
class QuantCache:
    """An 8-bit paged KV cache: code pools [NB][Hk][B][D] (uint8) and row-scale
    pools [NB][Hk][B] (fp32) for K and V, with the activation dtype of q,
    k_new and v_new. Holds the tensors; the library owns no memory."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales, code: str, act_dtype: torch.dtype):
        for t in (k_codes, v_codes, k_scales, v_scales):
            if not t.is_contiguous():
                raise ValueError("quantized pools must be contiguous")
        if k_codes.dtype != torch.uint8 or v_codes.shape != k_codes.shape:
            raise ValueError("code pools must be uint8 and of one shape")
        NB, Hk, B, D = k_codes.shape
        if k_scales.dtype != torch.float32 or k_scales.shape != (NB, Hk, B) or \
                v_scales.shape != k_scales.shape:
            raise ValueError("scale pools must be float32 [NB][Hk][B]")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.code, self.act_dtype = code, act_dtype
        self.desc = QCacheDesc(NB, B, Hk, D, CODE_DTYPES[code], DTYPE_CODE[act_dtype])

    @classmethod
    def empty(cls, num_blocks, num_kv_heads, block_size, head_dim, code: str,
              act_dtype: torch.dtype, device="cuda"):
        kc = torch.zeros(num_blocks, num_kv_heads, block_size, head_dim, dtype=torch.uint8,
                         device=device)
        ks = torch.zeros(num_blocks, num_kv_heads, block_size, dtype=torch.float32, device=device)
        return cls(kc, kc.clone(), ks, ks.clone(), code, act_dtype)

    def pointers(self):
        return (self.k_codes.data_ptr(), self.v_codes.data_ptr(), self.k_scales.data_ptr(),
                self.v_scales.data_ptr())


def append_quant(k_new, v_new, slot_mapping, cache: QuantCache, stream=None,
                 inputs_ready: bool = False) -> None:
    """Quantize k_new/v_new [N][Hk][D] (the cache's activation dtype) into their slots
    (inputs_ready: see append)."""
    k_new, v_new = k_new.contiguous(), v_new.contiguous()
    sm = slot_mapping.contiguous()
    assert sm.dtype == torch.int64 and k_new.dtype == cache.act_dtype == v_new.dtype
    opts = AppendOptions(int(inputs_ready))
    _check(lib().pkv_append_quant_ex(ctypes.byref(cache.desc), _ptr(k_new), _ptr(v_new), _ptr(sm),
                                     sm.numel(), *cache.pointers(), _stream(stream),
                                     ctypes.byref(opts)))


def quant_workspace_bytes(cache: QuantCache, num_q_heads: int, num_ctas: int = 0) -> int:
    return int(lib().pkv_decode_quant_workspace_bytes(ctypes.byref(cache.desc), num_q_heads,
                                                      num_ctas))


def alloc_quant_workspace(cache: QuantCache, num_q_heads: int, num_ctas: int = 0) -> torch.Tensor:
    """Zero-filled split-K workspace for pkv_decode_attention_quant."""
    n = quant_workspace_bytes(cache, num_q_heads, num_ctas)
    if n == 0:
        raise PkvError(-1, "workspace size query failed")
    return torch.zeros(n, dtype=torch.uint8, device=cache.k_codes.device)


def decode_attention_quant(q, cache: QuantCache, block_tables, context_lens, scale: float,
                           out: Optional[torch.Tensor] = None,
                           out_dtype: Optional[torch.dtype] = None,
                           workspace: Optional[torch.Tensor] = None, num_ctas: int = 0,
                           consumer: int = 0, timing_events: Optional[Sequence] = None,
                           stream=None, tables_ready: bool = False,
                           pending_tail: int = 0) -> torch.Tensor:
    """Paged decode attention over an 8-bit cache (tables_ready, pending_tail: see
    decode_attention)."""
    S, Hq, D = q.shape
    q = q.contiguous()
    bt, cl = block_tables.contiguous(), context_lens.contiguous()
    assert bt.dtype == torch.int32 and cl.dtype == torch.int32 and q.dtype == cache.act_dtype
    if out is None:
        out = torch.empty(S, Hq, D, dtype=out_dtype or q.dtype, device=q.device)
    if workspace is None:
        workspace = alloc_quant_workspace(cache, Hq, num_ctas)
    opts = DecodeOptions()
    opts.num_ctas = num_ctas
    opts.consumer = consumer
    opts.tables_ready = int(tables_ready)
    opts.pending_tail = int(pending_tail)
    if timing_events is not None:
        for i, ev in enumerate(timing_events):
            opts.timing_events[i] = None if ev is None else ev.cuda_event
    _check(lib().pkv_decode_attention_quant(
        ctypes.byref(cache.desc), _ptr(q), S, Hq, *cache.pointers(), _ptr(bt), bt.shape[1],
        _ptr(cl), float(scale), _ptr(out), DTYPE_CODE[out.dtype], _ptr(workspace),
        workspace.numel(), _stream(stream), ctypes.byref(opts)))
    return out


class PreparedDecodeQuant:
    """pkv_decode_attention_quant with its arguments marshalled once (see PreparedDecode)."""

    def __init__(self, q, cache: QuantCache, block_tables, context_lens, scale: float,
                 out: torch.Tensor, workspace: Optional[torch.Tensor] = None, num_ctas: int = 0,
                 tables_ready: bool = False, pending_tail: int = 0):
        for t in (q, block_tables, context_lens, out):
            if not t.is_contiguous():
                raise ValueError("prepared decode needs contiguous tensors")
        assert q.dtype == cache.act_dtype
        S, Hq, D = q.shape
        if workspace is None:
            workspace = alloc_quant_workspace(cache, Hq, num_ctas)
        self._keep = (q, cache, block_tables, context_lens, out, workspace)
        self._opts = DecodeOptions()
        self._opts.num_ctas = num_ctas
        self._opts.tables_ready = int(tables_ready)
        self._opts.pending_tail = int(pending_tail)
        self._args = (ctypes.byref(cache.desc), q.data_ptr(), S, Hq, *cache.pointers(),
                      block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(),
                      float(scale), out.data_ptr(), DTYPE_CODE[out.dtype], workspace.data_ptr(),
                      workspace.numel())
        self._fn = lib().pkv_decode_attention_quant
        self.out = out

    def __call__(self, stream, timing_events: Optional[Sequence] = None) -> None:
        opts = self._opts
        for i in range(2):
            ev = timing_events[i] if timing_events is not None else None
            opts.timing_events[i] = None if ev is None else ev.cuda_event
        _check(self._fn(*self._args, _stream(stream), ctypes.byref(opts)))


def append_decode_attention_quant(q, k_new, v_new, cache: QuantCache, block_tables,
                                  context_lens, scale: float, out: Optional[torch.Tensor] = None,
                                  out_dtype: Optional[torch.dtype] = None,
                                  workspace: Optional[torch.Tensor] = None, num_ctas: int = 0,
                                  stream=None, tables_ready: bool = False,
                                  pending_tail: int = 0) -> torch.Tensor:
    """One decode step over an 8-bit cache (pkv_append_decode_attention_quant):
    each sequence's new row k_new[s] / v_new[s] [S][Hk][D] is quantized into
    position context_lens[s] - 1 of its table row, and the attention runs over
    the context including it."""
    S, Hq, D = q.shape
    q, k_new, v_new = q.contiguous(), k_new.contiguous(), v_new.contiguous()
    bt, cl = block_tables.contiguous(), context_lens.contiguous()
    assert bt.dtype == torch.int32 and cl.dtype == torch.int32
    assert q.dtype == k_new.dtype == v_new.dtype == cache.act_dtype
    if out is None:
        out = torch.empty(S, Hq, D, dtype=out_dtype or q.dtype, device=q.device)
    if workspace is None:
        workspace = alloc_quant_workspace(cache, Hq, num_ctas)
    opts = DecodeOptions()
    opts.num_ctas = num_ctas
    opts.tables_ready = int(tables_ready)
    opts.pending_tail = int(pending_tail)
    _check(lib().pkv_append_decode_attention_quant(
        ctypes.byref(cache.desc), _ptr(q), S, Hq, _ptr(k_new), _ptr(v_new), *cache.pointers(),
        _ptr(bt), bt.shape[1], _ptr(cl), float(scale), _ptr(out), DTYPE_CODE[out.dtype],
        _ptr(workspace), workspace.numel(), _stream(stream), ctypes.byref(opts)))
    return out


class PreparedAppendQuant:
    """pkv_append_quant with its arguments marshalled once (see PreparedDecode)."""

    def __init__(self, k_new, v_new, slot_mapping, cache: QuantCache, inputs_ready: bool = False):
        for t in (k_new, v_new, slot_mapping):
            if not t.is_contiguous():
                raise ValueError("prepared append needs contiguous tensors")
        assert slot_mapping.dtype == torch.int64 and k_new.dtype == cache.act_dtype
        self._keep = (k_new, v_new, slot_mapping, cache)
        self._opts = AppendOptions(int(inputs_ready))
        self._args = (ctypes.byref(cache.desc), k_new.data_ptr(), v_new.data_ptr(),
                      slot_mapping.data_ptr(), slot_mapping.numel(), *cache.pointers())
        self._fn = lib().pkv_append_quant_ex

    def __call__(self, stream) -> None:
        _check(self._fn(*self._args, _stream(stream), ctypes.byref(self._opts)))


def block_copy_quant(pairs, cache: QuantCache, stream=None) -> None:
    """Copy whole blocks (codes and scales) src -> dst; pairs is host data [n][2]."""
    p = torch.as_tensor(pairs, dtype=torch.int64).reshape(-1, 2).contiguous()
    assert p.device.type == "cpu", "block-copy pairs are host memory"
    _check(lib().pkv_block_copy_quant(ctypes.byref(cache.desc), _ptr(p), p.shape[0],
                                      *cache.pointers(), _stream(stream)))


# ------------------------------------------------------------------ block manager
class BmStats(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("free_blocks", ctypes.c_int32),
                ("shared_blocks", ctypes.c_int32), ("prefix_entries", ctypes.c_int32),
                ("sequences", ctypes.c_int64), ("tokens", ctypes.c_int64)]


def _bm_lib():
    L = lib()
    if not getattr(L, "_bm_ready", False):
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.pkv_bm_create.argtypes = [i32, i32, ctypes.POINTER(vp)]
        L.pkv_bm_create.restype = i32
        L.pkv_bm_destroy.argtypes = [vp]
        L.pkv_bm_destroy.restype = None
        L.pkv_bm_add_sequence.argtypes = [vp, i64, vp, i32, vp]
        L.pkv_bm_add_sequence.restype = i32
        L.pkv_bm_append.argtypes = [vp, i64, i32, vp, vp, i32, ctypes.POINTER(i32)]
        L.pkv_bm_append.restype = i32
        L.pkv_bm_append_batch.argtypes = [vp, vp, vp, i32, vp, vp, i32, ctypes.POINTER(i32),
                                          ctypes.POINTER(i32)]
        L.pkv_bm_append_batch.restype = i32
        L.pkv_bm_fork.argtypes = [vp, i64, i64]
        L.pkv_bm_fork.restype = i32
        L.pkv_bm_free_sequence.argtypes = [vp, i64]
        L.pkv_bm_free_sequence.restype = i32
        L.pkv_bm_block_tables.argtypes = [vp, vp, i32, i32, vp, vp]
        L.pkv_bm_block_tables.restype = i32
        L.pkv_bm_stats_get.argtypes = [vp, ctypes.POINTER(BmStats)]
        L.pkv_bm_stats_get.restype = i32
        L.pkv_bm_refcount.argtypes = [vp, i32]
        L.pkv_bm_refcount.restype = i32
        L.pkv_bm_simulate_admission.argtypes = [i32, i32, vp, i32, i32, ctypes.POINTER(i32),
                                                ctypes.POINTER(ctypes.c_double)]
        L.pkv_bm_simulate_admission.restype = i32
        L._bm_ready = True
    return L


class NoBlocks(PkvError):
    """The block manager has too few free blocks; the call changed nothing."""


def _bm_check(status: int):
    if status == -7:
        raise NoBlocks(status, lib().pkv_last_error_message().decode())
    _check(status)


class BlockManager:
    """Host block manager of a paged KV cache (libpkv's pkv_bm_* calls)."""

    def __init__(self, num_blocks: int, block_size: int):
        L = _bm_lib()
        h = ctypes.c_void_p()
        _bm_check(L.pkv_bm_create(num_blocks, block_size, ctypes.byref(h)))
        self._h, self._L = h, L
        self.block_size = block_size

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            self._L.pkv_bm_destroy(h)
            self._h = None

    def add_sequence(self, seq: int, prefix_hashes=()) -> list:
        hs = (ctypes.c_uint64 * max(1, len(prefix_hashes)))(*[int(x) & (2 ** 64 - 1)
                                                              for x in prefix_hashes])
        hits = (ctypes.c_uint8 * max(1, len(prefix_hashes)))()
        _bm_check(self._L.pkv_bm_add_sequence(self._h, seq, hs, len(prefix_hashes), hits))
        return [bool(hits[i]) for i in range(len(prefix_hashes))]

    def append(self, seq: int, n: int):
        """Slots of n new tokens and the (src, dst) copies to run first."""
        slots = (ctypes.c_int64 * max(1, n))()
        pairs = (ctypes.c_int64 * 2)()
        nc = ctypes.c_int32(0)
        _bm_check(self._L.pkv_bm_append(self._h, seq, n, slots, pairs, 1, ctypes.byref(nc)))
        return [slots[i] for i in range(n)], [(pairs[2 * i], pairs[2 * i + 1])
                                               for i in range(nc.value)]

    def append_batch(self, seq_ids, num_tokens):
        """Slots (all sequences back to back) and copies of one step; raises on
        failure after the sequences before the failing one were applied."""
        ids = torch.as_tensor(list(seq_ids), dtype=torch.int64)
        nt = torch.as_tensor(list(num_tokens), dtype=torch.int32)
        total = int(nt.sum()) if len(nt) else 0
        slots = torch.empty(max(1, total), dtype=torch.int64)
        pairs = torch.empty(max(1, len(ids)), 2, dtype=torch.int64)
        nc, nd = ctypes.c_int32(0), ctypes.c_int32(0)
        _bm_check(self._L.pkv_bm_append_batch(self._h, ids.data_ptr(), nt.data_ptr(), len(ids),
                                              slots.data_ptr(), pairs.data_ptr(), len(ids),
                                              ctypes.byref(nc), ctypes.byref(nd)))
        return slots[:total], pairs[:nc.value]

    def fork(self, parent: int, child: int) -> None:
        _bm_check(self._L.pkv_bm_fork(self._h, parent, child))

    def free_sequence(self, seq: int) -> None:
        _bm_check(self._L.pkv_bm_free_sequence(self._h, seq))

    def block_tables(self, seq_ids, max_blocks_per_seq: int):
        """(block_tables [S][M] int32, context_lens [S] int32) as CPU tensors."""
        ids = torch.as_tensor(list(seq_ids), dtype=torch.int64)
        tables = torch.empty(len(ids), max_blocks_per_seq, dtype=torch.int32)
        lens = torch.empty(len(ids), dtype=torch.int32)
        _bm_check(self._L.pkv_bm_block_tables(self._h, ids.data_ptr(), len(ids),
                                              max_blocks_per_seq, tables.data_ptr(),
                                              lens.data_ptr()))
        return tables, lens

    def prepared_step(self, seq_ids, num_tokens, max_blocks_per_seq: int) -> "PreparedBmStep":
        """A decode step's two calls (append_batch, block_tables) for a fixed batch,
        with their argument and output buffers made once (see PreparedBmStep)."""
        return PreparedBmStep(self, seq_ids, num_tokens, max_blocks_per_seq)

    def table(self, seq: int) -> list:
        width = max(1, self.stats().num_blocks)
        while True:
            try:
                t, _ = self.block_tables([seq], width)
            except PkvError:
                if width >= 1 << 24:
                    raise
                width *= 4      # a prefix can repeat a block, so a table may exceed the pool
                continue
            return [int(b) for b in t[0].tolist() if b >= 0]

    def stats(self) -> BmStats:
        st = BmStats()
        _bm_check(self._L.pkv_bm_stats_get(self._h, ctypes.byref(st)))
        return st

    def refcount(self, block: int) -> int:
        return int(self._L.pkv_bm_refcount(self._h, block))

    def num_free(self) -> int:
        return int(self.stats().free_blocks)


def simulate_admission(num_blocks: int, block_size: int, context_lens, reserve_tokens: int = 0):
    """(admitted, utilisation) of requests admitted in order into a pool."""
    L = _bm_lib()
    cl = torch.as_tensor(list(context_lens), dtype=torch.int32)
    adm = ctypes.c_int32(0)
    u = ctypes.c_double(0.0)
    _bm_check(L.pkv_bm_simulate_admission(num_blocks, block_size, cl.data_ptr(), len(cl),
                                          reserve_tokens, ctypes.byref(adm), ctypes.byref(u)))
    return int(adm.value), float(u.value)


# ------------------------------------------------------------------ flat spans
class FlatInfo(ctypes.Structure):
    _fields_ = [("k_base", ctypes.c_void_p), ("slot_stride", ctypes.c_size_t),
                ("v_offset", ctypes.c_size_t), ("granularity", ctypes.c_size_t),
                ("committed_bytes", ctypes.c_size_t), ("committed_tokens", ctypes.c_void_p)]


def _flat_lib():
    L = lib()
    if not getattr(L, "_flat_ready", False):
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        L.pkv_flat_create.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(vp)]
        L.pkv_flat_create.restype = i32
        L.pkv_flat_destroy.argtypes = [vp]
        L.pkv_flat_destroy.restype = None
        L.pkv_flat_reserve.argtypes = [vp, i32, i32]
        L.pkv_flat_reserve.restype = i32
        L.pkv_flat_release.argtypes = [vp, i32]
        L.pkv_flat_release.restype = i32
        L.pkv_flat_get_info.argtypes = [vp, ctypes.POINTER(FlatInfo)]
        L.pkv_flat_get_info.restype = i32
        L.pkv_flat_append.argtypes = [vp, vp, vp, vp, vp, i32, vp]
        L.pkv_flat_append.restype = i32
        L.pkv_flat_decode_workspace_bytes.argtypes = [vp, i32, i32]
        L.pkv_flat_decode_workspace_bytes.restype = sz
        L.pkv_decode_attention_flat.argtypes = [vp, vp, i32, i32, vp, vp, ctypes.c_float, vp, i32,
                                                vp, sz, vp, ctypes.POINTER(DecodeOptions)]
        L.pkv_decode_attention_flat.restype = i32
        L._flat_ready = True
    return L


class FlatCache:
    """A KV cache kept contiguous in virtual memory (libpkv's pkv_flat_* calls):
    num_slots sequence slots of capacity tokens, physical chunks mapped as
    slots grow."""

    def __init__(self, num_slots: int, capacity: int, num_kv_heads: int, head_dim: int,
                 dtype: torch.dtype):
        L = _flat_lib()
        h = ctypes.c_void_p()
        _check(L.pkv_flat_create(num_slots, capacity, num_kv_heads, head_dim, DTYPE_CODE[dtype],
                                 ctypes.byref(h)))
        self._h, self._L = h, L
        self.num_slots, self.capacity = num_slots, capacity
        self.num_kv_heads, self.head_dim, self.dtype = num_kv_heads, head_dim, dtype

    def close(self):
        if getattr(self, "_h", None):
            self._L.pkv_flat_destroy(self._h)
            self._h = None

    def __del__(self):
        self.close()

    def reserve(self, slot: int, tokens: int) -> None:
        _check(self._L.pkv_flat_reserve(self._h, slot, tokens))

    def release(self, slot: int) -> None:
        _check(self._L.pkv_flat_release(self._h, slot))

    def info(self) -> FlatInfo:
        inf = FlatInfo()
        _check(self._L.pkv_flat_get_info(self._h, ctypes.byref(inf)))
        return inf

    def append(self, k_new, v_new, slots, positions, stream=None) -> None:
        """k_new/v_new [N][Hk][D] (device); slots/positions int32 [N] (device)."""
        k_new, v_new = k_new.contiguous(), v_new.contiguous()
        sl, pos = slots.contiguous(), positions.contiguous()
        assert sl.dtype == torch.int32 and pos.dtype == torch.int32 and k_new.dtype == self.dtype
        _check(self._L.pkv_flat_append(self._h, _ptr(k_new), _ptr(v_new), _ptr(sl), _ptr(pos),
                                       sl.numel(), _stream(stream)))

    def workspace(self, num_q_heads: int, num_ctas: int = 0) -> torch.Tensor:
        n = int(self._L.pkv_flat_decode_workspace_bytes(self._h, num_q_heads, num_ctas))
        if n == 0:
            raise PkvError(-1, "workspace size query failed")
        return torch.zeros(n, dtype=torch.uint8, device="cuda")

    def decode_attention(self, q, slots, context_lens, scale: float,
                         out: Optional[torch.Tensor] = None,
                         out_dtype: Optional[torch.dtype] = None,
                         workspace: Optional[torch.Tensor] = None, num_ctas: int = 0,
                         timing_events: Optional[Sequence] = None, stream=None,
                         tables_ready: bool = False, pending_tail: int = 0) -> torch.Tensor:
        S, Hq, D = q.shape
        q = q.contiguous()
        sl, cl = slots.contiguous(), context_lens.contiguous()
        assert sl.dtype == torch.int32 and cl.dtype == torch.int32 and q.dtype == self.dtype
        if out is None:
            out = torch.empty(S, Hq, D, dtype=out_dtype or q.dtype, device=q.device)
        if workspace is None:
            workspace = self.workspace(Hq, num_ctas)
        opts = DecodeOptions()
        opts.num_ctas = num_ctas
        opts.tables_ready = int(tables_ready)
        opts.pending_tail = int(pending_tail)
        if timing_events is not None:
            for i, ev in enumerate(timing_events):
                opts.timing_events[i] = None if ev is None else ev.cuda_event
        _check(self._L.pkv_decode_attention_flat(
            self._h, _ptr(q), S, Hq, _ptr(sl), _ptr(cl), float(scale), _ptr(out),
            DTYPE_CODE[out.dtype], _ptr(workspace), workspace.numel(), _stream(stream),
            ctypes.byref(opts)))
        return out


# ------------------------------------------------------------------ prefix-aware decode
class _Groups:
    """Host arrays of a prefix-group description, kept alive with the struct."""

    def __init__(self, group_of_seq, group_prefix_blocks):
        self.gos = torch.as_tensor(list(group_of_seq), dtype=torch.int32).contiguous()
        self.gpb = torch.as_tensor(list(group_prefix_blocks), dtype=torch.int32).contiguous()
        self.st = PrefixGroups(len(self.gpb), self.gos.data_ptr() if len(self.gos) else None,
                               self.gpb.data_ptr() if len(self.gpb) else None)


def prefix_workspace_bytes(k_pool, num_seqs, num_q_heads, max_blocks_per_seq, group_of_seq,
                           group_prefix_blocks, num_ctas: int = 0) -> int:
    g = _Groups(group_of_seq, group_prefix_blocks)
    desc = cache_desc(k_pool)
    return int(lib().pkv_decode_prefix_workspace_bytes(ctypes.byref(desc), num_seqs, num_q_heads,
                                                       max_blocks_per_seq, ctypes.byref(g.st),
                                                       num_ctas))


def decode_attention_prefix(q, k_pool, v_pool, block_tables, context_lens, scale: float,
                            group_of_seq, group_prefix_blocks,
                            out: Optional[torch.Tensor] = None,
                            out_dtype: Optional[torch.dtype] = None,
                            workspace: Optional[torch.Tensor] = None, num_ctas: int = 0,
                            stream=None, lse_out: Optional[torch.Tensor] = None,
                            tables_ready: bool = False, consumer: int = 0) -> torch.Tensor:
    """Decode where the sequences of each group share their first
    group_prefix_blocks[g] table entries (group_of_seq[s] = g, or -1)."""
    return PreparedDecodePrefix(q, k_pool, v_pool, block_tables, context_lens, scale,
                                group_of_seq, group_prefix_blocks, out=out, out_dtype=out_dtype,
                                workspace=workspace, num_ctas=num_ctas, lse_out=lse_out,
                                tables_ready=tables_ready, consumer=consumer)(stream)


class PreparedDecodePrefix:
    """A pkv_decode_attention_prefix call whose arguments (and group arrays)
    are marshalled once; each call passes the stream (see PreparedDecode)."""

    def __init__(self, q, k_pool, v_pool, block_tables, context_lens, scale: float,
                 group_of_seq, group_prefix_blocks, out: Optional[torch.Tensor] = None,
                 out_dtype: Optional[torch.dtype] = None,
                 workspace: Optional[torch.Tensor] = None, num_ctas: int = 0,
                 lse_out: Optional[torch.Tensor] = None, tables_ready: bool = False,
                 consumer: int = 0):
        self._desc = _pools(k_pool, v_pool)
        S, Hq, D = q.shape
        q = q.contiguous()
        bt, cl = block_tables.contiguous(), context_lens.contiguous()
        assert bt.dtype == torch.int32 and cl.dtype == torch.int32 and q.dtype == k_pool.dtype
        self._g = _Groups(group_of_seq, group_prefix_blocks)
        if out is None:
            out = torch.empty(S, Hq, D, dtype=out_dtype or q.dtype, device=q.device)
        if workspace is None:
            n = prefix_workspace_bytes(k_pool, S, Hq, bt.shape[1], group_of_seq,
                                       group_prefix_blocks, num_ctas)
            if n == 0:
                raise PkvError(-1, lib().pkv_last_error_message().decode())
            workspace = torch.zeros(n, dtype=torch.uint8, device=q.device)
        self._opts = DecodeOptions()
        self._opts.num_ctas = num_ctas
        self._opts.consumer = consumer
        self._opts.tables_ready = int(tables_ready)
        if lse_out is not None:
            assert lse_out.dtype == torch.float32 and lse_out.shape == (S, Hq) and lse_out.is_contiguous()
            self._opts.lse_out = lse_out.data_ptr()
        self._keep = (q, k_pool, v_pool, bt, cl, out, workspace, lse_out)
        self._args = (ctypes.byref(self._desc), _ptr(q), S, Hq, _ptr(k_pool), _ptr(v_pool),
                      _ptr(bt), bt.shape[1], _ptr(cl), float(scale), ctypes.byref(self._g.st),
                      _ptr(out), DTYPE_CODE[out.dtype], _ptr(workspace), workspace.numel())
        self._fn = lib().pkv_decode_attention_prefix
        self.out = out
        self.workspace = workspace

    def __call__(self, stream=None, timing_events: Optional[Sequence] = None) -> torch.Tensor:
        opts = self._opts
        for i in range(2):
            ev = timing_events[i] if timing_events is not None else None
            opts.timing_events[i] = None if ev is None else ev.cuda_event
        _check(self._fn(*self._args, _stream(stream), ctypes.byref(opts)))
        return self.out


# ------------------------------------------------------------- device block tables
TABLES_WORKSPACE_BYTES = 64


def _ops_lib():
    """libpkv with the signatures of pkv_tables.h, pkv_rope.h, pkv_q4.h, pkv_sparse.h and pkv_tree.h."""
    L = lib()
    if not getattr(L, "_ops_ready", False):
        vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                 ctypes.c_size_t)
        dp, q4, pools = (ctypes.POINTER(CacheDesc), ctypes.POINTER(Q4CacheDesc),
                         ctypes.POINTER(Q4Pools))
        plan, sel = ctypes.POINTER(_RopePlan), ctypes.POINTER(SparseSelect)
        axes = ctypes.POINTER(_RopeAxesPlan)
        for name, args in {
            "pkv_tables_append": [i32, i32, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, i32, vp,
                                  vp, vp],
            "pkv_tables_release": [i32, i32, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp],
            "pkv_rope_plan_init": [ctypes.POINTER(RopeDesc), plan],
            "pkv_rope": [i32, i32, plan, vp, i32, vp, i64, i32, vp, i64, vp, i64, i32, vp, i64, vp],
            "pkv_rope_append": [dp, plan, vp, vp, i32, vp, i64, i32, vp, i64, vp, i64, vp, i64, vp,
                                vp, vp],
            "pkv_tables_truncate": [i32, i32, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp],
            "pkv_rope_axes_plan_init": [ctypes.POINTER(RopeAxesDesc), axes],
            "pkv_rope_axes": [i32, i32, axes, vp, i64, i32, vp, i64, i32, vp, i64, vp, i64, i32, vp, i64, vp],
            "pkv_rope_axes_append": [dp, axes, vp, i64, vp, i32, vp, i64, i32, vp, i64, vp, i64, vp, i64,
                                     vp, vp, vp],
            "pkv_tree_plan": [i32, i32, vp, vp, vp, vp, vp, i32, vp, i32, vp],
            "pkv_tree_accept": [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp],
            "pkv_tree_commit": [dp, i32, i32, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp],
            "pkv_decode_attention_tree": [dp, vp, i32, i32, vp, vp, vp, i32, i32, vp, vp, vp, i32, i32,
                                          f32, vp, i32, vp, sz, vp, ctypes.POINTER(TreeOptions)],
            "pkv_append_q4": [q4, vp, vp, vp, i32, pools, vp],
            "pkv_gather_q4": [q4, pools, vp, i32, vp, vp, i32, vp],
            "pkv_decode_attention_q4": [q4, vp, i32, i32, pools, vp, i32, vp, f32, vp, i32, vp, sz,
                                        vp, ctypes.POINTER(DecodeOptions)],
            "pkv_block_copy_q4": [q4, vp, i32, pools, vp],
            "pkv_block_means": [dp, vp, i32, vp, vp, vp],
            "pkv_select_blocks": [dp, vp, i32, i32, vp, vp, i32, vp, sel, vp, vp, vp, sz, vp],
            "pkv_decode_attention_sparse": [dp, vp, i32, i32, vp, vp, vp, vp, i32, vp, f32, sel, vp,
                                            vp, vp, i32, vp, sz, vp],
        }.items():
            getattr(L, name).argtypes = args
            getattr(L, name).restype = i32
        for name, args in {
            "pkv_decode_q4_workspace_bytes": [q4, i32, i32],
            "pkv_select_workspace_bytes": [dp, i32, i32],
            "pkv_decode_sparse_workspace_bytes": [dp, i32, i32, i32],
            "pkv_decode_tree_workspace_bytes": [dp, i32, i32, i32],
        }.items():
            getattr(L, name).argtypes = args
            getattr(L, name).restype = sz
        L._ops_ready = True
    return L


class PreparedCall:
    """A call whose arguments are checked and marshalled once, for repeated steps on stable
    buffers (the usual serving loop, and CUDA-graph capture): each call only passes the stream
    (None: the current one) and returns `out`. The buffers are kept alive by this object and
    rewritten in place by the caller between steps. Outputs and workspaces that the caller did
    not give are made on the stream that was current at construction."""

    def __init__(self, name: str, args, keep, out=None, after=()):
        self._fn = getattr(_ops_lib(), name)
        self._device = _one_gpu(name, keep)
        # plain numbers become ctypes objects once, not at each call
        kinds = self._fn.argtypes
        self._args = tuple(k(a) if a is None or isinstance(a, (int, float)) else a
                           for k, a in zip(kinds, args))
        self._after, self._keep, self.out = tuple(after), keep, out

    def __call__(self, stream=None):
        raw = _raw_stream(self._device) if stream is None else _stream(stream)
        if torch.cuda.current_device() != self._device:
            with torch.cuda.device(self._device):
                _check(self._fn(*self._args, raw, *self._after))
        else:
            status = self._fn(*self._args, raw, *self._after)
            if status:
                _check(status)
        return self.out


def _one_gpu(name: str, keep) -> int:
    """The GPU that all tensors and caches of a call lie on."""
    devices = {t.device for t in keep if isinstance(t, torch.Tensor)}
    for c in keep:
        if isinstance(c, Q4Cache):
            devices |= {t.device for t in (c.k_codes, c.v_codes, c.k_params, c.v_params)}
    if len(devices) != 1 or next(iter(devices)).type != "cuda":
        raise ValueError(f"{name}: the tensors are not on one GPU ({sorted(map(str, devices))})")
    return next(iter(devices)).index


def _on(stream, device):
    """For one-shot calls: what they allocate (outputs, zero-filled workspaces) is made on the stream
    that the call runs on, so that it is filled before and not handed on before the call is done."""
    if stream is None or device.type != "cuda":
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device)
    return torch.cuda.stream(stream)


def _raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# the current stream's handle without a Stream object around it (1 us less a call), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _need(t: torch.Tensor, name: str, dtype, shape=None) -> torch.Tensor:
    """`t`, which has to be contiguous, of this dtype and (None: any) shape."""
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, not {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    return t


def alloc_tables_workspace(device="cuda") -> torch.Tensor:
    """Zero-filled workspace of tables_append / tables_release; one for calls that may overlap."""
    return torch.zeros(TABLES_WORKSPACE_BYTES, dtype=torch.uint8, device=device)


def _tables_state(block_tables, context_lens, free_blocks, num_free, context_lens_out, num_free_out):
    S, M = block_tables.shape
    i32 = torch.int32
    _need(block_tables, "block_tables", i32)
    _need(context_lens, "context_lens", i32, (S,))
    _need(free_blocks, "free_blocks", i32)
    _need(num_free, "num_free", i32, (1,))
    lens_out = context_lens if context_lens_out is None else context_lens_out
    free_out = num_free if num_free_out is None else num_free_out
    _need(lens_out, "context_lens_out", i32, (S,))
    _need(free_out, "num_free_out", i32, (1,))
    return S, M, free_blocks.numel(), lens_out, free_out


def prepared_tables_append(block_tables, context_lens, new_tokens, free_blocks, num_free,
                           block_size: int, slot_mapping, positions, token_offsets, workspace,
                           context_lens_out: Optional[torch.Tensor] = None,
                           num_free_out: Optional[torch.Tensor] = None) -> PreparedCall:
    """tables_append as a PreparedCall."""
    S, M, NB, lens_out, free_out = _tables_state(block_tables, context_lens, free_blocks, num_free,
                                                 context_lens_out, num_free_out)
    _need(new_tokens, "new_tokens", torch.int32, (S,))
    _need(slot_mapping, "slot_mapping", torch.int64)
    n = slot_mapping.numel()
    _need(positions, "positions", torch.int32, (n,))
    _need(token_offsets, "token_offsets", torch.int32, (S + 1,))
    if workspace.numel() * workspace.element_size() < TABLES_WORKSPACE_BYTES:
        raise ValueError("workspace is too small")
    return PreparedCall("pkv_tables_append", (
        NB, block_size, S, _ptr(new_tokens), _ptr(block_tables), M, _ptr(context_lens), _ptr(lens_out),
        _ptr(free_blocks), _ptr(num_free), _ptr(free_out), _ptr(slot_mapping), _ptr(positions), n,
        _ptr(token_offsets), _ptr(workspace)),
        keep=(block_tables, context_lens, new_tokens, free_blocks, num_free, lens_out, free_out,
              slot_mapping, positions, token_offsets, workspace),
        out=(slot_mapping, positions, token_offsets))


def tables_append(block_tables, context_lens, new_tokens, free_blocks, num_free, block_size: int,
                  slot_mapping, positions, token_offsets, workspace,
                  context_lens_out: Optional[torch.Tensor] = None,
                  num_free_out: Optional[torch.Tensor] = None, stream=None):
    """Blocks and slots of one step's new tokens, on the device (pkv_tables_append): fills
    slot_mapping / positions [max_tokens] and token_offsets [S + 1], writes the new blocks
    into block_tables [S][M], and updates the lengths and the free count (in place unless
    the *_out tensors are given). free_blocks [num_blocks] is the stack of free blocks.
    What it writes is never ready in the sense of tables_ready or inputs_ready for calls that
    follow on the stream (pkv_tables.h). Returns the three outputs."""
    return prepared_tables_append(block_tables, context_lens, new_tokens, free_blocks, num_free,
                                  block_size, slot_mapping, positions, token_offsets, workspace,
                                  context_lens_out, num_free_out)(stream)


def prepared_tables_release(block_tables, context_lens, released, free_blocks, num_free,
                            block_size: int, workspace,
                            context_lens_out: Optional[torch.Tensor] = None,
                            num_free_out: Optional[torch.Tensor] = None) -> PreparedCall:
    """tables_release as a PreparedCall."""
    S, M, NB, lens_out, free_out = _tables_state(block_tables, context_lens, free_blocks, num_free,
                                                 context_lens_out, num_free_out)
    _need(released, "released", torch.bool if released.dtype == torch.bool else torch.uint8, (S,))
    if workspace.numel() * workspace.element_size() < TABLES_WORKSPACE_BYTES:
        raise ValueError("workspace is too small")
    return PreparedCall("pkv_tables_release", (
        NB, block_size, S, _ptr(released), _ptr(block_tables), M, _ptr(context_lens), _ptr(lens_out),
        _ptr(free_blocks), _ptr(num_free), _ptr(free_out), _ptr(workspace)),
        keep=(block_tables, context_lens, released, free_blocks, num_free, lens_out, free_out, workspace),
        out=None)


def tables_release(block_tables, context_lens, released, free_blocks, num_free, block_size: int,
                   workspace, context_lens_out: Optional[torch.Tensor] = None,
                   num_free_out: Optional[torch.Tensor] = None, stream=None) -> None:
    """Push the blocks of the requests with released[s] (bool or uint8 [S]) onto the stack of
    free blocks and set their lengths to 0 (pkv_tables_release)."""
    return prepared_tables_release(block_tables, context_lens, released, free_blocks, num_free,
                                   block_size, workspace, context_lens_out, num_free_out)(stream)


def prepared_tables_truncate(block_tables, context_lens, kept_lens, free_blocks, num_free,
                             block_size: int, workspace,
                             context_lens_out: Optional[torch.Tensor] = None,
                             num_free_out: Optional[torch.Tensor] = None) -> PreparedCall:
    """tables_truncate as a PreparedCall."""
    S, M, NB, lens_out, free_out = _tables_state(block_tables, context_lens, free_blocks, num_free,
                                                 context_lens_out, num_free_out)
    _need(kept_lens, "kept_lens", torch.int32, (S,))
    if workspace.numel() * workspace.element_size() < TABLES_WORKSPACE_BYTES:
        raise ValueError("workspace is too small")
    return PreparedCall("pkv_tables_truncate", (
        NB, block_size, S, _ptr(kept_lens), _ptr(block_tables), M, _ptr(context_lens), _ptr(lens_out),
        _ptr(free_blocks), _ptr(num_free), _ptr(free_out), _ptr(workspace)),
        keep=(block_tables, context_lens, kept_lens, free_blocks, num_free, lens_out, free_out, workspace),
        out=None)


def tables_truncate(block_tables, context_lens, kept_lens, free_blocks, num_free, block_size: int,
                    workspace, context_lens_out: Optional[torch.Tensor] = None,
                    num_free_out: Optional[torch.Tensor] = None, stream=None) -> None:
    """Shorten each request to its first kept_lens[s] tokens (int32 [S], at most its length) and push
    the blocks behind them onto the stack of free blocks (pkv_tables_truncate)."""
    return prepared_tables_truncate(block_tables, context_lens, kept_lens, free_blocks, num_free,
                                    block_size, workspace, context_lens_out, num_free_out)(stream)


# ------------------------------------------------------------------ rotary positions
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "yarn": 4}


class RopeDesc(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("original_len", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("low_freq_factor", ctypes.c_double), ("high_freq_factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("attention_factor", ctypes.c_double)]


class _RopePlan(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turns", ctypes.c_uint64 * 64)]


class RopePlan:
    """Frequencies of a rotary embedding, made once (pkv_rope_plan_init). layout: "half" or
    "interleaved"; scaling: "none", "linear", "base", "bands" or "yarn" (include/pkv_rope.h)."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, layout: str = "half",
                 scaling: str = "none", factor: float = 1.0, original_len: int = 0,
                 low_freq_factor: float = 1.0, high_freq_factor: float = 4.0, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, attention_factor: float = 0.0):
        desc = RopeDesc(rotary_dim, ROPE_LAYOUTS[layout], ROPE_SCALINGS[scaling], original_len, base, factor,
                        low_freq_factor, high_freq_factor, beta_fast, beta_slow, attention_factor)
        self.c = _RopePlan()
        _check(_ops_lib().pkv_rope_plan_init(ctypes.byref(desc), ctypes.byref(self.c)))


def _heads(t: torch.Tensor, name: str, dtype=None, rows=None):
    """(heads, token stride) of a [T][H][D] tensor whose heads are contiguous."""
    if t.dim() != 3 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]) or t.stride(2) != 1:
        raise ValueError(f"{name} must be [tokens][heads][head_dim] with each token's heads contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, not {dtype}")
    if rows is not None and t.shape[0] != rows:
        raise ValueError(f"{name} has {t.shape[0]} tokens, not {rows}")
    # the stride of a single token says nothing
    return t.shape[1], t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def prepared_rope(q, k, positions, plan: RopePlan, q_out: Optional[torch.Tensor] = None,
                  k_out: Optional[torch.Tensor] = None) -> PreparedCall:
    """rope as a PreparedCall."""
    T, _, D = q.shape
    (Hq, qs), (Hk, ks) = _heads(q, "q"), _heads(k, "k", q.dtype, T)
    if k.shape[2] != D:
        raise ValueError("q and k differ in head_dim")
    q_out = torch.empty(T, Hq, D, dtype=q.dtype, device=q.device) if q_out is None else q_out
    k_out = torch.empty(T, Hk, D, dtype=q.dtype, device=q.device) if k_out is None else k_out
    if q_out.shape != q.shape or k_out.shape != k.shape:
        raise ValueError("q_out and k_out have the shapes of q and k")
    (_, qos), (_, kos) = _heads(q_out, "q_out", q.dtype, T), _heads(k_out, "k_out", q.dtype, T)
    _need(positions, "positions", torch.int32, (T,))
    return PreparedCall("pkv_rope", (
        DTYPE_CODE[q.dtype], D, ctypes.byref(plan.c), _ptr(positions), T, _ptr(q), qs,
                               Hq, _ptr(q_out), qos, _ptr(k), ks, Hk, _ptr(k_out), kos),
        keep=(q, k, positions, plan, q_out, k_out),
        out=(q_out, k_out))


def rope(q, k, positions, plan: RopePlan, q_out: Optional[torch.Tensor] = None,
         k_out: Optional[torch.Tensor] = None, stream=None):
    """q [T][Hq][D] and k [T][Hk][D] (token-strided views allowed) turned to their positions
    (int32 [T]); into new tensors unless q_out / k_out are given (q and k themselves allowed)."""
    with _on(stream, q.device):
        return prepared_rope(q, k, positions, plan, q_out, k_out)(stream)


def prepared_rope_append(q, k_new, v_new, positions, slot_mapping, plan: RopePlan, k_pool, v_pool,
                         q_out: Optional[torch.Tensor] = None) -> PreparedCall:
    """rope_append as a PreparedCall."""
    desc = _pools(k_pool, v_pool)
    T, _, D = q.shape
    dt = k_pool.dtype
    (Hq, qs), (Hk, ks), (Hv, vs) = _heads(q, "q", dt), _heads(k_new, "k_new", dt, T), _heads(v_new, "v_new", dt, T)
    if Hk != desc.num_kv_heads or Hv != Hk or not D == k_new.shape[2] == v_new.shape[2] == desc.head_dim:
        raise ValueError("q, k_new or v_new do not fit the pools")
    q_out = torch.empty(T, Hq, D, dtype=dt, device=q.device) if q_out is None else q_out
    if q_out.shape != q.shape:
        raise ValueError("q_out has the shape of q")
    _, qos = _heads(q_out, "q_out", dt, T)
    _need(positions, "positions", torch.int32, (T,))
    _need(slot_mapping, "slot_mapping", torch.int64, (T,))
    return PreparedCall("pkv_rope_append", (
        ctypes.byref(desc), ctypes.byref(plan.c), _ptr(positions), _ptr(slot_mapping), T, _ptr(q), qs, Hq,
        _ptr(q_out), qos, _ptr(k_new), ks, _ptr(v_new), vs, _ptr(k_pool), _ptr(v_pool)),
        keep=(q, k_new, v_new, positions, slot_mapping, plan, k_pool, v_pool, q_out, desc),
        out=q_out)


def rope_append(q, k_new, v_new, positions, slot_mapping, plan: RopePlan, k_pool, v_pool,
                q_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """rope and append in one launch (pkv_rope_append): returns the turned q; the turned k and
    v go to slot_mapping [T] (int64). q, k_new, v_new: [T][heads][D], token-strided views allowed."""
    with _on(stream, q.device):
        return prepared_rope_append(q, k_new, v_new, positions, slot_mapping, plan, k_pool, v_pool,
                                    q_out)(stream)


ROPE_ORDERS = {"sections": 0, "cycled": 1}
ROPE_FREQUENCIES = {"shared": 0, "own": 1}


class RopeAxesDesc(ctypes.Structure):
    _fields_ = [("rope", RopeDesc), ("num_axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 4),
                ("order", ctypes.c_int32), ("frequencies", ctypes.c_int32)]


class _RopeAxesPlan(ctypes.Structure):
    _fields_ = [("plan", _RopePlan), ("num_axes", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("axis", ctypes.c_uint8 * 64)]


class RopeAxesPlan:
    """A rotary embedding whose pairs turn by the positions of several axes (pkv_rope_axes_plan_init):
    sections[a] pairs for axis a, "sections" (one axis's pairs after another's) or "cycled" (dealt out in
    turn); frequencies "shared" (of the whole embedding) or "own" (each axis's own). The rest as RopePlan;
    the rotated part of a head is twice the sum of the sections."""

    def __init__(self, sections, order: str = "sections", frequencies: str = "shared", base: float = 10000.0,
                 layout: str = "half", scaling: str = "none", factor: float = 1.0, original_len: int = 0,
                 low_freq_factor: float = 1.0, high_freq_factor: float = 4.0, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, attention_factor: float = 0.0):
        sections = [int(n) for n in sections]
        if not 1 <= len(sections) <= 4:
            raise ValueError(f"{len(sections)} axes (1 to 4)")
        rope = RopeDesc(2 * sum(sections), ROPE_LAYOUTS[layout], ROPE_SCALINGS[scaling], original_len, base,
                        factor, low_freq_factor, high_freq_factor, beta_fast, beta_slow, attention_factor)
        desc = RopeAxesDesc(rope, len(sections), (ctypes.c_int32 * 4)(*sections), ROPE_ORDERS[order],
                            ROPE_FREQUENCIES[frequencies])
        self.c = _RopeAxesPlan()
        _check(_ops_lib().pkv_rope_axes_plan_init(ctypes.byref(desc), ctypes.byref(self.c)))


def _axes_positions(positions, plan: RopeAxesPlan, T: int) -> int:
    """The stride from one axis's positions to the next's."""
    if positions.dtype != torch.int32 or positions.dim() != 2 or tuple(positions.shape) != (plan.c.num_axes, T):
        raise ValueError(f"positions must be int32 [{plan.c.num_axes}][{T}]")
    if T > 1 and positions.stride(1) != 1:
        raise ValueError("positions: each axis's must be contiguous")
    return positions.stride(0)


def prepared_rope_axes(q, k, positions, plan: RopeAxesPlan, q_out: Optional[torch.Tensor] = None,
                       k_out: Optional[torch.Tensor] = None) -> PreparedCall:
    """rope_axes as a PreparedCall."""
    T, _, D = q.shape
    (Hq, qs), (Hk, ks) = _heads(q, "q"), _heads(k, "k", q.dtype, T)
    if k.shape[2] != D:
        raise ValueError("q and k differ in head_dim")
    q_out = torch.empty(T, Hq, D, dtype=q.dtype, device=q.device) if q_out is None else q_out
    k_out = torch.empty(T, Hk, D, dtype=q.dtype, device=q.device) if k_out is None else k_out
    if q_out.shape != q.shape or k_out.shape != k.shape:
        raise ValueError("q_out and k_out have the shapes of q and k")
    (_, qos), (_, kos) = _heads(q_out, "q_out", q.dtype, T), _heads(k_out, "k_out", q.dtype, T)
    ps = _axes_positions(positions, plan, T)
    return PreparedCall("pkv_rope_axes", (
        DTYPE_CODE[q.dtype], D, ctypes.byref(plan.c), _ptr(positions), ps, T, _ptr(q), qs, Hq, _ptr(q_out), qos,
        _ptr(k), ks, Hk, _ptr(k_out), kos),
        keep=(q, k, positions, plan, q_out, k_out), out=(q_out, k_out))


def rope_axes(q, k, positions, plan: RopeAxesPlan, q_out: Optional[torch.Tensor] = None,
              k_out: Optional[torch.Tensor] = None, stream=None):
    """rope with a position on each axis: positions int32 [axes][T] (pkv_rope_axes)."""
    with _on(stream, q.device):
        return prepared_rope_axes(q, k, positions, plan, q_out, k_out)(stream)


def prepared_rope_axes_append(q, k_new, v_new, positions, slot_mapping, plan: RopeAxesPlan, k_pool, v_pool,
                              q_out: Optional[torch.Tensor] = None) -> PreparedCall:
    """rope_axes_append as a PreparedCall."""
    desc = _pools(k_pool, v_pool)
    T, _, D = q.shape
    dt = k_pool.dtype
    (Hq, qs), (Hk, ks), (Hv, vs) = _heads(q, "q", dt), _heads(k_new, "k_new", dt, T), _heads(v_new, "v_new", dt, T)
    if Hk != desc.num_kv_heads or Hv != Hk or not D == k_new.shape[2] == v_new.shape[2] == desc.head_dim:
        raise ValueError("q, k_new or v_new do not fit the pools")
    q_out = torch.empty(T, Hq, D, dtype=dt, device=q.device) if q_out is None else q_out
    if q_out.shape != q.shape:
        raise ValueError("q_out has the shape of q")
    _, qos = _heads(q_out, "q_out", dt, T)
    ps = _axes_positions(positions, plan, T)
    _need(slot_mapping, "slot_mapping", torch.int64, (T,))
    return PreparedCall("pkv_rope_axes_append", (
        ctypes.byref(desc), ctypes.byref(plan.c), _ptr(positions), ps, _ptr(slot_mapping), T, _ptr(q), qs, Hq,
        _ptr(q_out), qos, _ptr(k_new), ks, _ptr(v_new), vs, _ptr(k_pool), _ptr(v_pool)),
        keep=(q, k_new, v_new, positions, slot_mapping, plan, k_pool, v_pool, q_out, desc), out=q_out)


def rope_axes_append(q, k_new, v_new, positions, slot_mapping, plan: RopeAxesPlan, k_pool, v_pool,
                     q_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """rope_append with a position on each axis: positions int32 [axes][T] (pkv_rope_axes_append)."""
    with _on(stream, q.device):
        return prepared_rope_axes_append(q, k_new, v_new, positions, slot_mapping, plan, k_pool, v_pool,
                                         q_out)(stream)


# ---------------------------------------------------------------------- drafted tokens
TREE_MAX_TOKENS = 256


class TreeOptions(ctypes.Structure):
    _fields_ = [("num_ctas", ctypes.c_int32), ("reserved", ctypes.c_int32), ("lse_out", ctypes.c_void_p)]


def _tree_batch(parents, token_offsets, context_lens, T: int) -> int:
    S = context_lens.shape[0]
    if parents is not None:
        _need(parents, "parents", torch.int32, (T,))
    _need(token_offsets, "token_offsets", torch.int32, (S + 1,))
    _need(context_lens, "context_lens", torch.int32, (S,))
    return S


def _mask_words(masks, T: int) -> int:
    if masks.dim() != 2 or not 1 <= masks.shape[1] <= 4:
        raise ValueError("masks must be int64 [tokens][1 to 4 words]")
    _need(masks, "masks", torch.int64, (T, masks.shape[1]))
    return masks.shape[1]


def prepared_tree_plan(parents, token_offsets, context_lens, masks=None, positions=None,
                       position_deltas: Optional[torch.Tensor] = None, mask_words: int = 4) -> PreparedCall:
    """tree_plan as a PreparedCall."""
    if masks is None and positions is None:
        raise ValueError("neither masks nor positions to write")
    T = masks.shape[0] if masks is not None else positions.shape[-1]
    S = _tree_batch(parents, token_offsets, context_lens, T)
    words = mask_words if masks is None else _mask_words(masks, T)
    axes = 1
    if positions is not None:
        axes = positions.shape[0] if positions.dim() == 2 else 1
        _need(positions, "positions", torch.int32, (axes, T) if positions.dim() == 2 else (T,))
    if position_deltas is not None:
        _need(position_deltas, "position_deltas", torch.int32, (S,))
    return PreparedCall("pkv_tree_plan", (
        S, T, _ptr(parents), _ptr(token_offsets), _ptr(context_lens), _ptr(position_deltas), _ptr(masks), words,
        _ptr(positions), axes),
        keep=(parents, token_offsets, context_lens, position_deltas, masks, positions), out=(masks, positions))


def tree_plan(parents, token_offsets, context_lens, masks=None, positions=None,
              position_deltas: Optional[torch.Tensor] = None, mask_words: int = 4, stream=None):
    """Masks (int64 [T][words]) and positions (int32 [T] or [axes][T]) of drafted tokens from their
    parents (int32 [T], None: chains); either output may be None (pkv_tree_plan). Returns both."""
    return prepared_tree_plan(parents, token_offsets, context_lens, masks, positions, position_deltas,
                              mask_words)(stream)


def tree_workspace_bytes(k_pool, num_q_heads: int, max_tree: int, num_ctas: int = 0) -> int:
    with torch.cuda.device(k_pool.device):
        return int(_ops_lib().pkv_decode_tree_workspace_bytes(ctypes.byref(cache_desc(k_pool)), num_q_heads, max_tree,
                                                              num_ctas))


def alloc_tree_workspace(k_pool, num_q_heads: int, max_tree: int, num_ctas: int = 0) -> torch.Tensor:
    """Workspace of decode_attention_tree, zeroed on the current stream. Every call leaves it fit for the
    next (after DEVERR_TIMEOUT it has to be zeroed again); calls that may overlap need one each."""
    n = tree_workspace_bytes(k_pool, num_q_heads, max_tree, num_ctas)
    if n == 0:
        raise PkvError(-1, lib().pkv_last_error_message().decode())
    return torch.zeros(n, dtype=torch.uint8, device=k_pool.device)


def prepared_decode_attention_tree(q, k_pool, v_pool, block_tables, context_lens, token_offsets, masks,
                                   scale: float, max_tree: int, out: Optional[torch.Tensor] = None,
                                   out_dtype: Optional[torch.dtype] = None,
                                   workspace: Optional[torch.Tensor] = None, num_ctas: int = 0,
                                   lse_out: Optional[torch.Tensor] = None) -> PreparedCall:
    """decode_attention_tree as a PreparedCall."""
    desc = _pools(k_pool, v_pool)
    T, Hq, D = q.shape
    _need(q, "q", k_pool.dtype, (T, Hq, desc.head_dim))
    S = _tree_batch(None, token_offsets, context_lens, T)
    _need(block_tables, "block_tables", torch.int32, (S, block_tables.shape[-1]))
    words = 0 if masks is None else _mask_words(masks, T)
    if out is None:
        out = torch.empty(T, Hq, D, dtype=out_dtype or q.dtype, device=q.device)
    _need(out, "out", out.dtype, q.shape)
    if workspace is None:
        workspace = alloc_tree_workspace(k_pool, Hq, max_tree, num_ctas)
    opts = TreeOptions(num_ctas, 0, None)
    if lse_out is not None:
        opts.lse_out = _need(lse_out, "lse_out", torch.float32, (T, Hq)).data_ptr()
    return PreparedCall("pkv_decode_attention_tree", (
        ctypes.byref(desc), _ptr(q), T, Hq, _ptr(k_pool), _ptr(v_pool), _ptr(block_tables), S, block_tables.shape[1],
        _ptr(context_lens), _ptr(token_offsets), _ptr(masks), words, max_tree, float(scale), _ptr(out),
        DTYPE_CODE[out.dtype], _ptr(workspace), workspace.numel() * workspace.element_size()),
        keep=(q, k_pool, v_pool, block_tables, context_lens, token_offsets, masks, out, workspace, lse_out, opts,
              desc),
        out=out, after=(ctypes.byref(opts),))


def decode_attention_tree(q, k_pool, v_pool, block_tables, context_lens, token_offsets, masks, scale: float,
                          max_tree: int, out: Optional[torch.Tensor] = None,
                          out_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None,
                          num_ctas: int = 0, lse_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of all drafted tokens over the cache, whose last tokens they are: q [T][Hq][D], one
    sequence's tokens after another's (token_offsets int32 [S + 1]), each sees the context before them
    and the drafted tokens of its mask (int64 [T][words]; None: chains). max_tree: tokens a sequence at
    most (pkv_decode_attention_tree)."""
    with _on(stream, q.device):
        return prepared_decode_attention_tree(q, k_pool, v_pool, block_tables, context_lens, token_offsets, masks,
                                              scale, max_tree, out, out_dtype, workspace, num_ctas,
                                              lse_out)(stream)


def prepared_tree_accept(parents, tokens, targets, token_offsets, context_lens, path, counts, next_tokens,
                         context_lens_out, max_tree: int) -> PreparedCall:
    """tree_accept as a PreparedCall."""
    T = tokens.shape[0]
    S = _tree_batch(parents, token_offsets, context_lens, T)
    for name, t, n in (("tokens", tokens, T), ("targets", targets, T), ("path", path, T), ("counts", counts, S),
                       ("next_tokens", next_tokens, S), ("context_lens_out", context_lens_out, S)):
        _need(t, name, torch.int32, (n,))
    return PreparedCall("pkv_tree_accept", (
        S, T, max_tree, _ptr(parents), _ptr(tokens), _ptr(targets), _ptr(token_offsets), _ptr(context_lens),
        _ptr(path), _ptr(counts), _ptr(next_tokens), _ptr(context_lens_out)),
        keep=(parents, tokens, targets, token_offsets, context_lens, path, counts, next_tokens, context_lens_out),
        out=(path, counts, next_tokens, context_lens_out))


def tree_accept(parents, tokens, targets, token_offsets, context_lens, max_tree: int,
                path: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                next_tokens: Optional[torch.Tensor] = None, context_lens_out: Optional[torch.Tensor] = None,
                stream=None):
    """The branch of each sequence's drafted tokens (int32 [T]) that the model's answers (targets) confirm
    (pkv_tree_accept): (path [T], counts [S], next_tokens [S], context_lens_out [S]), new tensors unless
    given. A new path is -1 past the last sequence's rows too."""
    with _on(stream, tokens.device):
        i32 = dict(dtype=torch.int32, device=tokens.device)
        S = context_lens.shape[0]
        path = torch.full(tokens.shape, -1, **i32) if path is None else path
        counts, next_tokens, context_lens_out = (torch.empty(S, **i32) if t is None else t
                                                 for t in (counts, next_tokens, context_lens_out))
        return prepared_tree_accept(parents, tokens, targets, token_offsets, context_lens, path, counts, next_tokens,
                                    context_lens_out, max_tree)(stream)


def prepared_tree_commit(path, counts, token_offsets, context_lens, block_tables, k_pool, v_pool,
                         max_tree: int) -> PreparedCall:
    """tree_commit as a PreparedCall."""
    desc = _pools(k_pool, v_pool)
    T = path.shape[0]
    S = _tree_batch(None, token_offsets, context_lens, T)
    _need(path, "path", torch.int32, (T,))
    _need(counts, "counts", torch.int32, (S,))
    _need(block_tables, "block_tables", torch.int32, (S, block_tables.shape[-1]))
    return PreparedCall("pkv_tree_commit", (
        ctypes.byref(desc), S, T, max_tree, _ptr(path), _ptr(counts), _ptr(token_offsets), _ptr(context_lens),
        _ptr(block_tables), block_tables.shape[1], _ptr(k_pool), _ptr(v_pool)),
        keep=(path, counts, token_offsets, context_lens, block_tables, k_pool, v_pool, desc), out=None)


def tree_commit(path, counts, token_offsets, context_lens, block_tables, k_pool, v_pool, max_tree: int,
                stream=None) -> None:
    """Move the accepted drafted rows of each sequence together in the cache, behind its context
    (pkv_tree_commit). context_lens: the lengths that count all drafted tokens."""
    return prepared_tree_commit(path, counts, token_offsets, context_lens, block_tables, k_pool, v_pool,
                                max_tree)(stream)


# --------------------------------------------------------------------- 4-bit KV cache
class Q4CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32)]


class Q4Pools(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_params", ctypes.c_void_p), ("v_params", ctypes.c_void_p)]


class Q4Cache:
    """A 4-bit K/V cache (include/pkv_q4.h): code pools [NB][Hk][B][D/2] uint8, K parameters
    [NB][Hk][B][2 NG] and V parameters [NB][Hk][2 NG][B] fp16, NG = D / 32."""

    def __init__(self, k_codes, v_codes, k_params, v_params, act_dtype: torch.dtype):
        NB, Hk, B, half = k_codes.shape
        NG = half // 16
        _need(k_codes, "k_codes", torch.uint8)
        _need(v_codes, "v_codes", torch.uint8, k_codes.shape)
        _need(k_params, "k_params", torch.float16, (NB, Hk, B, 2 * NG))
        _need(v_params, "v_params", torch.float16, (NB, Hk, 2 * NG, B))
        self.k_codes, self.v_codes, self.k_params, self.v_params = k_codes, v_codes, k_params, v_params
        self.act_dtype = act_dtype
        self.desc = Q4CacheDesc(NB, B, Hk, 2 * half, DTYPE_CODE[act_dtype])
        self.pools = Q4Pools(k_codes.data_ptr(), v_codes.data_ptr(), k_params.data_ptr(),
                             v_params.data_ptr())

    @classmethod
    def empty(cls, num_blocks, num_kv_heads, block_size, head_dim, act_dtype=torch.bfloat16,
              device="cuda") -> "Q4Cache":
        NG = head_dim // 32
        codes = [torch.zeros(num_blocks, num_kv_heads, block_size, head_dim // 2, dtype=torch.uint8,
                             device=device) for _ in range(2)]
        return cls(*codes, torch.zeros(num_blocks, num_kv_heads, block_size, 2 * NG, dtype=torch.float16,
                                       device=device),
                   torch.zeros(num_blocks, num_kv_heads, 2 * NG, block_size, dtype=torch.float16,
                               device=device), act_dtype)

    def head_view(self) -> "Q4Cache":
        """The same memory as a pool of one-head blocks [NB * Hk][1], for the tables of select_blocks."""
        NB, Hk = self.k_codes.shape[:2]
        return Q4Cache(*(t.view(NB * Hk, 1, *t.shape[2:]) for t in
                         (self.k_codes, self.v_codes, self.k_params, self.v_params)), self.act_dtype)


def prepared_append_q4(k_new, v_new, slot_mapping, cache: Q4Cache) -> PreparedCall:
    """append_q4 as a PreparedCall."""
    d = cache.desc
    _need(slot_mapping, "slot_mapping", torch.int64)
    shape = (slot_mapping.numel(), d.num_kv_heads, d.head_dim)
    _need(k_new, "k_new", cache.act_dtype, shape)
    _need(v_new, "v_new", cache.act_dtype, shape)
    return PreparedCall("pkv_append_q4", (
        ctypes.byref(d), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), shape[0],
                                    ctypes.byref(cache.pools)),
        keep=(k_new, v_new, slot_mapping, cache),
        out=None)


def append_q4(k_new, v_new, slot_mapping, cache: Q4Cache, stream=None) -> None:
    """Quantize k_new/v_new [T][Hk][D] into the cache at slot_mapping [T] (int64)."""
    return prepared_append_q4(k_new, v_new, slot_mapping, cache)(stream)


def prepared_gather_q4(slot_mapping, cache: Q4Cache, k_out: Optional[torch.Tensor] = None,
                       v_out: Optional[torch.Tensor] = None,
                       out_dtype: Optional[torch.dtype] = None) -> PreparedCall:
    """gather_q4 as a PreparedCall."""
    d = cache.desc
    _need(slot_mapping, "slot_mapping", torch.int64)
    shape = (slot_mapping.numel(), d.num_kv_heads, d.head_dim)
    dt = k_out.dtype if k_out is not None else out_dtype or cache.act_dtype
    k_out = torch.empty(shape, dtype=dt, device=cache.k_codes.device) if k_out is None else k_out
    v_out = torch.empty(shape, dtype=dt, device=cache.k_codes.device) if v_out is None else v_out
    _need(k_out, "k_out", dt, shape)
    _need(v_out, "v_out", dt, shape)
    return PreparedCall("pkv_gather_q4", (
        ctypes.byref(d), ctypes.byref(cache.pools), _ptr(slot_mapping), shape[0],
                                    _ptr(k_out), _ptr(v_out), DTYPE_CODE[dt]),
        keep=(slot_mapping, cache, k_out, v_out),
        out=(k_out, v_out))


def gather_q4(slot_mapping, cache: Q4Cache, k_out: Optional[torch.Tensor] = None,
              v_out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None, stream=None):
    """The cached rows at slot_mapping [T] as values: (k, v) [T][Hk][D]."""
    with _on(stream, slot_mapping.device):
        return prepared_gather_q4(slot_mapping, cache, k_out, v_out, out_dtype)(stream)


def q4_workspace_bytes(cache: Q4Cache, num_q_heads: int, num_ctas: int = 0) -> int:
    return int(_ops_lib().pkv_decode_q4_workspace_bytes(ctypes.byref(cache.desc), num_q_heads, num_ctas))


def alloc_q4_workspace(cache: Q4Cache, num_q_heads: int, num_ctas: int = 0) -> torch.Tensor:
    """Zero-filled workspace of decode_attention_q4 (every call leaves its counters zero)."""
    n = q4_workspace_bytes(cache, num_q_heads, num_ctas)
    if n == 0:
        raise PkvError(-1, "workspace size query failed")
    return torch.zeros(n, dtype=torch.uint8, device=cache.k_codes.device)


def prepared_decode_attention_q4(q, cache: Q4Cache, block_tables, context_lens, scale: float,
                                 out: Optional[torch.Tensor] = None,
                                 out_dtype: Optional[torch.dtype] = None,
                                 workspace: Optional[torch.Tensor] = None, num_ctas: int = 0,
                                 lse_out: Optional[torch.Tensor] = None,
                                 tables_ready: bool = False,
                                 timing_events: Optional[Sequence] = None) -> PreparedCall:
    """decode_attention_q4 as a PreparedCall."""
    d = cache.desc
    S, Hq, D = q.shape
    _need(q, "q", cache.act_dtype, (S, Hq, d.head_dim))
    _need(block_tables, "block_tables", torch.int32, (S, block_tables.shape[-1]))
    _need(context_lens, "context_lens", torch.int32, (S,))
    if out is None:
        out = torch.empty(S, Hq, D, dtype=out_dtype or q.dtype, device=q.device)
    _need(out, "out", out.dtype, q.shape)
    if workspace is None:
        workspace = alloc_q4_workspace(cache, Hq, num_ctas)
    opts = DecodeOptions()
    opts.num_ctas = num_ctas
    opts.tables_ready = int(tables_ready)
    if timing_events is not None:
        for i, ev in enumerate(timing_events):
            opts.timing_events[i] = None if ev is None else ev.cuda_event
    if lse_out is not None:
        opts.lse_out = _need(lse_out, "lse_out", torch.float32, (S, Hq)).data_ptr()
    return PreparedCall("pkv_decode_attention_q4", (
        ctypes.byref(d), _ptr(q), S, Hq, ctypes.byref(cache.pools), _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), float(scale), _ptr(out), DTYPE_CODE[out.dtype], _ptr(workspace),
        workspace.numel() * workspace.element_size()),
        keep=(q, cache, block_tables, context_lens, out, workspace, lse_out, opts),
        out=out, after=(ctypes.byref(opts),))


def decode_attention_q4(q, cache: Q4Cache, block_tables, context_lens, scale: float,
                        out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                        workspace: Optional[torch.Tensor] = None, num_ctas: int = 0, stream=None,
                        lse_out: Optional[torch.Tensor] = None, tables_ready: bool = False,
                        timing_events: Optional[Sequence] = None) -> torch.Tensor:
    """decode_attention over a 4-bit cache; q [S][Hq][D] in the cache's activation dtype."""
    with _on(stream, q.device):
        return prepared_decode_attention_q4(q, cache, block_tables, context_lens, scale, out, out_dtype,
                                            workspace, num_ctas, lse_out, tables_ready, timing_events)(stream)


def block_copy_q4(pairs, cache: Q4Cache, stream=None) -> None:
    """Copy whole blocks src -> dst of a 4-bit cache; pairs is host data [n][2]."""
    p = torch.as_tensor(pairs, dtype=torch.int64).reshape(-1, 2).contiguous()
    assert p.device.type == "cpu", "block-copy pairs are host memory"
    with torch.cuda.device(_one_gpu("pkv_block_copy_q4", (cache,))):
        _check(_ops_lib().pkv_block_copy_q4(ctypes.byref(cache.desc), _ptr(p), p.shape[0],
                                            ctypes.byref(cache.pools), _stream(stream)))


# ---------------------------------------------------------------- block-sparse decode
class SparseSelect(ctypes.Structure):
    _fields_ = [("top_blocks", ctypes.c_int32), ("first_blocks", ctypes.c_int32),
                ("last_blocks", ctypes.c_int32)]


def _means_desc(k_pool, k_means) -> CacheDesc:
    desc = cache_desc(k_pool)
    _need(k_pool, "k_pool", k_pool.dtype)
    _need(k_means, "k_means", k_pool.dtype, (desc.num_blocks, desc.num_kv_heads, desc.head_dim))
    return desc


def prepared_block_means(slot_mapping, k_pool, k_means) -> PreparedCall:
    """block_means as a PreparedCall."""
    desc = _means_desc(k_pool, k_means)
    _need(slot_mapping, "slot_mapping", torch.int64)
    return PreparedCall("pkv_block_means", (
        ctypes.byref(desc), _ptr(slot_mapping), slot_mapping.numel(),
                                      _ptr(k_pool), _ptr(k_means)),
        keep=(slot_mapping, k_pool, k_means, desc),
        out=None)


def block_means(slot_mapping, k_pool, k_means, stream=None) -> None:
    """Mean keys, into k_means [NB][Hk][D], of the blocks that the tokens at slot_mapping [T]
    (int64) have filled (pkv_block_means); after the append of those tokens."""
    return prepared_block_means(slot_mapping, k_pool, k_means)(stream)


def _selection(q, desc, block_tables, context_lens, select, sel_tables, sel_lens):
    S, Hq, _ = q.shape
    W = select.top_blocks + select.first_blocks + select.last_blocks
    _need(q, "q", CODE_DTYPE[desc.dtype], (S, Hq, desc.head_dim))
    _need(block_tables, "block_tables", torch.int32, (S, block_tables.shape[-1]))
    _need(context_lens, "context_lens", torch.int32, (S,))
    i32 = dict(dtype=torch.int32, device=q.device)
    shape = (S, desc.num_kv_heads, max(0, W))
    sel_tables = torch.empty(shape, **i32) if sel_tables is None else sel_tables
    sel_lens = torch.empty(shape[:2], **i32) if sel_lens is None else sel_lens
    _need(sel_tables, "sel_tables", torch.int32, shape)
    _need(sel_lens, "sel_lens", torch.int32, shape[:2])
    return S, Hq, sel_tables, sel_lens


def prepared_select_blocks(q, k_pool, k_means, block_tables, context_lens, top_blocks: int,
                           first_blocks: int = 1, last_blocks: int = 1,
                           sel_tables: Optional[torch.Tensor] = None,
                           sel_lens: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None) -> PreparedCall:
    """select_blocks as a PreparedCall."""
    desc = _means_desc(k_pool, k_means)
    sel = SparseSelect(top_blocks, first_blocks, last_blocks)
    S, Hq, st, sl = _selection(q, desc, block_tables, context_lens, sel, sel_tables, sel_lens)
    M = block_tables.shape[1]
    if workspace is None:
        n = int(_ops_lib().pkv_select_workspace_bytes(ctypes.byref(desc), S, M))
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
    return PreparedCall("pkv_select_blocks", (
        ctypes.byref(desc), _ptr(q), S, Hq, _ptr(k_means), _ptr(block_tables), M, _ptr(context_lens),
        ctypes.byref(sel), _ptr(st), _ptr(sl), _ptr(workspace),
        workspace.numel() * workspace.element_size()),
        keep=(q, k_means, block_tables, context_lens, st, sl, workspace, desc, sel),
        out=(st, sl))


def select_blocks(q, k_pool, k_means, block_tables, context_lens, top_blocks: int, first_blocks: int = 1,
                  last_blocks: int = 1, sel_tables: Optional[torch.Tensor] = None,
                  sel_lens: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None):
    """(sel_tables [S][Hk][W], sel_lens [S][Hk]): the blocks each kv head of each sequence reads
    (pkv_select_blocks), as tables over the pool viewed as [NB * Hk][1][B][D]. k_pool gives the
    shape only."""
    with _on(stream, q.device):
        return prepared_select_blocks(q, k_pool, k_means, block_tables, context_lens, top_blocks,
                                      first_blocks, last_blocks, sel_tables, sel_lens, workspace)(stream)


def alloc_sparse_workspace(k_pool, num_seqs: int, num_q_heads: int, max_blocks_per_seq: int) -> torch.Tensor:
    """Zero-filled workspace of decode_attention_sparse."""
    desc = cache_desc(k_pool)
    n = int(_ops_lib().pkv_decode_sparse_workspace_bytes(ctypes.byref(desc), num_seqs, num_q_heads,
                                                         max_blocks_per_seq))
    if n == 0:
        raise PkvError(-1, lib().pkv_last_error_message().decode())
    return torch.zeros(n, dtype=torch.uint8, device=k_pool.device)


def prepared_decode_attention_sparse(q, k_pool, v_pool, k_means, block_tables, context_lens,
                                     scale: float, top_blocks: int, first_blocks: int = 1,
                                     last_blocks: int = 1, out: Optional[torch.Tensor] = None,
                                     out_dtype: Optional[torch.dtype] = None,
                                     sel_tables: Optional[torch.Tensor] = None,
                                     sel_lens: Optional[torch.Tensor] = None,
                                     workspace: Optional[torch.Tensor] = None) -> PreparedCall:
    """decode_attention_sparse as a PreparedCall."""
    _pools(k_pool, v_pool)
    desc = _means_desc(k_pool, k_means)
    sel = SparseSelect(top_blocks, first_blocks, last_blocks)
    S, Hq, st, sl = _selection(q, desc, block_tables, context_lens, sel, sel_tables, sel_lens)
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    _need(out, "out", out.dtype, q.shape)
    if workspace is None:
        workspace = alloc_sparse_workspace(k_pool, S, Hq, block_tables.shape[1])
    return PreparedCall("pkv_decode_attention_sparse", (
        ctypes.byref(desc), _ptr(q), S, Hq, _ptr(k_pool), _ptr(v_pool), _ptr(k_means), _ptr(block_tables),
        block_tables.shape[1], _ptr(context_lens), float(scale), ctypes.byref(sel), _ptr(st), _ptr(sl),
        _ptr(out), DTYPE_CODE[out.dtype], _ptr(workspace), workspace.numel() * workspace.element_size()),
        keep=(q, k_pool, v_pool, k_means, block_tables, context_lens, st, sl, out, workspace, desc, sel),
        out=out)


def decode_attention_sparse(q, k_pool, v_pool, k_means, block_tables, context_lens, scale: float,
                            top_blocks: int, first_blocks: int = 1, last_blocks: int = 1,
                            out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                            sel_tables: Optional[torch.Tensor] = None,
                            sel_lens: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode attention over the blocks that the block means select for each (sequence, kv head):
    the top_blocks best, the first_blocks first and the last_blocks last (pkv_sparse.h)."""
    with _on(stream, q.device):
        return prepared_decode_attention_sparse(q, k_pool, v_pool, k_means, block_tables, context_lens,
                                                scale, top_blocks, first_blocks, last_blocks, out,
                                                out_dtype, sel_tables, sel_lens, workspace)(stream)
