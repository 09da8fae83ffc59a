"""ctypes binding of libattn.so (include/attn.h).

Argument marshalling only: every step of the attention path runs in the
library's CUDA kernels.  PyTorch provides device memory and the current
stream.  If the library has not been built (or cannot be loaded) every call
raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libattn.so")

ATTN_STATUS_CAPACITY = 1
ATTN_STATUS_SEQLENS = 2
ATTN_STATUS_TIMEOUT = 4
ATTN_STATUS_BOUNDS = 8
ATTN_STATUS_POSITION = 16
ATTN_STATUS_PAGES = 32


class AttnConfig(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rms_eps", ctypes.c_float),
                ("rope_theta", ctypes.c_float)]


class AttnKV(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("num_slots", ctypes.c_int64), ("slot_base", ctypes.c_void_p),
                ("cache_lens", ctypes.c_void_p), ("slot_capacity", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("page_size", ctypes.c_int32),
                ("pages_per_req", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
                ("k_block_scale", ctypes.c_void_p), ("v_block_scale", ctypes.c_void_p)]


class AttnRopeAxes(ctypes.Structure):
    _fields_ = [("num_axes", ctypes.c_int32), ("section", ctypes.c_int32 * 4), ("interleaved", ctypes.c_int32),
                ("positions", ctypes.c_void_p), ("ld", ctypes.c_int64)]


class AttnPages(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("ref_count", ctypes.c_void_p), ("cache_lens", ctypes.c_void_p),
                ("num_rows", ctypes.c_int32)]


ATTN_KV_BF16 = 0
ATTN_KV_E4M3 = 1
ATTN_KV_E2M1 = 2


class AttnError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"attn error {code}: {msg}")
        self.code = code


_lib = None

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t
_CFG = ctypes.POINTER(AttnConfig)
_KV = ctypes.POINTER(AttnKV)
_ROPE = ctypes.POINTER(AttnRopeAxes)
_PAGES = ctypes.POINTER(AttnPages)

EXPORTS = {
    "attn_workspace_size": (_SZ, [_CFG, _I32, _I32, _I32]),
    "attn_workspace_init": (ctypes.c_int, [_P, _SZ, _P]),
    "attn_kv_append": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _I32, _I32, _KV, _P, _SZ, _P]),
    "attn_prefill": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _I32, _I32, _I32, _KV, _P, _P, _SZ, _P]),
    "attn_decode": (ctypes.c_int, [_CFG, _P, _P, _P, _I32, _I32, _KV, _P, _P, _SZ, _P]),
    "attn_prefill_prepare": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _I32, _I32, _KV, _P, _P, _SZ, _P]),
    "attn_prefill_attend": (ctypes.c_int, [_CFG, _P, _P, _I32, _I32, _I32, _KV, _P, _P, _SZ, _P]),
    "attn_decode_attend": (ctypes.c_int, [_CFG, _P, _P, _I32, _I32, _KV, _P, _P, _SZ, _P]),
    "attn_decode_static_scratch": (ctypes.c_int, [_CFG, _P, _P, _P, _I32, _I32, _KV, _P, _P, _P]),
    "attn_decode_splits": (_I32, [_CFG, _I32, _I32]),
    "attn_decode_splits_of": (_I32, [_CFG, _I32, _I32, _I32, _I32]),
    "attn_qkv_proj_prepare": (ctypes.c_int, [_CFG, _P, _I32, _P, _P, _P, _P, _I32, _I32, _KV, _P, _P, _SZ, _P]),
    "attn_o_proj": (ctypes.c_int, [_CFG, _P, _I32, _P, _I32, _P, _P, _SZ, _P]),
    "attn_kv_append_axes": (ctypes.c_int, [_CFG, _P, _P, _P, _I32, _I32, _KV, _ROPE, _P, _SZ, _P]),
    "attn_prefill_prepare_axes": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _I32, _I32, _KV, _ROPE, _P, _P, _SZ, _P]),
    "attn_prefill_axes": (ctypes.c_int, [_CFG, _P, _P, _P, _P, _I32, _I32, _I32, _KV, _ROPE, _P, _P, _SZ, _P]),
    "attn_decode_axes": (ctypes.c_int, [_CFG, _P, _P, _P, _I32, _I32, _KV, _ROPE, _P, _P, _SZ, _P]),
    "attn_decode_attend_axes": (ctypes.c_int, [_CFG, _P, _P, _I32, _I32, _KV, _ROPE, _P, _P, _SZ, _P]),
    "attn_qkv_proj_prepare_axes": (ctypes.c_int, [_CFG, _P, _I32, _P, _P, _P, _P, _I32, _I32, _KV, _ROPE, _P, _P,
                                                  _SZ, _P]),
    "attn_kv_gather": (ctypes.c_int, [_CFG, _KV, _P, _P, _I32, _I32, _P, _P, _P, _SZ, _P]),
    "attn_pages_workspace_size": (_SZ, [ctypes.c_int64, _I32]),
    "attn_pages_reserve": (ctypes.c_int, [_KV, _PAGES, _P, _P, _I32, _P, _SZ, _P]),
    "attn_pages_fork": (ctypes.c_int, [_CFG, _KV, _PAGES, _P, _P, _I32, _P, _SZ, _P]),
    "attn_pages_free": (ctypes.c_int, [_KV, _PAGES, _P, _I32, _P, _SZ, _P]),
    "attn_pages_copy": (ctypes.c_int, [_CFG, _KV, _P, _P, _I32, _P, _SZ, _P]),
    "attn_pages_compact": (ctypes.c_int, [_CFG, _KV, _PAGES, _P, _SZ, _P]),
    "attn_get_status": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_int32)]),
    "attn_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "attn_sample_tokens": (ctypes.c_int, [_P, _I32, _I32, ctypes.c_int64, _P, _P, _P, _P, _P, _P]),
}


def load(path: str = LIB_PATH):
    """Load libattn.so and declare its exports (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built: run causal_gqa_attention_qkv_gb300.build.build()")
        lib = ctypes.CDLL(path)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(rc: int) -> None:
    if rc != 0:
        raise AttnError(rc, load().attn_strerror(rc).decode())


# Addresses and streams go to ctypes as plain integers (the argument types say
# what they are): an object less per argument on calls that take microseconds.
def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without building a torch Stream object per call
# (a few microseconds on every launch); torch.cuda.current_stream() otherwise.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(_device())
    return torch.cuda.current_stream().cuda_stream


def config(num_q_heads: int, num_kv_heads: int, head_dim: int, rms_eps: float = 1e-6,
           rope_theta: float = 1e6) -> AttnConfig:
    return AttnConfig(num_q_heads, num_kv_heads, head_dim, rms_eps, rope_theta)


@dataclasses.dataclass
class KVCache:
    """Device tensors of one layer's KV cache (see attn_kv_t)."""

    k_cache: torch.Tensor       # bf16, or uint8 E4M3 codes, [num_slots, Hkv, D]; E2M1: uint8 [num_slots, Hkv, D/2]
    v_cache: torch.Tensor       # same type and shape as k_cache
    slot_base: torch.Tensor     # int64 [B] (contiguous layout)
    cache_lens: torch.Tensor    # int32 [B]
    slot_capacity: torch.Tensor  # int32 [B]
    page_table: torch.Tensor | None = None  # int32 [B, pages_per_req] (paged layout)
    page_size: int = 0
    k_scale: float = 1.0        # E4M3 caches: entry = code * scale
    v_scale: float = 1.0
    # E2M1 caches: uint8 [Hkv, num_slots, D/16] E4M3 scales of 16 entries each
    # (entry = code * block scale * scale); given, the cache is E2M1
    k_block_scale: torch.Tensor | None = None
    v_block_scale: torch.Tensor | None = None

    # The C struct is built (and the tensors checked) once and rebuilt when a
    # field is assigned; tensors changed in place (resize_, set_) are not seen.
    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_built":
            object.__setattr__(self, "_built", None)
            object.__setattr__(self, "_built_pages", None)
            object.__setattr__(self, "_fits", None)

    @property
    def kv_dtype(self) -> int:
        """Element type, ATTN_KV_*."""
        if self.k_block_scale is not None or self.v_block_scale is not None:
            return ATTN_KV_E2M1
        return ATTN_KV_E4M3 if self.k_cache.dtype == torch.uint8 else ATTN_KV_BF16

    def struct(self) -> AttnKV:
        built = self.__dict__.get("_built")
        if built is None:
            built = self._make_struct()
            object.__setattr__(self, "_built", built)
        return built

    def struct_for(self, cfg: AttnConfig, exact: bool = False) -> AttnKV:
        """struct() for a call with ``cfg``: refused where the caches hold fewer
        entries per slot than cfg's heads, where cfg is not that of an E2M1 cache, and
        with ``exact`` (calls that move or read whole slots) where they hold others."""
        d = self.__dict__
        if (cfg.num_kv_heads, cfg.head_dim, exact) != d["_fits"]:  # not as in the last call with this struct
            H, D, k = cfg.num_kv_heads, cfg.head_dim, self.k_cache
            n = k.shape[0] * H * D
            if self.k_block_scale is not None:
                fits = tuple(k.shape[1:]) == (H, D // 2)
            else:
                fits = (k.numel() == n if exact else k.numel() >= n) and self.v_cache.numel() >= n
            if not fits and load().attn_decode_splits(ctypes.byref(cfg), 1, 0) < 0:
                return self.struct()  # a cfg that the library refuses by itself, with its own code
            assert fits, "cfg is not the cache's"
            self.struct()
            d["_fits"] = (H, D, exact)
        return d["_built"]

    def _make_struct(self) -> AttnKV:
        fp8 = self.k_cache.dtype == torch.uint8
        kbs, vbs = self.k_block_scale, self.v_block_scale
        fp4 = self.kv_dtype == ATTN_KV_E2M1
        if fp4:
            S, H, half = self.k_cache.shape
            assert self.v_cache.shape == self.k_cache.shape, "v_cache"
            for name in ("k_block_scale", "v_block_scale"):
                t = getattr(self, name)
                assert t is not None and t.dtype == torch.uint8 and t.is_contiguous() and t.is_cuda, name
                assert fp8 and tuple(t.shape) == (H, S, half // 8), name
        for name in ("k_cache", "v_cache"):
            t = getattr(self, name)
            assert t.dtype == (torch.uint8 if fp8 else torch.bfloat16), name
            assert t.is_contiguous() and t.is_cuda, name
        assert self.slot_base.dtype == torch.int64 and self.slot_base.is_contiguous()
        assert self.cache_lens.dtype == torch.int32 and self.cache_lens.is_contiguous()
        assert self.slot_capacity.dtype == torch.int32 and self.slot_capacity.is_contiguous()
        pt, ps, ppr = None, 0, 0
        if self.page_table is not None:
            assert self.page_table.dtype == torch.int32 and self.page_table.is_contiguous()
            assert self.page_table.dim() == 2
            pt, ps, ppr = self.page_table.data_ptr(), int(self.page_size), int(self.page_table.shape[1])
        return AttnKV(self.k_cache.data_ptr(), self.v_cache.data_ptr(), self.k_cache.shape[0],
                      self.slot_base.data_ptr(), self.cache_lens.data_ptr(),
                      self.slot_capacity.data_ptr(), pt, ps, ppr,
                      self.kv_dtype, float(self.k_scale), float(self.v_scale),
                      kbs.data_ptr() if fp4 else None, vbs.data_ptr() if fp4 else None)

    def pages_struct(self, ref_count: torch.Tensor) -> AttnPages:
        """The pool's bookkeeping for the page calls: this cache's page table and
        cached lengths (which they write; checked once, like struct()) and the
        pages' reference counts."""
        built = self.__dict__.get("_built_pages")
        if built is None:
            assert self.page_table is not None and self.page_size > 0, "the cache is not paged"
            n = int(self.page_table.shape[0])
            assert self.cache_lens.numel() >= n, "cache_lens"
            built = (_i32(self.page_table, "page_table"), _i32(self.cache_lens, "cache_lens"), n,
                     self.k_cache.shape[0] // self.page_size)
            object.__setattr__(self, "_built_pages", built)
        assert ref_count.numel() >= built[3], "ref_count"
        return AttnPages(built[0], _i32(ref_count, "ref_count"), built[1], built[2])

    def rows(self, lo: int, hi: int, cache_lens: torch.Tensor | None = None) -> "KVCache":
        """The same cache seen by the requests [lo, hi) (with other cached
        lengths for them, if given)."""
        pt = self.page_table
        return dataclasses.replace(self, slot_base=self.slot_base[lo:hi],
                                   cache_lens=self.cache_lens[lo:hi] if cache_lens is None else cache_lens,
                                   slot_capacity=self.slot_capacity[lo:hi],
                                   page_table=None if pt is None else pt[lo:hi].contiguous())


@dataclasses.dataclass
class RopeAxes:
    """Rotary positions with several axes (see attn_rope_axes_t): positions
    int32 [A, N] on the device (rows may be strided), sections the rotation
    pairs of each axis (they sum to D/2), interleaved the order of the axes
    over the pairs."""

    positions: torch.Tensor
    sections: tuple
    interleaved: bool = False

    def struct(self, n: int) -> AttnRopeAxes:
        t, A = self.positions, len(self.sections)
        assert t.dtype == torch.int32 and t.is_cuda and t.dim() == 2 and A <= 4, "positions"
        assert t.shape[0] == A and t.shape[1] >= n and (t.shape[1] <= 1 or t.stride(1) == 1), "positions"
        ld = t.stride(0) if A > 1 else t.shape[1]
        assert ld >= n, "positions"
        return AttnRopeAxes(A, (ctypes.c_int32 * 4)(*[int(x) for x in self.sections]), int(bool(self.interleaved)),
                            t.data_ptr(), ld)


def _rope(rope, n):
    """The C struct of ``rope`` (None: no axes) for a call over n tokens."""
    return None if rope is None else ctypes.byref(rope.struct(n))


def decode_splits(cfg: AttnConfig, B: int, max_cache_len: int, kv_dtype: int = ATTN_KV_BF16, axes: bool = False) -> int:
    """Number of KV splits a decode call over a cache of type ``kv_dtype`` (with
    ``axes``: rotary axes) uses for its longest request (the library's own policy,
    attn_decode_splits_of)."""
    n = load().attn_decode_splits_of(ctypes.byref(cfg), int(B), int(max_cache_len), int(kv_dtype), int(axes))
    if n < 0:
        raise AttnError(int(n), load().attn_strerror(int(n)).decode())
    return int(n)


def workspace_size(cfg: AttnConfig, max_tokens: int, max_batch: int, max_kv_len: int) -> int:
    n = load().attn_workspace_size(ctypes.byref(cfg), max_tokens, max_batch, max_kv_len)
    if n == 0:
        raise AttnError(-1, "invalid workspace query")
    return int(n)


def new_workspace(cfg: AttnConfig, max_tokens: int, max_batch: int, max_kv_len: int,
                  device="cuda") -> torch.Tensor:
    """Allocate (with torch) and initialise a workspace."""
    n = workspace_size(cfg, max_tokens, max_batch, max_kv_len)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    _check(load().attn_workspace_init(_ptr(ws), n, _stream()))
    return ws


def _i32(t, name):
    assert t.dtype == torch.int32 and t.is_cuda and t.is_contiguous(), name
    return t.data_ptr()


def _bf16(t, name):
    assert t.dtype == torch.bfloat16 and t.is_cuda and t.is_contiguous(), name
    return _ptr(t)


def kv_append(cfg: AttnConfig, qkv, k_norm_w, cu_seqlens, kv: KVCache, workspace, stream=None, rope=None):
    """K and V of the new tokens into the cache.  ``rope`` (here and below): a
    RopeAxes with the tokens' positions on several axes."""
    B = cu_seqlens.numel() - 1
    s = kv.struct_for(cfg)
    _check(load().attn_kv_append_axes(ctypes.byref(cfg), _bf16(qkv, "qkv"), _bf16(k_norm_w, "k_norm_w"),
                                      _ptr(cu_seqlens), B, qkv.shape[0], ctypes.byref(s), _rope(rope, qkv.shape[0]),
                                      _ptr(workspace), workspace.numel(), _stream(stream)))


def prefill(cfg: AttnConfig, qkv, q_norm_w, k_norm_w, cu_seqlens, max_seqlen: int, kv: KVCache,
            out, workspace, stream=None, rope=None):
    assert cu_seqlens.dtype == torch.int32 and cu_seqlens.is_cuda
    B = cu_seqlens.numel() - 1
    s = kv.struct_for(cfg)
    _check(load().attn_prefill_axes(ctypes.byref(cfg), _bf16(qkv, "qkv"), _bf16(q_norm_w, "q_norm_w"),
                                    _bf16(k_norm_w, "k_norm_w"), _ptr(cu_seqlens), B, qkv.shape[0],
                                    int(max_seqlen), ctypes.byref(s), _rope(rope, qkv.shape[0]), _bf16(out, "out"),
                                    _ptr(workspace), workspace.numel(), _stream(stream)))


def decode(cfg: AttnConfig, qkv, q_norm_w, k_norm_w, max_cache_len: int, kv: KVCache, out,
           workspace, stream=None, rope=None):
    B = qkv.shape[0]
    s = kv.struct_for(cfg)
    _check(load().attn_decode_axes(ctypes.byref(cfg), _bf16(qkv, "qkv"), _bf16(q_norm_w, "q_norm_w"),
                                   _bf16(k_norm_w, "k_norm_w"), B, int(max_cache_len), ctypes.byref(s),
                                   _rope(rope, B), _bf16(out, "out"), _ptr(workspace), workspace.numel(),
                                   _stream(stream)))


def prefill_prepare(cfg: AttnConfig, qkv, q_norm_w, k_norm_w, cu_seqlens, kv: KVCache, q_out,
                    workspace, stream=None, rope=None):
    """First half of ``prefill``: K/V appended to the cache, prepared Q
    (normed, rotated, bf16 [N, Hq, D]) written to ``q_out``."""
    B = cu_seqlens.numel() - 1
    s = kv.struct_for(cfg)
    _check(load().attn_prefill_prepare_axes(ctypes.byref(cfg), _bf16(qkv, "qkv"), _bf16(q_norm_w, "q_norm_w"),
                                            _bf16(k_norm_w, "k_norm_w"), _ptr(cu_seqlens), B, qkv.shape[0],
                                            ctypes.byref(s), _rope(rope, qkv.shape[0]), _bf16(q_out, "q_out"),
                                            _ptr(workspace), workspace.numel(), _stream(stream)))


def prefill_attend(cfg: AttnConfig, q, cu_seqlens, max_seqlen: int, kv: KVCache, out, workspace,
                   stream=None):
    """Second half of ``prefill``: attention over the prepared Q ``q``
    [N, Hq, D] (the cache already holds the new K/V)."""
    B = cu_seqlens.numel() - 1
    s = kv.struct_for(cfg)
    _check(load().attn_prefill_attend(ctypes.byref(cfg), _bf16(q, "q"), _ptr(cu_seqlens), B, q.shape[0],
                                      int(max_seqlen), ctypes.byref(s), _bf16(out, "out"), _ptr(workspace),
                                      workspace.numel(), _stream(stream)))


def decode_attend(cfg: AttnConfig, qkv, q_norm_w, max_cache_len: int, kv: KVCache, out, workspace,
                  stream=None, rope=None):
    """Attention half of ``decode`` (the cache already holds the new K/V)."""
    s = kv.struct_for(cfg)
    _check(load().attn_decode_attend_axes(ctypes.byref(cfg), _bf16(qkv, "qkv"), _bf16(q_norm_w, "q_norm_w"),
                                          qkv.shape[0], int(max_cache_len), ctypes.byref(s),
                                          _rope(rope, qkv.shape[0]), _bf16(out, "out"), _ptr(workspace),
                                          workspace.numel(), _stream(stream)))


def decode_static_scratch(cfg: AttnConfig, qkv, q_norm_w, k_norm_w, max_cache_len: int, kv: KVCache,
                          out, device_status=None, stream=None):
    """``decode`` with the split-KV scratch in the library's static device
    buffer (no workspace; for callers that cannot allocate)."""
    s = kv.struct_for(cfg)
    _check(load().attn_decode_static_scratch(
        ctypes.byref(cfg), _bf16(qkv, "qkv"), _bf16(q_norm_w, "q_norm_w"), _bf16(k_norm_w, "k_norm_w"),
        qkv.shape[0], int(max_cache_len), ctypes.byref(s), _bf16(out, "out"), _ptr(device_status),
        _stream(stream)))


def qkv_proj_prepare(cfg: AttnConfig, hidden, w_qkv, q_norm_w, k_norm_w, cu_seqlens, kv: KVCache, q_out,
                     workspace, stream=None, rope=None):
    """The merged Q/K/V projection fused with ``prefill_prepare``: qkv =
    hidden [N, C] . w_qkv^T in fp32, then Q/K norm + RoPE, K/V appended,
    prepared Q written to ``q_out`` [N, Hq, D]."""
    assert hidden.dim() == 2 and w_qkv.dim() == 2 and w_qkv.shape[1] == hidden.shape[1]
    B = cu_seqlens.numel() - 1
    s = kv.struct_for(cfg)
    _check(load().attn_qkv_proj_prepare_axes(ctypes.byref(cfg), _bf16(hidden, "hidden"), hidden.shape[1],
                                             _bf16(w_qkv, "w_qkv"), _bf16(q_norm_w, "q_norm_w"),
                                             _bf16(k_norm_w, "k_norm_w"), _ptr(cu_seqlens), B, hidden.shape[0],
                                             ctypes.byref(s), _rope(rope, hidden.shape[0]), _ptr(q_out),
                                             _ptr(workspace), workspace.numel(), _stream(stream)))


def o_proj(cfg: AttnConfig, attn_out, w_o, out, workspace, stream=None):
    """out [N, C] = attn_out [N, Hq*D] . w_o^T (w_o [C, Hq*D])."""
    assert w_o.dim() == 2 and out.shape == (attn_out.shape[0], w_o.shape[0])
    _check(load().attn_o_proj(ctypes.byref(cfg), _bf16(attn_out, "attn_out"), attn_out.shape[0],
                              _bf16(w_o, "w_o"), w_o.shape[0], _bf16(out, "out"), _ptr(workspace),
                              workspace.numel(), _stream(stream)))


def kv_gather(cfg: AttnConfig, kv: KVCache, cu_seqlens, start, k_out, v_out, workspace, stream=None):
    """Cached entries read back: the entries at positions start[b] + j of
    request b into rows cu_seqlens[b] + j of ``k_out`` and ``v_out`` (bf16
    [N, Hkv, D]; codes as the bf16 nearest to the value they stand for)."""
    assert cu_seqlens.dtype == torch.int32 and cu_seqlens.is_cuda and cu_seqlens.is_contiguous(), "cu_seqlens"
    B = cu_seqlens.numel() - 1
    assert start.dtype == torch.int32 and start.is_cuda and start.is_contiguous() and start.numel() >= B, "start"
    rows = kv.slot_base.numel() if kv.page_table is None else kv.page_table.shape[0]
    assert min(rows, kv.slot_capacity.numel()) >= B, "cu_seqlens"
    assert k_out.shape == v_out.shape and tuple(k_out.shape[1:]) == (cfg.num_kv_heads, cfg.head_dim), "k_out"
    s = kv.struct_for(cfg, exact=True)
    _check(load().attn_kv_gather(ctypes.byref(cfg), ctypes.byref(s), _ptr(cu_seqlens), _ptr(start), B,
                                 k_out.shape[0], _bf16(k_out, "k_out"), _bf16(v_out, "v_out"), _ptr(workspace),
                                 workspace.numel(), _stream(stream)))


# ---------------------------------------------------------------- pages (include/pages.h)
def new_pages_workspace(kv: KVCache, max_rows: int | None = None) -> torch.Tensor:
    """Allocate and initialise a workspace for the page calls on ``kv``'s pool
    (``max_rows``: most page-table rows, by default the table's)."""
    assert kv.page_table is not None and kv.page_size > 0, "the cache is not paged"
    rows = int(kv.page_table.shape[0]) if max_rows is None else int(max_rows)
    n = load().attn_pages_workspace_size(kv.k_cache.shape[0] // kv.page_size, rows)
    if n == 0:
        raise AttnError(-1, "invalid workspace query")
    ws = torch.empty(n, dtype=torch.uint8, device=kv.k_cache.device)
    _check(load().attn_workspace_init(_ptr(ws), n, _stream()))
    return ws


def pages_reserve(kv: KVCache, ref_count, rows, new_tokens, workspace, stream=None):
    """Room for new_tokens[i] more entries in request rows[i] (int32 device
    tensors): the lowest free pages into the open entries of kv.page_table."""
    assert rows.numel() == new_tokens.numel(), "new_tokens"
    s, p = kv.struct(), kv.pages_struct(ref_count)
    _check(load().attn_pages_reserve(ctypes.byref(s), ctypes.byref(p), _i32(rows, "rows"),
                                     _i32(new_tokens, "new_tokens"), rows.numel(), _ptr(workspace), workspace.numel(),
                                     _stream(stream)))


def pages_fork(cfg: AttnConfig, kv: KVCache, ref_count, src_rows, dst_rows, workspace, stream=None):
    """Row dst_rows[i] becomes a copy of the request in row src_rows[i]: full
    pages shared, the open one copied."""
    assert src_rows.numel() == dst_rows.numel(), "dst_rows"
    s, p = kv.struct_for(cfg, exact=True), kv.pages_struct(ref_count)
    _check(load().attn_pages_fork(ctypes.byref(cfg), ctypes.byref(s), ctypes.byref(p), _i32(src_rows, "src_rows"),
                                  _i32(dst_rows, "dst_rows"), src_rows.numel(), _ptr(workspace), workspace.numel(),
                                  _stream(stream)))


def pages_free(kv: KVCache, ref_count, rows, workspace, stream=None):
    """The requests in ``rows`` end: their pages lose a reference, the rows are
    emptied."""
    s, p = kv.struct(), kv.pages_struct(ref_count)
    _check(load().attn_pages_free(ctypes.byref(s), ctypes.byref(p), _i32(rows, "rows"), rows.numel(),
                                  _ptr(workspace), workspace.numel(), _stream(stream)))


def pages_copy(cfg: AttnConfig, kv: KVCache, src_pages, dst_pages, workspace, stream=None):
    """Page dst_pages[i] becomes a copy of page src_pages[i]."""
    assert src_pages.numel() == dst_pages.numel(), "dst_pages"
    s = kv.struct_for(cfg, exact=True)
    _check(load().attn_pages_copy(ctypes.byref(cfg), ctypes.byref(s), _i32(src_pages, "src_pages"),
                                  _i32(dst_pages, "dst_pages"), src_pages.numel(), _ptr(workspace), workspace.numel(),
                                  _stream(stream)))


def pages_compact(cfg: AttnConfig, kv: KVCache, ref_count, workspace, stream=None):
    """Moves the pages in use to the front of the pool; kv.page_table and
    ``ref_count`` follow."""
    s, p = kv.struct_for(cfg, exact=True), kv.pages_struct(ref_count)
    _check(load().attn_pages_compact(ctypes.byref(cfg), ctypes.byref(s), ctypes.byref(p), _ptr(workspace),
                                     workspace.numel(), _stream(stream)))


def get_status(workspace, stream=None) -> int:
    st = ctypes.c_int32(0)
    _check(load().attn_get_status(_ptr(workspace), _stream(stream), ctypes.byref(st)))
    return int(st.value)


def sample_tokens(logits, temperature, top_k, top_p, uniform, tokens=None, stream=None):
    """One token per row of fp32 logits [B, V] (include/sample.h): greedy where
    temperature <= 0, else temperature + top-k + top-p, sampled with the row's
    uniform number.  Returns the int32 [B] device tensor of tokens."""
    assert logits.dtype == torch.float32 and logits.is_cuda and logits.dim() == 2 and logits.stride(1) == 1
    B, V = logits.shape
    for t, dt in ((temperature, torch.float32), (top_k, torch.int32), (top_p, torch.float32),
                  (uniform, torch.float32)):
        assert t.dtype == dt and t.is_cuda and t.is_contiguous() and t.numel() == B
    if tokens is None:
        tokens = torch.empty(B, dtype=torch.int32, device=logits.device)
    _check(load().attn_sample_tokens(_ptr(logits), B, V, logits.stride(0), _ptr(temperature), _ptr(top_k),
                                     _ptr(top_p), _ptr(uniform), _ptr(tokens), _stream(stream)))
    return tokens
