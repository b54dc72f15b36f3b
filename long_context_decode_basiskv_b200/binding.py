"""ctypes binding of libbasiskv.so (include/basiskv.h).

Argument marshalling only: torch tensors are checked for device, dtype,
shape and contiguity and their device pointers are passed to the C ABI.
Every step of the decode path runs in the library's CUDA kernels; there is
no fallback.  ``lib()`` raises if the shared library is missing.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbasiskv.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE = 0, 1, 2, 3, 4
F32, BF16 = 0, 1
GROUP_SUM, GROUP_MAX = 1, 2
DEVERR_BLOCK_TABLE, DEVERR_SELECTION, DEVERR_SEQ_LEN, DEVERR_TIMEOUT, DEVERR_WORKSPACE = 1, 2, 4, 8, 16
DEVERR_PAGES = 32
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "llama3": 4}

# every function include/basiskv.h declares
SYMBOLS = [
    "basiskv_append", "basiskv_route", "basiskv_decode_attn", "basiskv_out_proj",
    "basiskv_fuse_out_factor", "basiskv_workspace_bytes", "basiskv_status_string",
    "basiskv_abi_version", "basiskv_decode_attn_noalloc", "basiskv_route_group", "basiskv_prefill",
    "basiskv_copy", "basiskv_append_route", "basiskv_assign_pages", "basiskv_release_pages",
    "basiskv_rope_init", "basiskv_rotary", "basiskv_dense_attn", "basiskv_dense_attn_workspace_bytes",
]


class CConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ["num_q_heads", "num_kv_heads", "head_dim", "rank_v", "rank_k", "page_size",
                 "hidden", "top_k", "dtype"]]


class CCache(ctypes.Structure):
    _fields_ = [("k_raw", ctypes.c_void_p), ("c_lat", ctypes.c_void_p), ("r_res", ctypes.c_void_p),
                ("summary", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("seq_len", ctypes.c_void_p), ("num_phys_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


class CFactors(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("P", ctypes.c_void_p), ("E", ctypes.c_void_p),
                ("Gt", ctypes.c_void_p)]


class CRopeParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ["layout", "rotary_dim", "scaling"]]
                + [(n, ctypes.c_double) for n in ["base", "factor", "original_len", "beta_fast", "beta_slow",
                                                  "low_freq_factor", "high_freq_factor"]])


class CRope(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("mscale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("inv_freq", ctypes.c_double * 64)]


class CAttnOptions(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("slopes", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p)]


_lib = None


def lib():
    """Load libbasiskv.so (once) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libbasiskv.so not built ({LIB_PATH}); run "
                           "`python -m long_context_decode_basiskv_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    pc, pk, pf = ctypes.POINTER(CConfig), ctypes.POINTER(CCache), ctypes.POINTER(CFactors)
    L.basiskv_append.argtypes = [pc, pk, pf, vp, vp, i32, i32, vp, vp]
    L.basiskv_prefill.argtypes = [pc, pk, pf, vp, vp, i32, i32, vp, vp]
    L.basiskv_route.argtypes = [pc, pk, vp, i32, vp, vp, vp, vp, sz, vp, vp]
    L.basiskv_route_group.argtypes = [pc, pk, vp, i32, i32, vp, vp, vp, vp, sz, vp, vp]
    L.basiskv_decode_attn.argtypes = [pc, pk, vp, i32, vp, vp, vp, vp, sz, vp, vp]
    L.basiskv_out_proj.argtypes = [pc, pf, vp, i32, vp, vp, sz, vp]
    L.basiskv_decode_attn_noalloc.argtypes = [pc, pk, vp, i32, vp, vp, vp, vp, vp]
    L.basiskv_fuse_out_factor.argtypes = [pc, vp, vp, vp, vp]
    L.basiskv_copy.argtypes = [vp, vp, sz, vp]
    L.basiskv_append_route.argtypes = [pc, pk, pf, vp, vp, vp, i32, i32, vp, vp, vp, sz, vp, vp]
    i64, pr, pa = ctypes.c_int64, ctypes.POINTER(CRope), ctypes.POINTER(CAttnOptions)
    L.basiskv_assign_pages.argtypes = [pc, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp]
    L.basiskv_release_pages.argtypes = [pc, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.basiskv_rope_init.argtypes = [pr, ctypes.POINTER(CRopeParams)]
    L.basiskv_rotary.argtypes = [pc, pr, vp, i64, vp, i64, vp, vp, vp, vp, i32, i32, vp]
    L.basiskv_dense_attn.argtypes = [pc, pk, vp, i32, i32, pa, vp, vp, vp, sz, vp, vp]
    L.basiskv_dense_attn_workspace_bytes.argtypes = [pc, i32, i32, i32]
    L.basiskv_dense_attn_workspace_bytes.restype = sz
    L.basiskv_workspace_bytes.argtypes = [pc, i32, i32]
    L.basiskv_workspace_bytes.restype = sz
    L.basiskv_status_string.argtypes = [i32]
    L.basiskv_status_string.restype = ctypes.c_char_p
    L.basiskv_abi_version.argtypes = []
    for name in ["basiskv_append", "basiskv_route", "basiskv_decode_attn", "basiskv_out_proj",
                 "basiskv_fuse_out_factor", "basiskv_abi_version", "basiskv_decode_attn_noalloc",
                 "basiskv_route_group", "basiskv_prefill", "basiskv_copy", "basiskv_append_route",
                 "basiskv_assign_pages", "basiskv_release_pages", "basiskv_rope_init", "basiskv_rotary",
                 "basiskv_dense_attn"]:
        getattr(L, name).restype = i32
    _lib = L
    return L


class BasisKVError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib().basiskv_status_string(status).decode()} (status {status})")


def _check(status: int, what: str):
    if status != OK:
        raise BasisKVError(status, what)


@dataclass(frozen=True)
class Config:
    num_q_heads: int
    num_kv_heads: int
    head_dim: int
    rank_v: int
    rank_k: int
    page_size: int
    hidden: int
    top_k: int
    dtype: torch.dtype

    @property
    def group(self) -> int:
        return self.num_q_heads // self.num_kv_heads

    def c(self) -> CConfig:
        """The C struct, a new one every time."""
        return CConfig(self.num_q_heads, self.num_kv_heads, self.head_dim, self.rank_v, self.rank_k,
                       self.page_size, self.hidden, self.top_k,
                       BF16 if self.dtype == torch.bfloat16 else F32)

    def _ref(self):
        """The C struct as the calls here pass it: made once, written to by none of them, not handed out."""
        made = self.__dict__.get("_c")
        if made is None:
            made = self.c()
            object.__setattr__(self, "_c", made)
        return ctypes.byref(made)


_I32 = 2 ** 31 - 1  # ctypes takes a larger number's low 32 bits; this one the library takes, or refuses


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype=None, shape=None):
    if (type(t) is torch.Tensor and t.is_cuda and (dtype is None or t.dtype is dtype)
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        return  # the common case, in one line: a decode step makes dozens of these checks
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _need_reachable(t: torch.Tensor, name: str, dtype=None, shape=None):
    """_need, but a page-locked CPU tensor is also accepted (the kernels reach it
    through the runtime's mapping of pinned host memory)."""
    if isinstance(t, torch.Tensor) and not t.is_cuda:
        if not t.is_pinned():
            raise ValueError(f"{name} must be a CUDA tensor or a pinned CPU tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        return
    _need(t, name, dtype, shape)


# the current stream's handle without a Stream object around it (3 us less per call), where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


class PagedCache:
    """Device tensors of the paged cache (allocated by torch, owned by this object)."""

    def __init__(self, cfg: Config, num_phys_pages: int, block_table: torch.Tensor,
                 seq_len: torch.Tensor, device="cuda"):
        self.cfg = cfg
        Hkv, P, d, r, s = cfg.num_kv_heads, cfg.page_size, cfg.head_dim, cfg.rank_v, cfg.rank_k
        self.k_raw = torch.empty((num_phys_pages, Hkv, P, d), dtype=cfg.dtype, device=device)
        self.c_lat = torch.empty((num_phys_pages, Hkv, P, r), dtype=cfg.dtype, device=device)
        self.r_res = torch.empty((num_phys_pages, Hkv, P, s), dtype=cfg.dtype, device=device)
        self.summary = torch.empty((num_phys_pages, Hkv, d), dtype=torch.float32, device=device)
        self.block_table = block_table.to(device=device, dtype=torch.int32).contiguous()
        self.seq_len = seq_len.to(device=device, dtype=torch.int32).contiguous()
        self.num_phys_pages = num_phys_pages

    @property
    def batch(self) -> int:
        return self.block_table.shape[0]

    @property
    def max_pages(self) -> int:
        return self.block_table.shape[1]

    def c(self) -> CCache:
        return CCache(self.k_raw.data_ptr(), self.c_lat.data_ptr(), self.r_res.data_ptr(),
                      self.summary.data_ptr(), self.block_table.data_ptr(), self.seq_len.data_ptr(),
                      self.num_phys_pages, self.max_pages)


@dataclass
class Factors:
    A: torch.Tensor    # [Hkv, d, r]
    P: torch.Tensor    # [Hkv, r, d]
    E: torch.Tensor    # [Hkv, d, s]
    Gt: torch.Tensor   # [hidden, Hq, r]

    def c(self) -> CFactors:
        return CFactors(self.A.data_ptr(), self.P.data_ptr(), self.E.data_ptr(), self.Gt.data_ptr())


def workspace_bytes(cfg: Config, batch: int, max_pages: int) -> int:
    return int(lib().basiskv_workspace_bytes(cfg._ref(), batch, max_pages))


def alloc_workspace(cfg: Config, batch: int, max_pages: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace (the library keeps its counters at zero between calls)."""
    return torch.zeros(max(workspace_bytes(cfg, batch, max_pages), 256), dtype=torch.uint8, device=device)


def fuse_out_factor(cfg: Config, Bf: torch.Tensor, W_O: torch.Tensor, Gt: torch.Tensor, stream=None):
    _need(Bf, "Bf", cfg.dtype, (cfg.num_kv_heads, cfg.rank_v, cfg.head_dim))
    _need(W_O, "W_O", cfg.dtype, (cfg.num_q_heads * cfg.head_dim, cfg.hidden))
    _need(Gt, "Gt", cfg.dtype, (cfg.hidden, cfg.num_q_heads, cfg.rank_v))
    _check(lib().basiskv_fuse_out_factor(cfg._ref(), _ptr(Bf), _ptr(W_O), _ptr(Gt),
                                         _stream(stream)), "basiskv_fuse_out_factor")


def append(cfg: Config, cache: PagedCache, f: Factors, k_new: torch.Tensor, v_new: torch.Tensor,
           err: torch.Tensor, stream=None):
    """k_new, v_new: [B, n_new, Hkv, d]; cache.seq_len must already count them."""
    B, n_new = k_new.shape[0], k_new.shape[1]
    shape = (B, n_new, cfg.num_kv_heads, cfg.head_dim)
    _need(k_new, "k_new", cfg.dtype, shape)
    _need(v_new, "v_new", cfg.dtype, shape)
    _need(err, "err", torch.int32)
    _check(lib().basiskv_append(cfg._ref(), ctypes.byref(cache.c()), ctypes.byref(f.c()),
                                _ptr(k_new), _ptr(v_new), B, n_new, _ptr(err), _stream(stream)),
           "basiskv_append")


def prefill(cfg: Config, cache: PagedCache, f: Factors, k_new: torch.Tensor, v_new: torch.Tensor,
            err: torch.Tensor, stream=None):
    """basiskv_append for long appends on the tensor cores (bf16): k_new, v_new [B, n_new, Hkv, d]."""
    B, n_new = k_new.shape[0], k_new.shape[1]
    shape = (B, n_new, cfg.num_kv_heads, cfg.head_dim)
    _need(k_new, "k_new", cfg.dtype, shape)
    _need(v_new, "v_new", cfg.dtype, shape)
    _need(err, "err", torch.int32)
    _check(lib().basiskv_prefill(cfg._ref(), ctypes.byref(cache.c()), ctypes.byref(f.c()),
                                 _ptr(k_new), _ptr(v_new), B, n_new, _ptr(err), _stream(stream)),
           "basiskv_prefill")


def route(cfg: Config, cache: PagedCache, q: torch.Tensor, sel: torch.Tensor, sel_cnt: torch.Tensor,
          ws: torch.Tensor, err: torch.Tensor, scores: Optional[torch.Tensor] = None, stream=None):
    B = q.shape[0]
    _need(q, "q", cfg.dtype, (B, cfg.num_q_heads, cfg.head_dim))
    _need(sel, "sel", torch.int32, (B, cfg.num_q_heads, cfg.top_k + 2))
    _need(sel_cnt, "sel_cnt", torch.int32, (B, cfg.num_q_heads))
    _need(ws, "workspace", torch.uint8)
    _need(err, "err", torch.int32)
    if scores is not None:
        _need(scores, "scores", torch.float32, (B, cfg.num_q_heads, cache.max_pages))
    _check(lib().basiskv_route(cfg._ref(), ctypes.byref(cache.c()), _ptr(q), B, _ptr(sel),
                               _ptr(sel_cnt), _ptr(scores), _ptr(ws), ws.numel(), _ptr(err),
                               _stream(stream)), "basiskv_route")


def append_route(cfg: Config, cache: PagedCache, f: Factors, k_new: torch.Tensor, v_new: torch.Tensor,
                 q: torch.Tensor, reduce: int, sel: torch.Tensor, sel_cnt: torch.Tensor, ws: torch.Tensor,
                 err: torch.Tensor, stream=None):
    """append (one token per sequence) then route (reduce = 0) or route_group in one call,
    the scoring running beside the append (basiskv_append_route)."""
    B = q.shape[0]
    _need(k_new, "k_new", cfg.dtype, (B, 1, cfg.num_kv_heads, cfg.head_dim))
    _need(v_new, "v_new", cfg.dtype, (B, 1, cfg.num_kv_heads, cfg.head_dim))
    _need(q, "q", cfg.dtype, (B, cfg.num_q_heads, cfg.head_dim))
    _need(sel, "sel", torch.int32, (B, cfg.num_q_heads, cfg.top_k + 2))
    _need(sel_cnt, "sel_cnt", torch.int32, (B, cfg.num_q_heads))
    _need(ws, "workspace", torch.uint8)
    _need(err, "err", torch.int32)
    _check(lib().basiskv_append_route(cfg._ref(), ctypes.byref(cache.c()), ctypes.byref(f.c()),
                                      _ptr(k_new), _ptr(v_new), _ptr(q), B, reduce, _ptr(sel), _ptr(sel_cnt),
                                      _ptr(ws), ws.numel(), _ptr(err), _stream(stream)), "basiskv_append_route")


def route_group(cfg: Config, cache: PagedCache, q: torch.Tensor, reduce: int, sel: torch.Tensor,
                sel_cnt: torch.Tensor, ws: torch.Tensor, err: torch.Tensor,
                scores: Optional[torch.Tensor] = None, stream=None):
    """One selection per KV group (reduce = GROUP_SUM or GROUP_MAX of its heads' scores),
    written to the sel rows of every head of the group; scores [B][Hkv][max_pages]."""
    B = q.shape[0]
    _need(q, "q", cfg.dtype, (B, cfg.num_q_heads, cfg.head_dim))
    _need(sel, "sel", torch.int32, (B, cfg.num_q_heads, cfg.top_k + 2))
    _need(sel_cnt, "sel_cnt", torch.int32, (B, cfg.num_q_heads))
    _need(ws, "workspace", torch.uint8)
    _need(err, "err", torch.int32)
    if scores is not None:
        _need(scores, "scores", torch.float32, (B, cfg.num_kv_heads, cache.max_pages))
    _check(lib().basiskv_route_group(cfg._ref(), ctypes.byref(cache.c()), _ptr(q), B, reduce,
                                     _ptr(sel), _ptr(sel_cnt), _ptr(scores), _ptr(ws), ws.numel(),
                                     _ptr(err), _stream(stream)), "basiskv_route_group")


def decode_attn(cfg: Config, cache: PagedCache, q: torch.Tensor, sel: Optional[torch.Tensor],
                sel_cnt: Optional[torch.Tensor], o_lat: torch.Tensor, ws: torch.Tensor, err: torch.Tensor,
                stream=None):
    """Attention over the pages in sel / sel_cnt, or (both None) over the selection the
    last route / route_group call left in the same workspace."""
    B = q.shape[0]
    _need(q, "q", cfg.dtype, (B, cfg.num_q_heads, cfg.head_dim))
    if (sel is None) != (sel_cnt is None):
        raise ValueError("sel and sel_cnt are given together or not at all")
    if sel is not None:
        _need(sel, "sel", torch.int32, (B, cfg.num_q_heads, cfg.top_k + 2))
        _need(sel_cnt, "sel_cnt", torch.int32, (B, cfg.num_q_heads))
    _need(o_lat, "o_lat", torch.float32, (B, cfg.num_q_heads, cfg.rank_v))
    _need(ws, "workspace", torch.uint8)
    _need(err, "err", torch.int32)
    _check(lib().basiskv_decode_attn(cfg._ref(), ctypes.byref(cache.c()), _ptr(q), B,
                                     _ptr(sel), _ptr(sel_cnt), _ptr(o_lat), _ptr(ws), ws.numel(),
                                     _ptr(err), _stream(stream)), "basiskv_decode_attn")


def out_proj(cfg: Config, f: Factors, o_lat: torch.Tensor, y: torch.Tensor, ws: torch.Tensor,
             stream=None):
    B = o_lat.shape[0]
    _need(o_lat, "o_lat", torch.float32, (B, cfg.num_q_heads, cfg.rank_v))
    _need_reachable(y, "y", torch.float32, (B, cfg.hidden))  # device, or pinned host: stored there directly
    _need(ws, "workspace", torch.uint8)
    _check(lib().basiskv_out_proj(cfg._ref(), ctypes.byref(f.c()), _ptr(o_lat), B, _ptr(y),
                                  _ptr(ws), ws.numel(), _stream(stream)), "basiskv_out_proj")


def copy(dst: torch.Tensor, src: torch.Tensor, stream=None):
    """dst <- src (same dtype and element count) by a kernel: either may be a CUDA tensor
    or a pinned CPU tensor (basiskv_copy)."""
    _need_reachable(dst, "dst")
    _need_reachable(src, "src", dst.dtype)
    if dst.numel() != src.numel():
        raise ValueError(f"copy: {src.numel()} elements into {dst.numel()}")
    _check(lib().basiskv_copy(_ptr(dst), _ptr(src), src.numel() * src.element_size(), _stream(stream)),
           "basiskv_copy")


def decode_attn_noalloc(cfg: Config, cache: PagedCache, q: torch.Tensor, sel: torch.Tensor,
                        sel_cnt: torch.Tensor, o_lat: torch.Tensor, err: torch.Tensor, stream=None):
    """decode_attn for callers that cannot allocate: the library's fixed 16 MiB scratch
    stands in for the workspace (see basiskv_decode_attn_noalloc in include/basiskv.h)."""
    B = q.shape[0]
    _need(q, "q", cfg.dtype, (B, cfg.num_q_heads, cfg.head_dim))
    _need(sel, "sel", torch.int32, (B, cfg.num_q_heads, cfg.top_k + 2))
    _need(sel_cnt, "sel_cnt", torch.int32, (B, cfg.num_q_heads))
    _need(o_lat, "o_lat", torch.float32, (B, cfg.num_q_heads, cfg.rank_v))
    _need(err, "err", torch.int32)
    _check(lib().basiskv_decode_attn_noalloc(cfg._ref(), ctypes.byref(cache.c()), _ptr(q), B,
                                             _ptr(sel), _ptr(sel_cnt), _ptr(o_lat), _ptr(err),
                                             _stream(stream)), "basiskv_decode_attn_noalloc")


def _same_device(first: torch.Tensor, *others: Optional[torch.Tensor]):
    """Every tensor on `first`'s device, which must be the current one (the kernels launch there)."""
    d = first.get_device()
    if d != torch.cuda.current_device():
        raise ValueError(f"tensors are on cuda:{d}, the current device is cuda:{torch.cuda.current_device()}")
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError(f"a tensor is on {t.device}, the others are on cuda:{d}")


def _same_count(free_count_out: torch.Tensor, free_count: torch.Tensor, stream):
    """What a page call leaves as the free list's count for an empty batch, for which the library writes nothing."""
    if free_count_out.data_ptr() != free_count.data_ptr():
        with torch.cuda.stream(stream):  # (None: the current one)
            free_count_out.copy_(free_count)


def assign_pages(cfg: Config, block_table: torch.Tensor, seq_len: torch.Tensor, add_len: torch.Tensor,
                 free_pages: torch.Tensor, free_count: torch.Tensor, seq_len_out: torch.Tensor,
                 free_count_out: torch.Tensor, slots: Optional[torch.Tensor], err: torch.Tensor, stream=None):
    """Pages for add_len[b] new tokens of every request b: entries of block_table [B, max_pages] taken
    from the free list (free_pages [num_phys], its first free_count[0] entries), seq_len_out = seq_len +
    add_len, free_count_out, and (slots [B, cols], or None) the slot page * P + position % P of each new
    token.  seq_len_out may be seq_len and free_count_out may be free_count (basiskv_assign_pages)."""
    i32, B, pages = torch.int32, seq_len.numel(), free_pages.numel()
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch, max_pages]")
    max_pages = block_table.shape[1]
    _need(seq_len, "seq_len", i32, (B,))
    _need(block_table, "block_table", i32, (B, max_pages))
    _need(add_len, "add_len", i32, (B,))
    _need(free_pages, "free_pages", i32, (pages,))
    _need(free_count, "free_count", i32, (1,))
    _need(seq_len_out, "seq_len_out", i32, (B,))
    _need(free_count_out, "free_count_out", i32, (1,))
    _need(err, "err", i32)
    cols = 0
    if slots is not None:
        cols = slots.shape[1] if slots.dim() == 2 else -1
        _need(slots, "slots", i32, (B, cols))
    _same_device(seq_len, block_table, add_len, free_pages, free_count, seq_len_out, free_count_out, slots, err)
    if B == 0:
        _same_count(free_count_out, free_count, stream)
    _check(lib().basiskv_assign_pages(cfg._ref(), B, max_pages, pages if pages <= _I32 else _I32, _ptr(seq_len),
                                      _ptr(add_len), _ptr(block_table), _ptr(free_pages), _ptr(free_count),
                                      _ptr(seq_len_out), _ptr(free_count_out), _ptr(slots),
                                      cols if cols <= _I32 else _I32, _ptr(err), _stream(stream)),
           "basiskv_assign_pages")


def release_pages(cfg: Config, block_table: torch.Tensor, seq_len: torch.Tensor, release: torch.Tensor,
                  free_pages: torch.Tensor, free_count: torch.Tensor, seq_len_out: torch.Tensor,
                  free_count_out: torch.Tensor, err: torch.Tensor, stream=None):
    """Back to the free list with the pages of every request whose release[b] is not zero;
    seq_len_out is 0 for them (basiskv_release_pages)."""
    i32, B, pages = torch.int32, seq_len.numel(), free_pages.numel()
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch, max_pages]")
    max_pages = block_table.shape[1]
    _need(seq_len, "seq_len", i32, (B,))
    _need(block_table, "block_table", i32, (B, max_pages))
    _need(release, "release", i32, (B,))
    _need(free_pages, "free_pages", i32, (pages,))
    _need(free_count, "free_count", i32, (1,))
    _need(seq_len_out, "seq_len_out", i32, (B,))
    _need(free_count_out, "free_count_out", i32, (1,))
    _need(err, "err", i32)
    _same_device(seq_len, block_table, release, free_pages, free_count, seq_len_out, free_count_out, err)
    if B == 0:
        _same_count(free_count_out, free_count, stream)
    _check(lib().basiskv_release_pages(cfg._ref(), B, max_pages, pages if pages <= _I32 else _I32, _ptr(seq_len),
                                       _ptr(release), _ptr(block_table), _ptr(free_pages), _ptr(free_count),
                                       _ptr(seq_len_out), _ptr(free_count_out), _ptr(err), _stream(stream)),
           "basiskv_release_pages")


class Rope:
    """Rotary frequencies of a model (basiskv_rope_init), made once and passed to every rotary call.

    layout: "half" (pair i is elements i and i + rotary_dim / 2) or "interleaved" (2i, 2i + 1);
    rotary_dim: how much of each head is rotated (default: all of it);
    scaling: "none", "linear", "ntk", "yarn" or "llama3" with their parameters."""

    def __init__(self, cfg: Config, base: float = 10000.0, rotary_dim: Optional[int] = None, layout: str = "half",
                 scaling: str = "none", factor: float = 1.0, original_len: float = 0.0, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, low_freq_factor: float = 1.0, high_freq_factor: float = 4.0):
        if layout not in ROPE_LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}, not {layout!r}")
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, not {scaling!r}")
        self.rotary_dim = cfg.head_dim if rotary_dim is None else int(rotary_dim)
        if self.rotary_dim > cfg.head_dim:
            raise ValueError(f"rotary_dim {self.rotary_dim} > head_dim {cfg.head_dim}")
        self.c = CRope()
        par = CRopeParams(ROPE_LAYOUTS[layout], self.rotary_dim, ROPE_SCALINGS[scaling], base, factor, original_len,
                          beta_fast, beta_slow, low_freq_factor, high_freq_factor)
        _check(lib().basiskv_rope_init(ctypes.byref(self.c), ctypes.byref(par)), "basiskv_rope_init")

    @property
    def inv_freq(self):
        """Radians per position of each pair (a list)."""
        return list(self.c.inv_freq)[:self.rotary_dim // 2]

    @property
    def mscale(self) -> float:
        return float(self.c.mscale)


def _token_stride(t: torch.Tensor, name: str, dtype, shape) -> int:
    """Elements from one token of t [B, n, heads, d] to the next: dense heads, tokens evenly spaced
    (a slice of a packed projection's heads is)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    B, n, h, d = shape
    st = t.stride()
    step = st[1] if n > 1 else st[0] if B > 1 else h * d
    if (st[3] != 1 or (h > 1 and st[2] != d) or (B > 1 and n > 1 and st[0] != n * st[1]) or step < h * d):
        raise ValueError(f"{name}: heads must be dense and tokens evenly spaced, strides are {st}")
    return step


def rotary(cfg: Config, rope: Rope, q: Optional[torch.Tensor], k: Optional[torch.Tensor],
           q_out: Optional[torch.Tensor], k_out: Optional[torch.Tensor], seq_len: Optional[torch.Tensor] = None,
           positions: Optional[torch.Tensor] = None, stream=None):
    """q [B, n, Hq, d] and k [B, n, Hkv, d] (either may be None, with its output) rotated by their
    tokens' positions into q_out and k_out, which may be q and k: positions [B, n], or seq_len [B], which
    counts the n new tokens already (token t is at seq_len - n + t).  q and k may be head slices of one
    packed projection [B, n, heads, d]; the outputs are dense (basiskv_rotary)."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("rotary: neither q nor k given")
    B, n = first.shape[0], first.shape[1]
    strides = [0, 0]
    for x, (t, out, heads, name) in enumerate(((q, q_out, cfg.num_q_heads, "q"), (k, k_out, cfg.num_kv_heads, "k"))):
        if (t is None) != (out is None):
            raise ValueError(f"{name} and {name}_out are given together or not at all")
        if t is not None:
            shape = (B, n, heads, cfg.head_dim)
            strides[x] = _token_stride(t, name, cfg.dtype, shape)
            _need(out, name + "_out", cfg.dtype, shape)
    if (positions is None) == (seq_len is None):
        raise ValueError("give either positions or seq_len")
    if positions is not None:
        _need(positions, "positions", torch.int32, (B, n))
    else:
        _need(seq_len, "seq_len", torch.int32, (B,))
    _same_device(first, q, k, q_out, k_out, positions, seq_len)
    _check(lib().basiskv_rotary(cfg._ref(), ctypes.byref(rope.c), _ptr(q), strides[0], _ptr(k), strides[1],
                                _ptr(q_out), _ptr(k_out), _ptr(positions), _ptr(seq_len), B, n, _stream(stream)),
           "basiskv_rotary")


@dataclass
class AttnOptions:
    """What a layer's scores are besides scaled dot products (basiskv_attn_options)."""
    scale: float = 0.0                          # 0: 1 / sqrt(head_dim)
    softcap: float = 0.0                        # c > 0: c tanh(s / c)
    window: int = 0                             # w > 0: the last w tokens, itself included (however large)
    slopes: Optional[torch.Tensor] = None       # [Hq] fp32: slope * distance is taken off
    prefix_len: Optional[torch.Tensor] = None   # [B] int32: tokens that every new token sees


def dense_workspace_bytes(cfg: Config, batch: int, n_new: int, max_pages: int) -> int:
    return int(lib().basiskv_dense_attn_workspace_bytes(cfg._ref(), batch, n_new, max_pages))


def alloc_dense_workspace(cfg: Config, batch: int, n_new: int, max_pages: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of dense_attn for this shape and any that needs no more bytes, in any order (its
    counters are left at zero between calls)."""
    return torch.zeros(max(dense_workspace_bytes(cfg, batch, n_new, max_pages), 256), dtype=torch.uint8, device=device)


def dense_attn(cfg: Config, cache: PagedCache, q: torch.Tensor, o_lat: torch.Tensor, ws: torch.Tensor,
               err: torch.Tensor, options: Optional[AttnOptions] = None, lse: Optional[torch.Tensor] = None,
               stream=None):
    """Attention of the last n tokens of every sequence over its whole cache: q [B, n, Hq, d] ->
    o_lat [B, n, Hq, r] and, where given, lse [B, n, Hq] (fp32).  Without the n axis (q [B, Hq, d]) one token
    each.  ws from alloc_dense_workspace (basiskv_dense_attn)."""
    if q.dim() not in (3, 4):
        raise ValueError("q must be [B, n, Hq, d] or [B, Hq, d]")
    lead = tuple(q.shape[:-2])
    B, n = lead[0], lead[1] if len(lead) == 2 else 1
    _need(q, "q", cfg.dtype, lead + (cfg.num_q_heads, cfg.head_dim))
    _need(o_lat, "o_lat", torch.float32, lead + (cfg.num_q_heads, cfg.rank_v))
    _need(ws, "workspace", torch.uint8)
    _need(err, "err", torch.int32)
    if B != cache.batch:
        raise ValueError(f"q has {B} sequences, the cache {cache.batch}")
    if lse is not None:
        _need(lse, "lse", torch.float32, lead + (cfg.num_q_heads,))
    opt, slopes, prefix = None, None, None
    if options is not None:
        slopes, prefix = options.slopes, options.prefix_len
        if slopes is not None:
            _need(slopes, "slopes", torch.float32, (cfg.num_q_heads,))
        if prefix is not None:
            _need(prefix, "prefix_len", torch.int32, (B,))
        opt = CAttnOptions(options.scale, options.softcap, max(-1, min(options.window, _I32)), 0, _ptr(slopes),
                           _ptr(prefix))
        if (opt.scale == 0 and options.scale != 0) or (opt.softcap == 0 and options.softcap != 0):
            raise ValueError(f"scale {options.scale} or softcap {options.softcap} is 0 in fp32, which stands for none")
        opt = ctypes.byref(opt)
    _same_device(q, cache.k_raw, cache.c_lat, cache.block_table, cache.seq_len, o_lat, ws, err, lse, slopes, prefix)
    _check(lib().basiskv_dense_attn(cfg._ref(), ctypes.byref(cache.c()), _ptr(q), B, n, opt, _ptr(o_lat),
                                    _ptr(lse), _ptr(ws), ws.numel(), _ptr(err), _stream(stream)), "basiskv_dense_attn")
