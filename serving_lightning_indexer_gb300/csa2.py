"""Thin Python binding of the CSA2 C ABI (``include/csa2.h``).

Argument marshalling only: every step runs in the CUDA kernels of
``libcsa2.so``.  Tensors are torch CUDA tensors (their device pointers are
passed); there is no CPU fallback -- a missing library or a CPU tensor raises.
Workspace is allocated by torch on first use and cached per device.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import torch

from . import _build

_P = C.c_void_p
_I32 = C.c_int32
_I64 = C.c_int64


class Csa2Error(RuntimeError):
    def __init__(self, code: int, where: str, detail: str):
        super().__init__(f"{where}: status {code} ({detail})")
        self.code = code


# ---------------------------------------------------------------- C structs
class Rows(C.Structure):
    _fields_ = [("T", _I32), ("B", _I32), ("row_seq", _P), ("row_pos", _P), ("n_visible", _P), ("ratio_m", _I32)]


class IndexScoreArgs(C.Structure):
    _fields_ = [("q_fp8", _P), ("q_scale", _P), ("w", _P), ("index_k", _P), ("index_k_pages", _I64),
                ("page_table", _P), ("pt_stride", _I32), ("rows", Rows), ("scores", _P), ("ld_scores", _I64),
                ("block_max", _P), ("ld_block_max", _I64), ("hist", _P), ("index_k_format", _I32)]


class TopkArgs(C.Structure):
    _fields_ = [("scores", _P), ("ld_scores", _I64), ("block_max", _P), ("ld_block_max", _I64),
                ("page_table", _P), ("pt_stride", _I32), ("rows", Rows), ("k", _I32), ("topk_pos", _P),
                ("topk_slot", _P), ("ld_topk", _I64), ("pool_blocks", _P), ("pool_n", _I32), ("hist", _P),
                ("order", _I32)]


class ReindexArgs(C.Structure):
    _fields_ = [("q_fp8", _P), ("q_scale", _P), ("w", _P), ("index_k", _P), ("index_k_pages", _I64),
                ("page_table", _P), ("pt_stride", _I32), ("rows", Rows), ("pool_blocks", _P), ("pool_n", _I32),
                ("k", _I32), ("topk_pos", _P), ("topk_slot", _P), ("ld_topk", _I64), ("pool_scores", _P),
                ("index_k_format", _I32), ("order", _I32)]


class SparseAttnArgs(C.Structure):
    _fields_ = [("q", _P), ("main_kv", _P), ("main_kv_slots", _I64), ("topk_slot", _P), ("k", _I32),
                ("ld_topk", _I64), ("swa_kv", _P), ("swa_slots", _I64), ("swa_slot", _P), ("n_swa", _I32),
                ("ld_swa", _I64), ("sink", _P), ("softmax_scale", C.c_float), ("T", _I32), ("out_bf16", _I32),
                ("out", _P), ("lse", _P), ("kv_ready", _I32), ("q_pos", _P), ("out_inv_rope", _I32),
                ("rope_theta", C.c_float), ("swa_seg_start", _P)]


class CompressArgs(C.Structure):
    _fields_ = [("C", _P), ("Z", _P), ("n_tokens", _I64), ("ratio_m", _I32), ("gamma", _P), ("eps", C.c_float),
                ("apply_rope", _I32), ("rope_theta", C.c_float), ("first_entry", _I64), ("entry_pos", _P),
                ("main_kv", _P), ("main_kv_slots", _I64), ("page_table", _P), ("pt_len", _I64),
                ("entry_slot", _P), ("latent_out", _P), ("w_ik", _P), ("k_gamma", _P), ("index_k", _P),
                ("index_k_pages", _I64), ("index_k_format", _I32), ("index_latent_out", _P)]


class KvProjectArgs(C.Structure):
    _fields_ = [("hidden", _P), ("w", _P), ("T", _I32), ("hidden_dim", _I32), ("out", _P)]


class QuantFp8Args(C.Structure):
    _fields_ = [("x", _P), ("ld_x", _I64), ("T", _I32), ("K", _I32), ("block_rows", _I32), ("gamma", _P),
                ("eps", C.c_float), ("codes", _P), ("ld_codes", _I64), ("scale", _P), ("ld_scale", _I64)]


class Fp8LinearArgs(C.Structure):
    _fields_ = [("x", _P), ("ld_x", _I64), ("x_scale", _P), ("ld_x_scale", _I64), ("w", _P), ("ld_w", _I64),
                ("w_scale", _P), ("ld_w_scale", _I64), ("T", _I32), ("N", _I32), ("K", _I32), ("out_format", _I32),
                ("out", _P), ("ld_out", _I64), ("out_scale", _P), ("ld_out_scale", _I64), ("row_pos", _P),
                ("rope_head", _I32), ("rope_theta", C.c_float), ("w_ready", _I32)]


class BatchPlanArgs(C.Structure):
    _fields_ = [("B", _I32), ("ctx_len", _P), ("new_len", _P), ("ratio_m", _I32), ("page_table", _P),
                ("pt_stride", _I32), ("free_pages", _P), ("n_free", _I32), ("free_head", _P), ("free_head_out", _P),
                ("row_start", _P), ("n_visible", _P), ("entry_start", _P), ("max_rows", _I32), ("row_seq", _P),
                ("row_pos", _P), ("max_entries", _I32), ("entry_slot", _P), ("entry_pos", _P), ("entry_row", _P),
                ("swa_ring", _I32), ("ring_id", _P), ("swa_new", _P), ("swa_slot", _P), ("n_swa", _I32),
                ("ld_swa", _I64), ("pad", _I32)]


CALL_INDEX_SCORE, CALL_TOPK, CALL_REINDEX, CALL_SPARSE_ATTN = 1, 2, 3, 4
EXPORTED = ("csa2_status_string", "csa2_last_error_detail", "csa2_index_score", "csa2_topk_with_candidates",
            "csa2_reindex", "csa2_sparse_attn", "csa2_compress_m2", "csa2_workspace_size",
            "csa2_check_device_error", "csa2_version", "csa2_topk_with_candidates_noalloc",
            "csa2_debug_bounded_wait", "csa2_kv_project", "csa2_quant_fp8", "csa2_fp8_linear", "csa2_batch_plan")

_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False) -> C.CDLL:
    """Load libcsa2.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"libcsa2.so is not built ({path}); run __graft_entry__.build()")
        _build.build()
    lib = C.CDLL(path)
    lib.csa2_status_string.restype = C.c_char_p
    lib.csa2_status_string.argtypes = [C.c_int]
    lib.csa2_last_error_detail.restype = C.c_char_p
    lib.csa2_version.restype = C.c_char_p
    for name, st in (("csa2_index_score", IndexScoreArgs), ("csa2_topk_with_candidates", TopkArgs),
                     ("csa2_reindex", ReindexArgs), ("csa2_sparse_attn", SparseAttnArgs)):
        f = getattr(lib, name)
        f.restype = C.c_int
        f.argtypes = [C.POINTER(st), _P, C.c_size_t, _P]
    lib.csa2_topk_with_candidates_noalloc.restype = C.c_int
    lib.csa2_topk_with_candidates_noalloc.argtypes = [C.POINTER(TopkArgs), _P]
    lib.csa2_compress_m2.restype = C.c_int
    lib.csa2_compress_m2.argtypes = [C.POINTER(CompressArgs), _P]
    lib.csa2_workspace_size.restype = C.c_int
    lib.csa2_workspace_size.argtypes = [C.c_int, _P, C.POINTER(C.c_size_t)]
    lib.csa2_check_device_error.restype = C.c_int
    lib.csa2_check_device_error.argtypes = [_P]
    lib.csa2_kv_project.restype = C.c_int
    lib.csa2_kv_project.argtypes = [C.POINTER(KvProjectArgs), _P]
    for name in ("csa2_quant_fp8", "csa2_fp8_linear", "csa2_batch_plan"):
        f = getattr(lib, name)
        f.restype = C.c_int
        f.argtypes = [_P, _P]   # the packed struct or a pointer to one
    lib.csa2_debug_bounded_wait.restype = C.c_int
    lib.csa2_debug_bounded_wait.argtypes = [C.c_uint32, _P]
    _lib = lib
    return lib


def _check(rc: int, where: str):
    if rc != 0:
        lib = load()
        raise Csa2Error(rc, where, (lib.csa2_last_error_detail() or b"").decode())


# ---------------------------------------------------------------- helpers
def _ptr(t) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda:
        raise ValueError("CSA2 calls take CUDA tensors (no CPU path)")
    if not t.is_contiguous():
        raise ValueError("CSA2 calls take contiguous tensors")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_ws_cache: dict = {}


def workspace(nbytes: int, device, tag: str = "main") -> torch.Tensor | None:
    """A cached device buffer of at least nbytes (16-B aligned), or None."""
    if nbytes == 0:
        return None
    key = (str(device), tag)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


INDEX_FP8, INDEX_FP4 = 0, 1
INDEX_PAGE_BYTES = {8448: INDEX_FP8, 4352: INDEX_FP4}


def index_format(index_k) -> int:
    """Page format of an index-K cache [n_pages, page bytes]: FP8 (8448 B) or FP4 (4352 B)."""
    fmt = INDEX_PAGE_BYTES.get(int(index_k.shape[-1]))
    if fmt is None:
        raise ValueError(f"index-K pages of {index_k.shape[-1]} B: expected 8448 (FP8) or 4352 (FP4)")
    return fmt


def rows(T, B, row_seq=None, row_pos=None, n_visible=None, ratio_m=1) -> Rows:
    """Row description of a call.  The struct holds device pointers; it also
    keeps the tensors themselves, so that they stay allocated as long as the
    struct is in use."""
    r = Rows(T, B, _ptr(row_seq), _ptr(row_pos), _ptr(n_visible), ratio_m)
    r._tensors = (row_seq, row_pos, n_visible)
    return r


# ---------------------------------------------------------------- calls
def index_score(q_fp8, q_scale, w, index_k, page_table, r: Rows, scores, block_max=None, stream=None, hist=None):
    """Lightning-Indexer scores (csa2_index_score); `hist` ([2,T,2048] int32) optionally
    receives the key histograms that csa2_topk_with_candidates can reuse."""
    lib = load()
    a = IndexScoreArgs(_ptr(q_fp8), _ptr(q_scale), _ptr(w), _ptr(index_k), index_k.shape[0], _ptr(page_table),
                       page_table.shape[-1], r, _ptr(scores), scores.shape[-1], _ptr(block_max),
                       block_max.shape[-1] if block_max is not None else 0, _ptr(hist), index_format(index_k))
    _check(lib.csa2_index_score(C.byref(a), None, 0, _stream(stream)), "csa2_index_score")


def topk_with_candidates(scores, r: Rows, k, topk_pos, topk_slot=None, page_table=None, block_max=None,
                         pool_blocks=None, stream=None, ws=None, hist=None, order=0):
    """Top-k positions / slots and the optional candidate pool (csa2_topk_with_candidates)."""
    lib = load()
    a = TopkArgs(_ptr(scores), scores.shape[-1], _ptr(block_max), block_max.shape[-1] if block_max is not None else 0,
                 _ptr(page_table), page_table.shape[-1] if page_table is not None else 0, r, k, _ptr(topk_pos),
                 _ptr(topk_slot), topk_pos.shape[-1], _ptr(pool_blocks),
                 pool_blocks.shape[-1] if pool_blocks is not None else 0, _ptr(hist), order)
    need = C.c_size_t(0)
    _check(lib.csa2_workspace_size(CALL_TOPK, C.cast(C.byref(a), _P), C.byref(need)), "csa2_workspace_size")
    buf = ws if ws is not None else workspace(need.value, scores.device, "topk")
    _check(lib.csa2_topk_with_candidates(C.byref(a), _ptr(buf), buf.numel() if buf is not None else 0,
                                         _stream(stream)), "csa2_topk_with_candidates")


def topk_with_candidates_noalloc(scores, r: Rows, k, topk_pos, topk_slot=None, page_table=None, block_max=None,
                                 pool_blocks=None, stream=None, hist=None, order=0):
    """csa2_topk_with_candidates_noalloc: the same selection without a workspace; its
    scratch is a static device array inside the library (for callers that cannot
    allocate device memory)."""
    lib = load()
    a = TopkArgs(_ptr(scores), scores.shape[-1], _ptr(block_max), block_max.shape[-1] if block_max is not None else 0,
                 _ptr(page_table), page_table.shape[-1] if page_table is not None else 0, r, k, _ptr(topk_pos),
                 _ptr(topk_slot), topk_pos.shape[-1], _ptr(pool_blocks),
                 pool_blocks.shape[-1] if pool_blocks is not None else 0, _ptr(hist), order)
    _check(lib.csa2_topk_with_candidates_noalloc(C.byref(a), _stream(stream)), "csa2_topk_with_candidates_noalloc")


def reindex(q_fp8, q_scale, w, index_k, page_table, r: Rows, pool_blocks, k, topk_pos, topk_slot=None,
            pool_scores=None, stream=None, ws=None, order=0):
    """Pool-only rescoring and top-k of a Reindex layer (csa2_reindex)."""
    lib = load()
    a = ReindexArgs(_ptr(q_fp8), _ptr(q_scale), _ptr(w), _ptr(index_k), index_k.shape[0], _ptr(page_table),
                    page_table.shape[-1], r, _ptr(pool_blocks), pool_blocks.shape[-1], k, _ptr(topk_pos),
                    _ptr(topk_slot), topk_pos.shape[-1], _ptr(pool_scores), index_format(index_k), order)
    need = C.c_size_t(0)
    _check(lib.csa2_workspace_size(CALL_REINDEX, C.cast(C.byref(a), _P), C.byref(need)), "csa2_workspace_size")
    buf = ws if ws is not None else workspace(need.value, q_fp8.device, "reindex")
    _check(lib.csa2_reindex(C.byref(a), _ptr(buf), buf.numel() if buf is not None else 0, _stream(stream)),
           "csa2_reindex")


def sparse_attn(q, main_kv, topk_slot, swa_kv, swa_slot, sink, out, lse=None, softmax_scale=0.0, k=None,
                n_swa=None, stream=None, ws=None, kv_ready=False, q_pos=None, out_inv_rope=False, rope_theta=0.0,
                swa_seg_start=None):
    """MQA sparse attention with SWA keys and sink (csa2_sparse_attn); with q_pos
    ([T] int32) optionally the output's inverse RoPE and the SWA bounded-replay
    mask (swa_seg_start, [T] int32)."""
    lib = load()
    T = q.shape[0]
    kk = topk_slot.shape[-1] if (k is None and topk_slot is not None) else (k or 0)
    ns = swa_slot.shape[-1] if (n_swa is None and swa_slot is not None) else (n_swa or 0)
    a = SparseAttnArgs(_ptr(q), _ptr(main_kv), main_kv.shape[0] if main_kv is not None else 0, _ptr(topk_slot), kk,
                       topk_slot.shape[-1] if topk_slot is not None else 0, _ptr(swa_kv),
                       swa_kv.shape[0] if swa_kv is not None else 0, _ptr(swa_slot), ns,
                       swa_slot.shape[-1] if swa_slot is not None else 0, _ptr(sink), float(softmax_scale), T,
                       1 if out.dtype == torch.bfloat16 else 0, _ptr(out), _ptr(lse), 1 if kv_ready else 0,
                       _ptr(q_pos), 1 if out_inv_rope else 0, float(rope_theta), _ptr(swa_seg_start))
    need = C.c_size_t(0)
    _check(lib.csa2_workspace_size(CALL_SPARSE_ATTN, C.cast(C.byref(a), _P), C.byref(need)), "csa2_workspace_size")
    buf = ws if ws is not None else workspace(need.value, q.device, "attn")
    _check(lib.csa2_sparse_attn(C.byref(a), _ptr(buf), buf.numel() if buf is not None else 0, _stream(stream)),
           "csa2_sparse_attn")


def compress_m2(Cm, Z, ratio_m, gamma, main_kv, page_table=None, entry_slot=None, eps=1e-6, rope_theta=10000.0,
                apply_rope=True, first_entry=0, entry_pos=None, latent_out=None, stream=None,
                w_ik=None, k_gamma=None, index_k=None, index_latent_out=None):
    """Main-KV entry build: m=2 softmax pooling (or m=1), RMSNorm, RoPE, FP4 (csa2_compress_m2);
    with w_ik ([512,128] bf16), k_gamma and index_k also the entries' index keys."""
    lib = load()
    a = CompressArgs(_ptr(Cm), _ptr(Z), Cm.shape[0], ratio_m, _ptr(gamma), eps, 1 if apply_rope else 0, rope_theta,
                     first_entry, _ptr(entry_pos), _ptr(main_kv), main_kv.shape[0], _ptr(page_table),
                     page_table.numel() if page_table is not None else 0, _ptr(entry_slot), _ptr(latent_out),
                     _ptr(w_ik), _ptr(k_gamma), _ptr(index_k), index_k.shape[0] if index_k is not None else 0,
                     index_format(index_k) if index_k is not None else 0, _ptr(index_latent_out))
    _check(lib.csa2_compress_m2(C.byref(a), _stream(stream)), "csa2_compress_m2")


def kv_project(hidden, w, out, stream=None):
    """out [T,512] bf16 = hidden [T,H] bf16 @ w [H,512] bf16 (csa2_kv_project)."""
    lib = load()
    a = KvProjectArgs(_ptr(hidden), _ptr(w), hidden.shape[0], hidden.shape[1], _ptr(out))
    _check(lib.csa2_kv_project(C.byref(a), _stream(stream)), "csa2_kv_project")


_EMPTY = 16  # stands for a given tensor without elements (its data_ptr is 0); the length 0 goes along
_Tensor = torch.Tensor
_BF16, _F32, _U8, _INT32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def _packer(st):
    """Packs a struct's fields in order into bytes (a fifth of the time of filling the ctypes struct)."""
    code = {_P: "P", _I32: "i", _I64: "q", C.c_float: "f"}
    fmt = "@" + "".join(code[f[1]] for f in st._fields_)
    pad = C.sizeof(st) - struct.calcsize(fmt)
    return struct.Struct(fmt + "x" * pad).pack


_pack_quant, _pack_linear, _pack_plan = _packer(QuantFp8Args), _packer(Fp8LinearArgs), _packer(BatchPlanArgs)


def _device(t, name: str) -> int:
    """Device of a call's first tensor."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: CSA2 calls take CUDA tensors (no CPU path)")
    return dev


def _refuse(t, name: str, dtype, dev: int):
    """Says what is wrong with a tensor of another type or device than a call's."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() < 0:
        raise ValueError(f"{name}: CSA2 calls take CUDA tensors (no CPU path)")
    raise ValueError(f"{name}: on cuda:{t.get_device()}, the call's first tensor on cuda:{dev}")


# The checks below run on every call, before a launch of a few microseconds: each
# attribute of a tensor is asked for once.
def _mat(t, name: str, dtype, dev: int, shape):
    """(pointer, row stride) of a 2-D tensor of the given shape whose rows are contiguous
    (the rows may be apart)."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {list(shape)}, got {list(t.shape)}")
    m = shape[1]
    if t.is_contiguous():
        return t.data_ptr() or _EMPTY, m
    ld, step = t.stride()
    if (step != 1 and m > 1) or ld < m:
        raise ValueError(f"{name}: expected contiguous rows that do not overlap, got strides {t.stride()}")
    return t.data_ptr() or _EMPTY, ld


def _vec(t, name: str, dtype, dev: int, n: int) -> int:
    """Pointer of a contiguous 1-D tensor of n elements (0 for None)."""
    if t is None:
        return 0
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, name, dtype, dev)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: expected {n} contiguous elements, got {list(t.shape)}")
    return t.data_ptr() or _EMPTY


def _two_d(t, name: str):
    """Shape of a 2-D tensor."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name}: expected a torch tensor")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: expected a 2-D tensor, got {list(shape)}")
    return shape


def _issue(fn, packed: bytes, where: str, dev: int, stream):
    """Issues a call on its tensors' device: the device's current stream unless one is given."""
    if dev == torch._C._cuda_getDevice():
        rc = fn(packed, torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(dev):
            rc = fn(packed, _stream(stream))
    if rc != 0:
        _check(rc, where)


def quant_fp8(x, codes, scale, gamma=None, eps=1e-6, block_rows=1, stream=None):
    """e4m3 codes of x [T,K] bf16 with a fp32 scale per 128 columns of a row (block_rows=1;
    with gamma [K] of the row's RMSNorm) or per 128 x 128 tile (block_rows=128, weights):
    codes uint8 [T,K], scale [ceil(T/block_rows), ceil(K/128)] (csa2_quant_fp8)."""
    dev = _device(x, "x")
    T, K = shape = _two_d(x, "x")
    px, ldx = _mat(x, "x", _BF16, dev, shape)
    pc, ldc = _mat(codes, "codes", _U8, dev, shape)
    ps, lds = _mat(scale, "scale", _F32, dev, (T if block_rows == 1 else (T + 127) // 128, (K + 127) // 128))
    _issue(load().csa2_quant_fp8, _pack_quant(px, ldx, T, K, block_rows, _vec(gamma, "gamma", _F32, dev, K), eps, pc, ldc,
                                              ps, lds), "csa2_quant_fp8", dev, stream)


OUT_F32, OUT_BF16, OUT_FP8 = 0, 1, 2
_OUT_FORMAT = {_F32: OUT_F32, _BF16: OUT_BF16, _U8: OUT_FP8}


def fp8_linear(x, x_scale, w, w_scale, out, out_scale=None, row_pos=None, rope_head=0, rope_theta=0.0, w_ready=False,
               stream=None):
    """out [T,N] = x [T,K] @ w [N,K]^T on e4m3 codes (uint8) with their scales: x_scale
    [T,ceil(K/128)], w_scale [ceil(N/128),ceil(K/128)].  out fp32, bf16, or uint8 codes with
    out_scale [T,N/128]; rope_head turns the last 64 columns of every head of that many
    columns by row_pos [T] (csa2_fp8_linear)."""
    dev = _device(x, "x")
    T, K = x_shape = _two_d(x, "x")
    N, _ = w_shape = _two_d(w, "w")
    nb = (K + 127) // 128
    px, ldx = _mat(x, "x", _U8, dev, x_shape)
    pw, ldw = _mat(w, "w", _U8, dev, (N, K))
    pxs, ldxs = _mat(x_scale, "x_scale", _F32, dev, (T, nb))
    pws, ldws = _mat(w_scale, "w_scale", _F32, dev, ((N + 127) // 128, nb))
    kind = getattr(out, "dtype", None)
    fmt = _OUT_FORMAT.get(kind)
    if fmt is None:
        raise TypeError(f"out: expected float32, bfloat16 or uint8, got {kind}")
    po, ldo = _mat(out, "out", kind, dev, (T, N))
    pos, ldos = (0, 0) if out_scale is None else _mat(out_scale, "out_scale", _F32, dev, (T, N // 128))
    _issue(load().csa2_fp8_linear,
           _pack_linear(px, ldx, pxs, ldxs, pw, ldw, pws, ldws, T, N, K, fmt, po, ldo, pos, ldos,
                        _vec(row_pos, "row_pos", _INT32, dev, T), rope_head, rope_theta, 1 if w_ready else 0),
           "csa2_fp8_linear", dev, stream)


def batch_plan(ctx_len, new_len, ratio_m=1, page_table=None, free_pages=None, free_head=None, free_head_out=None,
               row_start=None, n_visible=None, entry_start=None, row_seq=None, row_pos=None, entry_slot=None,
               entry_pos=None, entry_row=None, swa_ring=0, ring_id=None, swa_new=None, swa_slot=None, pad=False,
               stream=None):
    """Rows, pages and slots of a step whose sequences hold ctx_len [B] tokens and get
    new_len [B] more (csa2_batch_plan).  Every output is optional, int32, and written in
    place; row arrays share one length (rows the step may have), entry arrays another;
    page_table [B, pages] is extended from free_pages when that is given."""
    dev = _device(ctx_len, "ctx_len")
    i32 = _INT32
    B = ctx_len.shape[0] if ctx_len.dim() == 1 else -1
    row_cap = entry_cap = 0   # the one length of the row arrays, and of the entry arrays
    for t in (row_seq, row_pos, swa_new, swa_slot):
        if t is not None:
            row_cap = len(t)
            break
    for t in (entry_slot, entry_pos, entry_row):
        if t is not None:
            entry_cap = len(t)
            break
    pt = pt_stride = ss = lds = n_swa = fp = n_free = 0
    if page_table is not None:
        pt_stride = _two_d(page_table, "page_table")[1]
        pt, ld = _mat(page_table, "page_table", i32, dev, (B, pt_stride))
        if ld != pt_stride:
            raise ValueError("page_table: expected a contiguous tensor")
    if swa_slot is not None:
        n_swa = _two_d(swa_slot, "swa_slot")[1]
        ss, lds = _mat(swa_slot, "swa_slot", i32, dev, (row_cap, n_swa))
    if free_pages is not None:
        n_free = len(free_pages)
        fp = _vec(free_pages, "free_pages", i32, dev, n_free)
    _issue(load().csa2_batch_plan, _pack_plan(
        B, _vec(ctx_len, "ctx_len", i32, dev, B), _vec(new_len, "new_len", i32, dev, B), ratio_m, pt, pt_stride, fp, n_free,
        _vec(free_head, "free_head", i32, dev, 1), _vec(free_head_out, "free_head_out", i32, dev, 1),
        _vec(row_start, "row_start", i32, dev, B + 1), _vec(n_visible, "n_visible", i32, dev, B),
        _vec(entry_start, "entry_start", i32, dev, B + 1),
        row_cap, _vec(row_seq, "row_seq", i32, dev, row_cap), _vec(row_pos, "row_pos", i32, dev, row_cap),
        entry_cap, _vec(entry_slot, "entry_slot", i32, dev, entry_cap), _vec(entry_pos, "entry_pos", i32, dev, entry_cap),
        _vec(entry_row, "entry_row", i32, dev, entry_cap),
        swa_ring, _vec(ring_id, "ring_id", i32, dev, B), _vec(swa_new, "swa_new", i32, dev, row_cap), ss, n_swa, lds,
        1 if pad else 0), "csa2_batch_plan", dev, stream)


def check_device_error(stream=None) -> int:
    """Synchronise the stream and return the device error status (0 = ok)."""
    lib = load()
    return lib.csa2_check_device_error(_stream(stream))


def version() -> str:
    return load().csa2_version().decode()
