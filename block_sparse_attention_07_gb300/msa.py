"""Thin ctypes binding over libmsa.so (include/msa.h).

Argument marshalling only: every step of the MSA decode path runs in the
library's CUDA kernels. Tensors are torch tensors (used for device memory and
streams); each call passes their data pointers and the current CUDA stream.
Importing this module loads the library and raises if it was not built: there
is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import dataclasses
import math
import os

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libmsa.so")

F32, BF16, FP8_E4M3, NVFP4 = 0, 1, 2, 3
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_NONE, ROPE_LINEAR, ROPE_BY_PARTS, ROPE_BY_TURNS = 0, 1, 2, 3

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE, ERR_DEVICE_FLAG = range(6)

FLAG_BAD_PAGE, FLAG_BAD_BLOCK, FLAG_BAD_SEQLEN, FLAG_BAD_SLOT, FLAG_TIMEOUT, FLAG_Q_RANGE, FLAG_NO_PAGES = (
    0x1, 0x2, 0x4, 0x8, 0x10, 0x20, 0x40)

# Every function include/msa.h declares.
EXPORTED = ("msa_abi_version", "msa_status_string", "msa_get_last_dispatch", "msa_kv_insert_quant",
            "msa_index_score", "msa_insert_index_score", "msa_select_blocks", "msa_sparse_gqa_workspace_size",
            "msa_sparse_gqa_decode", "msa_sparse_gqa_decode_noalloc", "msa_read_device_flags",
            "msa_qk_norm_rope_insert", "msa_select_sparse_gqa_decode", "msa_selftest_bounded_wait",
            "msa_build_step", "msa_qk_norm_mrope_insert", "msa_paged_gqa_workspace_size", "msa_paged_gqa_decode",
            "msa_add_norm_quant", "msa_fp8_linear", "msa_make_rope", "msa_qkv_rope_insert")


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("q_len", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("n_idx_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("topk", ctypes.c_int32), ("local_blocks", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float)]


class _KVCache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("k_global", ctypes.c_float),
                ("v_global", ctypes.c_float)]


class _IndexCache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("keys", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("block_scale", ctypes.c_void_p), ("global_scale", ctypes.c_float)]


class NormRope(ctypes.Structure):
    """msa_norm_rope_t: device fp32 [D] RMSNorm weights (pointers), eps, rotary base."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("idx_q_weight", ctypes.c_void_p),
                ("idx_k_weight", ctypes.c_void_p), ("eps", ctypes.c_float), ("rope_theta", ctypes.c_float)]


class RopeAxes(ctypes.Structure):
    """msa_rope_axes_t: the number of position axes and the axis of each of the 64 rotary pairs."""
    _fields_ = [("num_axes", ctypes.c_int32), ("axis", ctypes.c_uint8 * 64)]


class Rope(ctypes.Structure):
    """msa_rope_t: pair layout, rotated dims, factor on cosine and sine, angles per position."""
    _fields_ = [("layout", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("gain", ctypes.c_float),
                ("freq", ctypes.c_double * 64)]


class MSAError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)}")
        self.status = status


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"libmsa.so is not built ({_LIB_PATH}); run __graft_entry__.build()")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.msa_abi_version.restype = ctypes.c_int
    lib.msa_status_string.restype = ctypes.c_char_p
    lib.msa_status_string.argtypes = [ctypes.c_int]
    lib.msa_get_last_dispatch.argtypes = [ctypes.c_char_p, sz]
    lib.msa_kv_insert_quant.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, ctypes.c_int, vp, i32,
                                        ctypes.POINTER(_KVCache), ctypes.POINTER(_IndexCache), vp, vp]
    lib.msa_index_score.argtypes = [ctypes.POINTER(Dims), vp, ctypes.c_int, ctypes.POINTER(_IndexCache), vp, vp,
                                    vp, vp, vp]
    lib.msa_insert_index_score.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, vp, ctypes.POINTER(_KVCache), vp,
                                           ctypes.POINTER(_IndexCache), vp, vp, vp, vp, vp]
    lib.msa_select_blocks.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, vp, vp]
    lib.msa_sparse_gqa_workspace_size.restype = sz
    lib.msa_sparse_gqa_workspace_size.argtypes = [ctypes.POINTER(Dims), ctypes.c_int]
    lib.msa_sparse_gqa_decode.argtypes = [ctypes.POINTER(Dims), vp, ctypes.POINTER(_KVCache), vp, vp, vp, vp, vp,
                                          vp, sz, vp, vp]
    lib.msa_select_sparse_gqa_decode.argtypes = [ctypes.POINTER(Dims), vp, ctypes.POINTER(_KVCache), vp, vp, vp,
                                                 vp, vp, vp, vp, sz, vp, vp]
    lib.msa_sparse_gqa_decode_noalloc.argtypes = [ctypes.POINTER(Dims), vp, ctypes.POINTER(_KVCache), vp, vp, vp,
                                                  vp, vp, vp, vp]
    lib.msa_read_device_flags.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
    lib.msa_selftest_bounded_wait.argtypes = [vp, vp]
    lib.msa_qk_norm_rope_insert.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, vp, vp, vp, vp, i32,
                                            ctypes.POINTER(NormRope), vp, vp, ctypes.POINTER(_KVCache),
                                            ctypes.POINTER(_IndexCache), vp, vp]
    lib.msa_build_step.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, i32,
                                   ctypes.c_int64, i32, vp, vp, vp]
    lib.msa_qk_norm_mrope_insert.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, vp, vp, vp, ctypes.c_int64, vp, i32,
                                             ctypes.POINTER(NormRope), ctypes.POINTER(RopeAxes), vp, vp,
                                             ctypes.POINTER(_KVCache), ctypes.POINTER(_IndexCache), vp, vp]
    lib.msa_paged_gqa_workspace_size.restype = sz
    lib.msa_paged_gqa_workspace_size.argtypes = [ctypes.POINTER(Dims), ctypes.c_int]
    lib.msa_paged_gqa_decode.argtypes = [ctypes.POINTER(Dims), vp, ctypes.POINTER(_KVCache), vp, vp, vp, vp, vp, sz,
                                         vp, vp]
    f32, f64, i64 = ctypes.c_float, ctypes.c_double, ctypes.c_int64
    lib.msa_add_norm_quant.argtypes = [i32, i32, vp, i64, vp, vp, ctypes.c_int, vp, f32, vp, vp, vp, vp]
    lib.msa_fp8_linear.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, ctypes.c_int, i64, vp, vp]
    lib.msa_make_rope.argtypes = [ctypes.POINTER(Rope), i32, f64, ctypes.c_int, ctypes.c_int, f64, f64, f64, f64]
    lib.msa_qkv_rope_insert.argtypes = [ctypes.POINTER(Dims), vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, i32,
                                        ctypes.POINTER(NormRope), ctypes.POINTER(Rope), vp, vp,
                                        ctypes.POINTER(_KVCache), ctypes.POINTER(_IndexCache), vp, vp]
    for name in EXPORTED:       # every other entry point returns msa_status_t
        if name not in ("msa_abi_version", "msa_status_string", "msa_sparse_gqa_workspace_size",
                        "msa_paged_gqa_workspace_size"):
            getattr(lib, name).restype = ctypes.c_int
    return lib


lib = _load()
LIB_PATH = _LIB_PATH


def status_string(status: int) -> str:
    return lib.msa_status_string(status).decode()


def last_dispatch() -> str:
    buf = ctypes.create_string_buffer(512)
    lib.msa_get_last_dispatch(buf, 512)
    return buf.value.decode()


def _check(status: int, what: str):
    if status != OK:
        raise MSAError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(stream if isinstance(stream, int) else stream.cuda_stream)
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def make_dims(batch, q_len, n_heads=64, n_kv_heads=4, n_idx_heads=4, head_dim=128, block_size=128,
              max_blocks_per_seq=1, num_pages=1, topk=16, local_blocks=1, softmax_scale=None) -> Dims:
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(head_dim)
    return Dims(batch, q_len, n_heads, n_kv_heads, n_idx_heads, head_dim, block_size, max_blocks_per_seq,
                num_pages, topk, local_blocks, softmax_scale)


@dataclasses.dataclass
class KVCache:
    """bf16: k, v [P, G, BS, D]. FP8_E4M3: k, v uint8 E4M3 [P, G, BS, D], k_global / v_global the
    per-tensor scales. NVFP4: k, v uint8 [P, G, BS, D/2], k_scale, v_scale uint8 [P, G, BS, D/16]."""
    dtype: int
    k: object
    v: object
    k_scale: object = None
    v_scale: object = None
    k_global: float = 1.0
    v_global: float = 1.0

    def c(self):
        return _KVCache(self.dtype, _ptr(self.k), _ptr(self.v), _ptr(self.k_scale), _ptr(self.v_scale),
                        self.k_global, self.v_global)


@dataclasses.dataclass
class IndexCache:
    """F32: keys f32 [P, I, BS, D]. FP8_E4M3: keys uint8 [P, I, BS, D], scale f32 [P, I, BS].
    NVFP4: keys uint8 [P, I, BS, D/2], block_scale uint8 [P, I, BS, D/16], global_scale (host float)."""
    dtype: int
    keys: object
    scale: object = None
    block_scale: object = None
    global_scale: float = 1.0

    def c(self):
        return _IndexCache(self.dtype, _ptr(self.keys), _ptr(self.scale), _ptr(self.block_scale), self.global_scale)


@functools.cache
def _bare(name):
    """The entry point without declared argument types: it takes converted arguments as they are."""
    fn = lib[name]
    fn.restype = ctypes.c_int
    return fn


def _converted(kind, arg):
    """An argument converted to its declared type, as ctypes would for every call."""
    if isinstance(arg, ctypes.c_void_p):
        arg = arg.value
    return kind.from_param(arg)


class Prepared:
    """A library call whose arguments were marshalled once; calling it launches again.

    Holds the ctypes structures the arguments point to; the tensors are kept
    alive by the caller. Launches on the stream that was given, or current,
    when it was made. Used on launch-bound paths (the same call issued every
    decode step)."""
    __slots__ = ("fn", "args", "keep", "what", "_bare", "_raw")

    def __init__(self, fn, args, keep, what):
        self.fn, self.args, self.keep, self.what = fn, args, keep, what
        # The arguments as the call passes them, for a function object that converts none: 0.5 to 1 us less per call.
        self._bare, self._raw = _bare(fn.__name__), tuple(_converted(t, a) for t, a in zip(fn.argtypes, args, strict=True))

    def __call__(self):
        st = self._bare(*self._raw)
        if st != OK:
            raise MSAError(st, self.what)


def _call(fn, args, keep, what, prepare):
    if prepare:
        return Prepared(fn, args, keep, what)
    _check(fn(*args), what)
    return None


def kv_insert_quant(dims: Dims, k_new, v_new, idx_k_new, idx_new_dtype: int, slot_mapping, cache: KVCache,
                    idx_cache: IndexCache | None, flags, stream=None, prepare=False):
    kc = cache.c()
    ic = idx_cache.c() if idx_cache is not None else None
    args = (ctypes.byref(dims), _ptr(k_new), _ptr(v_new), _ptr(idx_k_new), idx_new_dtype, _ptr(slot_mapping),
            int(k_new.shape[0]), ctypes.byref(kc), ctypes.byref(ic) if ic is not None else None, _ptr(flags),
            _stream(stream))
    return _call(lib.msa_kv_insert_quant, args, (dims, kc, ic), "msa_kv_insert_quant", prepare)


def select_sparse_gqa_decode(dims: Dims, q, cache: KVCache, block_table, seq_lens, scores, selected, out, lse,
                             workspace, flags, stream=None, prepare=False):
    """Selection (written to ``selected``) and sparse GQA in one launch."""
    kc = cache.c()
    args = (ctypes.byref(dims), _ptr(q), ctypes.byref(kc), _ptr(block_table), _ptr(seq_lens), _ptr(scores),
            _ptr(selected), _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
            _ptr(flags), _stream(stream))
    return _call(lib.msa_select_sparse_gqa_decode, args, (dims, kc), "msa_select_sparse_gqa_decode", prepare)


def make_norm_rope(q_weight, k_weight, idx_q_weight=None, idx_k_weight=None, eps=1e-6, rope_theta=10000.0):
    """msa_norm_rope_t from device fp32 [D] weight tensors (kept alive by the caller)."""
    nr = NormRope(_ptr(q_weight), _ptr(k_weight), _ptr(idx_q_weight), _ptr(idx_k_weight), eps, rope_theta)
    # what the addresses came from, for qk_norm_mrope_insert's checks
    nr.tensors = dict(q_weight=q_weight, k_weight=k_weight, idx_q_weight=idx_q_weight, idx_k_weight=idx_k_weight)
    return nr


def qk_norm_rope_insert(dims: Dims, q, k, v, idx_q, idx_k, positions, slot_mapping, nr: NormRope, q_out,
                        idx_q_out, cache: KVCache, idx_cache: IndexCache | None, flags, stream=None, prepare=False):
    kc = cache.c()
    ic = idx_cache.c() if idx_cache is not None else None
    args = (ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(idx_q), _ptr(idx_k), _ptr(positions),
            _ptr(slot_mapping), int(q.shape[0]), ctypes.byref(nr), _ptr(q_out), _ptr(idx_q_out), ctypes.byref(kc),
            ctypes.byref(ic) if ic is not None else None, _ptr(flags), _stream(stream))
    return _call(lib.msa_qk_norm_rope_insert, args, (dims, nr, kc, ic), "msa_qk_norm_rope_insert", prepare)


def index_score(dims: Dims, idx_q, q_dtype: int, idx_cache: IndexCache, block_table, seq_lens, scores, flags,
                stream=None, prepare=False):
    ic = idx_cache.c()
    args = (ctypes.byref(dims), _ptr(idx_q), q_dtype, ctypes.byref(ic), _ptr(block_table), _ptr(seq_lens),
            _ptr(scores), _ptr(flags), _stream(stream))
    return _call(lib.msa_index_score, args, (dims, ic), "msa_index_score", prepare)


def insert_index_score(dims: Dims, k_new, v_new, idx_k_new, slot_mapping, cache: KVCache, idx_q,
                       idx_cache: IndexCache, block_table, seq_lens, scores, flags, stream=None, prepare=False):
    """msa_insert_index_score: the step's new tokens (one per request, at its last position)
    inserted and every block scored, in one launch; one query position only."""
    kc, ic = cache.c(), idx_cache.c()
    args = (ctypes.byref(dims), _ptr(k_new), _ptr(v_new), _ptr(idx_k_new), _ptr(slot_mapping), ctypes.byref(kc),
            _ptr(idx_q), ctypes.byref(ic), _ptr(block_table), _ptr(seq_lens), _ptr(scores), _ptr(flags),
            _stream(stream))
    return _call(lib.msa_insert_index_score, args, (dims, kc, ic), "msa_insert_index_score", prepare)


def select_blocks(dims: Dims, scores, seq_lens, selected, flags, stream=None, prepare=False):
    args = (ctypes.byref(dims), _ptr(scores), _ptr(seq_lens), _ptr(selected), _ptr(flags), _stream(stream))
    return _call(lib.msa_select_blocks, args, (dims,), "msa_select_blocks", prepare)


def sparse_gqa_workspace_size(dims: Dims, kv_dtype: int) -> int:
    return int(lib.msa_sparse_gqa_workspace_size(ctypes.byref(dims), kv_dtype))


def sparse_gqa_decode(dims: Dims, q, cache: KVCache, block_table, seq_lens, selected, out, lse, workspace, flags,
                      stream=None, prepare=False):
    kc = cache.c()
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (ctypes.byref(dims), _ptr(q), ctypes.byref(kc), _ptr(block_table), _ptr(seq_lens), _ptr(selected),
            _ptr(out), _ptr(lse), _ptr(workspace), nbytes, _ptr(flags), _stream(stream))
    return _call(lib.msa_sparse_gqa_decode, args, (dims, kc), "msa_sparse_gqa_decode", prepare)


def sparse_gqa_decode_noalloc(dims: Dims, q, cache: KVCache, block_table, seq_lens, selected, out, lse, flags,
                              stream=None):
    """msa_sparse_gqa_decode without a workspace argument, for callers that cannot allocate
    device memory; its scratch is a fixed 64 MiB array inside the library (see include/msa.h)."""
    kc = cache.c()
    st = lib.msa_sparse_gqa_decode_noalloc(ctypes.byref(dims), _ptr(q), ctypes.byref(kc), _ptr(block_table),
                                           _ptr(seq_lens), _ptr(selected), _ptr(out), _ptr(lse), _ptr(flags),
                                           _stream(stream))
    _check(st, "msa_sparse_gqa_decode_noalloc")


def _want(what: str, name: str, t, dtype: str, shape, strided_rows=False):
    """Refuses (ERR_INVALID_ARG) a tensor of another type, shape or layout than the call reads."""
    import torch
    if t is None:
        raise MSAError(ERR_INVALID_ARG, f"{what}: {name} is missing")
    ok = t.dtype == getattr(torch, dtype) and tuple(t.shape) == tuple(shape)
    ok = ok and (t.is_contiguous() or (strided_rows and t.stride(-1) == 1))
    if not ok:
        raise MSAError(ERR_INVALID_ARG, f"{what}: {name} has to be {dtype} {list(shape)}, contiguous "
                                        f"(got {t.dtype} {list(t.shape)} strides {t.stride()})")


def _want_flags(what: str, flags):
    """The device flags: 32 bits at least, in 32-bit words."""
    import torch
    if flags is None:
        raise MSAError(ERR_INVALID_ARG, f"{what}: flags is missing")
    if flags.dtype not in (torch.int32, torch.uint32) or flags.numel() < 1 or not flags.is_contiguous():
        raise MSAError(ERR_INVALID_ARG, f"{what}: flags has to be int32 or uint32, one element at least, contiguous "
                                        f"(got {flags.dtype} {list(flags.shape)} strides {flags.stride()})")


def _want_on_device(what: str, **tensors):
    """Refuses (ERR_INVALID_ARG) tensors (None aside) that do not lie on the current GPU: their addresses go to its
    kernels. After the other checks, which need no GPU."""
    import torch
    for name, t in tensors.items():
        if t is not None and (t.device.type != "cuda" or t.device.index != torch.cuda.current_device()):
            raise MSAError(ERR_INVALID_ARG, f"{what}: {name} has to be on the current CUDA device (got {t.device})")


def _want_cache(what: str, dims: Dims, cache: KVCache):
    P, G, BS, D = dims.num_pages, dims.n_kv_heads, dims.block_size, dims.head_dim
    kind, row = {BF16: ("bfloat16", D), FP8_E4M3: ("uint8", D), NVFP4: ("uint8", D // 2)}.get(cache.dtype, (None, 0))
    if kind is None:
        raise MSAError(ERR_UNSUPPORTED, f"{what}: no K/V cache of dtype {cache.dtype}")
    for name in ("k", "v"):
        _want(what, "cache." + name, getattr(cache, name), kind, (P, G, BS, row))
        if cache.dtype == NVFP4:
            if getattr(cache, name + "_scale") is None:
                raise MSAError(ERR_INVALID_ARG, f"{what}: an NVFP4 cache needs {name}_scale")
            _want(what, f"cache.{name}_scale", getattr(cache, name + "_scale"), "uint8", (P, G, BS, D // 16))


def _want_idx_cache(what: str, dims: Dims, ic: IndexCache):
    P, I, BS, D = dims.num_pages, dims.n_idx_heads, dims.block_size, dims.head_dim
    if ic.dtype == FP8_E4M3:
        wants = (("keys", "uint8", (P, I, BS, D)), ("scale", "float32", (P, I, BS)))
    elif ic.dtype == NVFP4:
        wants = (("keys", "uint8", (P, I, BS, D // 2)), ("block_scale", "uint8", (P, I, BS, D // 16)))
    else:
        raise MSAError(ERR_UNSUPPORTED, f"{what}: no index cache of dtype {ic.dtype}")
    for name, kind, shape in wants:
        if getattr(ic, name) is None:
            raise MSAError(ERR_INVALID_ARG, f"{what}: an index cache of this type needs {name}")
        _want(what, "idx_cache." + name, getattr(ic, name), kind, shape)
    return {"idx_" + name: getattr(ic, name) for name, _, _ in wants}


def build_step(dims: Dims, ctx_lens, new_lens, free_pages, free_head, block_table, seq_lens, token_starts,
               slot_mapping, positions, free_head_out, flags, pos_offset=None, stream=None, prepare=False):
    """msa_build_step: block tables, slot map and positions ([axes, tokens]) of a step from its
    requests' lengths. ``slot_mapping``'s length is the step's token capacity."""
    what, B = "msa_build_step", dims.batch
    T = int(slot_mapping.shape[0])
    for name, t, shape in (("ctx_lens", ctx_lens, (B,)), ("new_lens", new_lens, (B,)),
                           ("free_pages", free_pages, (free_pages.numel(),)), ("free_head", free_head, (1,)),
                           ("block_table", block_table, (B, dims.max_blocks_per_seq)), ("seq_lens", seq_lens, (B,)),
                           ("token_starts", token_starts, (B + 1,)), ("free_head_out", free_head_out, (1,))):
        _want(what, name, t, "int32", shape)
    _want(what, "slot_mapping", slot_mapping, "int64", (T,))
    _want(what, "positions", positions, "int32", (positions.shape[0], T), strided_rows=True)
    if pos_offset is not None:
        _want(what, "pos_offset", pos_offset, "int32", (B,))
    _want_flags(what, flags)
    _want_on_device(what, ctx_lens=ctx_lens, new_lens=new_lens, free_pages=free_pages, free_head=free_head,
                    block_table=block_table, seq_lens=seq_lens, token_starts=token_starts, slot_mapping=slot_mapping,
                    positions=positions, free_head_out=free_head_out, pos_offset=pos_offset,
                    flags=flags)
    axes = int(positions.shape[0])
    pos_stride = int(positions.stride(0)) if axes > 1 else T
    args = (ctypes.byref(dims), _ptr(ctx_lens), _ptr(new_lens), _ptr(free_pages), int(free_pages.numel()),
            _ptr(free_head), _ptr(pos_offset), _ptr(block_table), _ptr(seq_lens), _ptr(token_starts),
            _ptr(slot_mapping), _ptr(positions), axes, pos_stride, T, _ptr(free_head_out), _ptr(flags),
            _stream(stream))
    return _call(lib.msa_build_step, args, (dims,), what, prepare)


def make_rope_axes(sections, interleaved: bool = False) -> RopeAxes:
    """msa_rope_axes_t from the number of rotary pairs of each axis (sections sum to 64). Contiguous: the first
    sections[0] pairs turn with axis 0, the next with axis 1, and so on. Interleaved: pair i turns with axis
    i mod A while i // A < sections[i mod A], and with axis 0 otherwise, so axis 0 takes what the others leave."""
    A = len(sections)
    if not 1 <= A <= 4 or sum(sections) != 64 or min(sections) < 0:
        raise MSAError(ERR_INVALID_ARG, "make_rope_axes: 1 to 4 sections that sum to 64")
    if interleaved:
        axis = [i % A if i // A < sections[i % A] else 0 for i in range(64)]
        if any(axis.count(a) != n for a, n in enumerate(sections)):
            raise MSAError(ERR_INVALID_ARG, f"make_rope_axes: sections {tuple(sections)} do not interleave over 64 pairs")
    else:
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    return RopeAxes(A, (ctypes.c_uint8 * 64)(*axis))


def qk_norm_mrope_insert(dims: Dims, q, k, v, idx_q, idx_k, positions, slot_mapping, nr: NormRope, axes: RopeAxes,
                         q_out, idx_q_out, cache: KVCache, idx_cache: IndexCache | None, flags, stream=None,
                         prepare=False):
    """msa_qk_norm_mrope_insert: ``positions`` [axes.num_axes, T]; otherwise as qk_norm_rope_insert."""
    what, T, D = "msa_qk_norm_mrope_insert", int(q.shape[0]), dims.head_dim
    for name, t, h in (("q", q, dims.n_heads), ("k", k, dims.n_kv_heads), ("v", v, dims.n_kv_heads),
                       ("q_out", q_out, dims.n_heads), ("idx_q", idx_q, dims.n_idx_heads),
                       ("idx_k", idx_k, dims.n_idx_heads), ("idx_q_out", idx_q_out, dims.n_idx_heads)):
        if t is not None:
            _want(what, name, t, "bfloat16", (T, h, D))
    _want(what, "positions", positions, "int32", (axes.num_axes, T), strided_rows=True)
    _want(what, "slot_mapping", slot_mapping, "int64", (T,))
    _want_cache(what, dims, cache)
    _want_flags(what, flags)
    wts = {n: t for n, t in getattr(nr, "tensors", {}).items() if t is not None}     # (a hand-made struct has addresses only)
    for name, t in wts.items():
        _want(what, name, t, "float32", (D,))
    ics = {}
    if idx_q is not None and idx_cache is not None:
        ics = _want_idx_cache(what, dims, idx_cache)
    _want_on_device(what, q=q, k=k, v=v, idx_q=idx_q, idx_k=idx_k, positions=positions, slot_mapping=slot_mapping,
                    q_out=q_out, idx_q_out=idx_q_out, k_cache=cache.k, v_cache=cache.v, k_scale=cache.k_scale,
                    v_scale=cache.v_scale, flags=flags, **wts, **ics)
    kc = cache.c()
    ic = idx_cache.c() if idx_cache is not None else None
    pos_stride = int(positions.stride(0)) if axes.num_axes > 1 else T
    args = (ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(idx_q), _ptr(idx_k), _ptr(positions), pos_stride,
            _ptr(slot_mapping), T, ctypes.byref(nr), ctypes.byref(axes), _ptr(q_out), _ptr(idx_q_out),
            ctypes.byref(kc), ctypes.byref(ic) if ic is not None else None, _ptr(flags), _stream(stream))
    return _call(lib.msa_qk_norm_mrope_insert, args, (dims, nr, axes, kc, ic), what, prepare)


def paged_gqa_workspace_size(dims: Dims, kv_dtype: int) -> int:
    return int(lib.msa_paged_gqa_workspace_size(ctypes.byref(dims), kv_dtype))


def paged_gqa_decode(dims: Dims, q, cache: KVCache, block_table, seq_lens, out, lse, workspace, flags, stream=None,
                     prepare=False):
    """msa_paged_gqa_decode: attention of the step's tokens over every cached token."""
    what = "msa_paged_gqa_decode"
    shape = (dims.batch, dims.q_len, dims.n_heads, dims.head_dim)
    _want(what, "q", q, "bfloat16", shape)
    _want(what, "out", out, "bfloat16", shape)
    if lse is not None:
        _want(what, "lse", lse, "float32", shape[:3])
    _want(what, "block_table", block_table, "int32", (dims.batch, dims.max_blocks_per_seq))
    _want(what, "seq_lens", seq_lens, "int32", (dims.batch,))
    _want_cache(what, dims, cache)
    _want_flags(what, flags)
    if workspace is not None and not workspace.is_contiguous():
        raise MSAError(ERR_INVALID_ARG, f"{what}: workspace has to be contiguous (got strides {workspace.stride()})")
    _want_on_device(what, q=q, out=out, lse=lse, block_table=block_table, seq_lens=seq_lens, k_cache=cache.k,
                    v_cache=cache.v, k_scale=cache.k_scale, v_scale=cache.v_scale, workspace=workspace, flags=flags)
    kc = cache.c()
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (ctypes.byref(dims), _ptr(q), ctypes.byref(kc), _ptr(block_table), _ptr(seq_lens), _ptr(out), _ptr(lse),
            _ptr(workspace), nbytes, _ptr(flags), _stream(stream))
    return _call(lib.msa_paged_gqa_decode, args, (dims, kc), what, prepare)


def _want_rows(what: str, name: str, t, dtype: str, shape):
    """Refuses a tensor whose rows are not contiguous; the rows themselves may lie apart, but not on one another."""
    import torch
    if t is None:
        raise MSAError(ERR_INVALID_ARG, f"{what}: {name} is missing")
    ok = t.dtype == getattr(torch, dtype) and tuple(t.shape) == tuple(shape)
    if ok and t.numel() > 0:
        row = 1
        for n, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
            ok = ok and (n == 1 or stride == row)
            row *= n
        ok = ok and (t.shape[0] == 1 or t.stride(0) >= row)
    if not ok:
        raise MSAError(ERR_INVALID_ARG, f"{what}: {name} has to be {dtype} {list(shape)}, contiguous within a row "
                                        f"(got {t.dtype} {list(t.shape)} strides {t.stride()})")


def _row_stride(t):
    """Elements between rows; a single row's tensor may say anything."""
    return int(t.stride(0)) if t.shape[0] > 1 else math.prod(t.shape[1:])


def add_norm_quant(x, weight, residual=None, residual_out=None, out=None, codes=None, scales=None, eps=1e-6,
                   stream=None, prepare=False):
    """msa_add_norm_quant: ``x`` bf16 [T, width] (rows may lie apart), ``residual`` / ``residual_out`` bf16 or fp32,
    ``weight`` fp32 [width] or None (no norm); results in ``out`` (bf16) and / or ``codes`` with ``scales``."""
    what = "msa_add_norm_quant"
    if x is None or x.dim() != 2:
        raise MSAError(ERR_INVALID_ARG, f"{what}: x has to be bfloat16 [tokens, width]")
    T, W = (int(n) for n in x.shape)
    _want_rows(what, "x", x, "bfloat16", (T, W))
    kind = BF16
    if residual is not None:
        import torch
        kind = F32 if residual.dtype == torch.float32 else BF16
        _want(what, "residual", residual, "float32" if kind == F32 else "bfloat16", (T, W))
    if residual_out is not None:
        _want(what, "residual_out", residual_out, "float32" if kind == F32 else "bfloat16", (T, W))
    if weight is not None:
        _want(what, "weight", weight, "float32", (W,))
    if out is not None:
        _want(what, "out", out, "bfloat16", (T, W))
    if codes is not None:
        _want(what, "codes", codes, "uint8", (T, W))
    if scales is not None:
        _want(what, "scales", scales, "float32", (T, (W + 127) // 128))
    _want_on_device(what, x=x, residual=residual, residual_out=residual_out, weight=weight, out=out, codes=codes,
                    scales=scales)
    args = (T, W, _ptr(x), _row_stride(x), _ptr(residual), _ptr(residual_out), kind, _ptr(weight), eps, _ptr(out),
            _ptr(codes), _ptr(scales), _stream(stream))
    return _call(lib.msa_add_norm_quant, args, (), what, prepare)


def fp8_linear(a, a_scales, w, w_scales, out, flags, stream=None, prepare=False):
    """msa_fp8_linear: ``out`` [T, N] (bf16 or fp32, rows may lie apart) from codes ``a`` [T, K] and ``w`` [N, K] (uint8
    E4M3) with their scales per 128 values and per 128 x 128 block, whose products are fp32 values."""
    what = "msa_fp8_linear"
    for name, t in (("a", a), ("w", w), ("out", out)):
        if t is None or t.dim() != 2:
            raise MSAError(ERR_INVALID_ARG, f"{what}: {name} has to be a matrix")
    import torch
    T, N, K = int(a.shape[0]), int(w.shape[0]), int(a.shape[1])
    KB = (K + 127) // 128
    f32 = out.dtype == torch.float32
    for name, t, dtype, shape in (("a", a, "uint8", (T, K)), ("a_scales", a_scales, "float32", (T, KB)),
                                  ("w", w, "uint8", (N, K)), ("w_scales", w_scales, "float32", ((N + 127) // 128, KB))):
        _want(what, name, t, dtype, shape)
    _want_rows(what, "out", out, "float32" if f32 else "bfloat16", (T, N))
    _want_flags(what, flags)
    _want_on_device(what, a=a, a_scales=a_scales, w=w, w_scales=w_scales, out=out, flags=flags)
    args = (T, N, K, _ptr(a), _ptr(a_scales), _ptr(w), _ptr(w_scales), _ptr(out), F32 if f32 else BF16,
            _row_stride(out), _ptr(flags), _stream(stream))
    return _call(lib.msa_fp8_linear, args, (), what, prepare)


def make_rope(rotary_dim=128, theta=10000.0, layout=ROPE_HALF, scaling=ROPE_NONE, factor=1.0, trained_len=0,
              low_turns=1.0, high_turns=32.0) -> Rope:
    """msa_make_rope: a rotary embedding's layout, rotated dims and (scaled) frequencies."""
    rope = Rope()
    _check(lib.msa_make_rope(ctypes.byref(rope), rotary_dim, theta, layout, scaling, factor, trained_len, low_turns,
                             high_turns), "msa_make_rope")
    return rope


def qkv_rope_insert(dims: Dims, q, k, v, idx_q, idx_k, positions, slot_mapping, nr: NormRope | None, rope: Rope, q_out,
                    idx_q_out, cache: KVCache, idx_cache: IndexCache | None, flags, stream=None, prepare=False):
    """msa_qkv_rope_insert: ``q`` [T, H, D], ``k``, ``v`` [T, G, D], ``idx_q``, ``idx_k`` [T, I, D] may be views of packed
    rows (heads contiguous, tokens apart); ``positions`` [T]."""
    what, D = "msa_qkv_rope_insert", dims.head_dim
    if q is None or q.dim() != 3:
        raise MSAError(ERR_INVALID_ARG, f"{what}: q has to be bfloat16 [tokens, heads, {D}]")
    T = int(q.shape[0])
    for name, t, h in (("q", q, dims.n_heads), ("k", k, dims.n_kv_heads), ("v", v, dims.n_kv_heads),
                       ("idx_q", idx_q, dims.n_idx_heads), ("idx_k", idx_k, dims.n_idx_heads)):
        if t is not None or not name.startswith("idx"):
            _want_rows(what, name, t, "bfloat16", (T, h, D))
    _want(what, "q_out", q_out, "bfloat16", (T, dims.n_heads, D))
    if idx_q_out is not None:
        _want(what, "idx_q_out", idx_q_out, "bfloat16", (T, dims.n_idx_heads, D))
    _want(what, "positions", positions, "int32", (T,))
    _want(what, "slot_mapping", slot_mapping, "int64", (T,))
    _want_cache(what, dims, cache)
    _want_flags(what, flags)
    wts = {n: t for n, t in getattr(nr, "tensors", {}).items() if t is not None}     # (a hand-made struct has addresses only)
    for name, t in wts.items():
        _want(what, name, t, "float32", (D,))
    ics = {}
    if idx_q is not None and idx_cache is not None:
        ics = _want_idx_cache(what, dims, idx_cache)
    _want_on_device(what, q=q, k=k, v=v, idx_q=idx_q, idx_k=idx_k, positions=positions, slot_mapping=slot_mapping,
                    q_out=q_out, idx_q_out=idx_q_out, k_cache=cache.k, v_cache=cache.v, k_scale=cache.k_scale,
                    v_scale=cache.v_scale, flags=flags, **wts, **ics)
    kc = cache.c()
    ic = idx_cache.c() if idx_cache is not None else None
    args = [ctypes.byref(dims)]
    for t in (q, k, v, idx_q, idx_k):
        args += [_ptr(t), 0 if t is None else _row_stride(t)]
    args += [_ptr(positions), _ptr(slot_mapping), T, ctypes.byref(nr) if nr is not None else None, ctypes.byref(rope),
             _ptr(q_out), _ptr(idx_q_out), ctypes.byref(kc), ctypes.byref(ic) if ic is not None else None, _ptr(flags),
             _stream(stream)]
    return _call(lib.msa_qkv_rope_insert, tuple(args), (dims, nr, rope, kc, ic), what, prepare)


def selftest_bounded_wait(flags, stream=None):
    """msa_selftest_bounded_wait: a kernel whose barrier wait runs out (about 2 s)
    and reports MSA_FLAG_TIMEOUT in ``flags``."""
    _check(lib.msa_selftest_bounded_wait(_ptr(flags), _stream(stream)), "msa_selftest_bounded_wait")


def read_device_flags(flags, stream=None) -> int:
    """Synchronises the stream and returns the flag word (0 = no kernel-reported problem)."""
    host = ctypes.c_uint32(0)
    st = lib.msa_read_device_flags(_ptr(flags), ctypes.byref(host), _stream(stream))
    if st not in (OK, ERR_DEVICE_FLAG):
        _check(st, "msa_read_device_flags")
    return int(host.value)


def decode_step(dims: Dims, q, idx_q, q_idx_dtype: int, idx_cache: IndexCache, cache: KVCache, block_table,
                seq_lens, scores, selected, out, lse, workspace, flags, stream=None):
    """The three MSA stages back to back on one stream: score, select, sparse GQA."""
    index_score(dims, idx_q, q_idx_dtype, idx_cache, block_table, seq_lens, scores, flags, stream)
    select_blocks(dims, scores, seq_lens, selected, flags, stream)
    sparse_gqa_decode(dims, q, cache, block_table, seq_lens, selected, out, lse, workspace, flags, stream)
