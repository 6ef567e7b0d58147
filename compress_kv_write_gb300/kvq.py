"""Thin Python binding of libkvq.so (include/kvq.h): argument marshalling only.

Every function takes torch CUDA tensors, checks dtype / shape / device, and
passes raw device pointers and the current CUDA stream to the C entry point
of the same name.  All compute runs in the library's kernels; there is no
CPU path.  A missing library raises ImportError.
"""
from __future__ import annotations

import ctypes as C
import functools
import os

import torch

from . import build as _build

V41, V41_FP4 = 1, 2
F32, BF16 = 0, 1
I32, I64 = 0, 1
FLAG_ROPE, FLAG_NORM = 1, 2
ROPE_HALF, ROPE_INVERSE = 1, 2
DEVERR_SLOT, DEVERR_POS, DEVERR_PAGE, DEVERR_LOC, DEVERR_WAIT, DEVERR_STATE, DEVERR_LEN = 1, 2, 4, 8, 16, 32, 64
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CAPACITY, ERR_LAUNCH = 0, 1, 2, 3, 4
HEAD_DIM = 512

_lib = None


class KVQError(RuntimeError):
    def __init__(self, status: int, fn: str):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


_SIGS = {
    "kvq_bytes_per_token": (C.c_size_t, [C.c_int]),
    "kvq_page_bytes": (C.c_size_t, [C.c_int, C.c_int]),
    "kvq_page_bits_supported": (C.c_int, [C.c_int]),
    "kvq_status_string": (C.c_char_p, [C.c_int]),
    "kvq_translate_loc": (C.c_int, [C.c_void_p, C.c_int, C.c_int64, C.c_void_p, C.c_int64,
                                    C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p]),
    "kvq_store": (C.c_int, [C.c_int, C.c_int, C.c_uint, C.c_void_p, C.c_int, C.c_int64,
                            C.c_int64, C.c_void_p, C.c_int, C.c_void_p, C.c_float, C.c_void_p,
                            C.c_int64, C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p,
                            C.c_void_p]),
    "kvq_compress": (C.c_int, [C.c_int, C.c_int, C.c_int, C.c_uint, C.c_void_p, C.c_void_p,
                               C.c_int64, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                               C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p]),
    "kvq_compress_decode": (C.c_int, [C.c_int, C.c_int, C.c_int, C.c_uint, C.c_void_p, C.c_void_p,
                                      C.c_int64, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64,
                                      C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p, C.c_void_p,
                                      C.c_int64, C.c_void_p, C.c_void_p]),
    "kvq_dequant_slots": (C.c_int, [C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_int,
                                    C.c_int64, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p]),
    "kvq_attend_workspace": (C.c_size_t, [C.c_int64]),
    "kvq_attend_wait_limit": (C.c_uint32, [C.c_uint32]),
    "kvq_attend": (C.c_int, [C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_int64, C.c_int64, C.c_int64,
                             C.c_int64, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_int64, C.c_int64,
                             C.c_void_p, C.c_void_p, C.c_float, C.c_void_p, C.c_int, C.c_int64, C.c_int64,
                             C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p]),
    "kvq_mass_workspace": (C.c_size_t, [C.c_int64, C.c_int64, C.c_int64]),
    "kvq_attend_mass": (C.c_int, [C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_int64, C.c_int64, C.c_int64, C.c_int64,
                                  C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_int64, C.c_int64, C.c_void_p,
                                  C.c_void_p, C.c_void_p, C.c_float, C.c_void_p, C.c_int64, C.c_int64, C.c_int64, C.c_void_p,
                                  C.c_void_p, C.c_int64, C.c_float, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p]),
    "kvq_tree_mask": (C.c_int, [C.c_void_p, C.c_int64, C.c_int64, C.c_int64, C.c_void_p, C.c_void_p, C.c_void_p,
                                C.c_void_p, C.c_void_p]),
    "kvq_attend_tree": (C.c_int, [C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_int64, C.c_int64, C.c_int64,
                                  C.c_int64, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_int64, C.c_int64,
                                  C.c_void_p, C.c_void_p, C.c_void_p, C.c_float, C.c_void_p, C.c_int, C.c_int64, C.c_int64,
                                  C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p]),
    "kvq_attend_slots": (C.c_int, [C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_int64, C.c_int64, C.c_int64,
                                   C.c_void_p, C.c_int64, C.c_void_p, C.c_int, C.c_int64, C.c_int64,
                                   C.c_float, C.c_void_p, C.c_int, C.c_int64, C.c_int64, C.c_void_p,
                                   C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p]),
    "kvq_norm_quant": (C.c_int, [C.c_void_p, C.c_int, C.c_int64, C.c_int64, C.c_int64, C.c_void_p, C.c_int64,
                                 C.c_void_p, C.c_int64, C.c_void_p, C.c_float, C.c_void_p, C.c_int64,
                                 C.c_void_p, C.c_int64, C.c_void_p]),
    "kvq_rope_table": (C.c_int, [C.c_void_p, C.c_int64, C.c_int64, C.c_int64, C.c_float, C.c_void_p, C.c_void_p]),
    "kvq_rope": (C.c_int, [C.c_void_p, C.c_int, C.c_int64, C.c_int64, C.c_int64, C.c_int64, C.c_int64, C.c_int64,
                           C.c_int64, C.c_uint, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p, C.c_int64, C.c_int64,
                           C.c_void_p, C.c_void_p]),
    "kvq_evict_select": (C.c_int, [C.c_void_p, C.c_int64, C.c_int64, C.c_int64, C.c_void_p, C.c_void_p, C.c_int64,
                                   C.c_int64, C.c_int64, C.c_int64, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                                   C.c_void_p]),
    "kvq_evict_move": (C.c_int, [C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_int64, C.c_int64,
                                 C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_void_p, C.c_int64, C.c_int64,
                                 C.c_int64, C.c_void_p, C.c_int64, C.c_int64, C.c_int64, C.c_void_p, C.c_void_p,
                                 C.c_int64, C.c_void_p, C.c_void_p]),
    "kvq_dequant": (C.c_int, [C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64,
                              C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p]),
}


def library_path() -> str:
    return _build.SO


def lib():
    """The loaded libkvq.so.  Raises ImportError when it has not been built."""
    global _lib
    if _lib is None:
        path = _build.SO
        if not os.path.exists(path):
            raise ImportError(f"libkvq.so is not built ({path}); run compress_kv_write_gb300.build.build()")
        L = C.CDLL(path)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().kvq_status_string(status).decode()


@functools.lru_cache(maxsize=None)
def bytes_per_token(layout: int) -> int:
    return int(lib().kvq_bytes_per_token(layout))


@functools.lru_cache(maxsize=None)
def page_bytes(layout: int, page_bits: int) -> int:
    return int(lib().kvq_page_bytes(layout, page_bits))


def page_bits_supported(page_bits: int) -> bool:
    return bool(lib().kvq_page_bits_supported(page_bits))


# ------------------------------------------------------------------ helpers

def _check(status: int, fn: str):
    if status != OK:
        raise KVQError(status, fn)


def _cuda(t, name, dtypes=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(dev):
    """The current stream of a device.  torch's raw handle where it has one: a Stream object costs more than the rest
    of a small call's binding."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(dev) if raw is not None else torch.cuda.current_stream(dev).cuda_stream


def _stream(stream):
    return _raw_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def _idx_dtype(t, name):
    if t.dtype == torch.int32:
        return I32
    if t.dtype == torch.int64:
        return I64
    raise TypeError(f"{name} must be int32 or int64")


def _contig1d(t, name):
    if t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D tensor")


def _same_device(first, *others):
    """The device index of `first`; raises when another tensor lives elsewhere."""
    dev = first.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"every tensor must be on {first.device}, got one on {t.device}")
    return dev


def _err_word(err):
    if err is not None:
        _cuda(err, "err", (torch.int32,))
        if err.numel() < 1:
            raise ValueError("err must hold one int32")


def _on(dev, stream, call):
    """status = call(stream pointer) with `dev` current; the default stream is that device's current one."""
    s = _raw_stream(dev) if stream is None else stream.cuda_stream
    if dev == torch.cuda.current_device():
        return call(s)
    with torch.cuda.device(dev):
        return call(s)


# What every call asks torch for, its private form where this torch has that: the public ones cost more than a call's checks.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _raw_stream


def _run(name, dev, stream, *args):
    """The C call `name` with `dev` current, on the stream given or that device's current one (the last argument)."""
    f = getattr(lib(), name)
    s = _current_raw(dev) if stream is None else stream.cuda_stream
    if dev == _current_device():
        st = f(*args, s)
    else:
        with torch.cuda.device(dev):
            st = f(*args, s)
    if st != OK:
        raise KVQError(st, name)


def _at(t, name, dtype, dev=None):
    """The device index of a CUDA tensor of this type (on device `dev`)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")
    d = t.get_device()
    if d < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if dev is not None and d != dev:
        raise ValueError(f"every tensor must be on cuda:{dev}, got {name} on {t.device}")
    return d


def _vec(t, name, dtype, dev, n):
    """Address of a contiguous 1-D tensor of n elements; None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev:
        _at(t, name, dtype, dev)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D tensor of {n}")
    return t.data_ptr()


def _mat(t, name, dtype, dev):
    """(address, rows, width, row stride) of a 2-D tensor with unit inner stride; the stride of a single row is its width."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev:  # _at, which says why, costs a call
        _at(t, name, dtype, dev)
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D with unit inner stride")
    rows, width = shape
    stride = width
    if not t.is_contiguous():
        strides = t.stride()
        if width > 1 and strides[1] != 1:
            raise ValueError(f"{name} must be 2-D with unit inner stride")
        if rows > 1:
            stride = strides[0]
    return t.data_ptr(), rows, width, stride


def _err(err, dev):
    if err is None:
        return None
    _at(err, "err", torch.int32, dev)
    if err.numel() < 1:
        raise ValueError("err must hold one int32")
    return err.data_ptr()


# ------------------------------------------------------------------ entry points

def kvq_translate_loc(full_loc, full_to_swa, out, n=None, err=None, stream=None):
    """out[:n] = full_to_swa[full_loc] (int32), out[n:] = 0; once per step.
    Raises KVQError(ERR_CAPACITY) when n > out.numel()."""
    _cuda(full_loc, "full_loc")
    _cuda(full_to_swa, "full_to_swa", (torch.int32,))
    _cuda(out, "out", (torch.int32,))
    for t, nm in ((full_loc, "full_loc"), (full_to_swa, "full_to_swa"), (out, "out")):
        _contig1d(t, nm)
    n = full_loc.numel() if n is None else int(n)
    st = lib().kvq_translate_loc(_ptr(full_loc), _idx_dtype(full_loc, "full_loc"), n,
                                 _ptr(full_to_swa), full_to_swa.numel(), _ptr(out), out.numel(),
                                 _ptr(err), _stream(stream))
    _check(st, "kvq_translate_loc")
    return out


def kvq_store(layout, page_bits, flags, x, loc, pool, pool_slots, *, norm_weight=None,
              eps=1e-6, cos_sin=None, pos=None, err=None, stream=None):
    """Quantise rows x [n, >=512] (fp32 / bf16) into slots loc of the paged pool."""
    _cuda(x, "x", (torch.float32, torch.bfloat16))
    _cuda(loc, "loc")
    _cuda(pool, "pool", (torch.uint8,))
    if x.dim() != 2 or x.shape[1] < HEAD_DIM or x.stride(1) != 1:
        raise ValueError("x must be [n, >=512] with unit inner stride")
    _contig1d(loc, "loc")
    if loc.numel() != x.shape[0]:
        raise ValueError("loc must hold one slot per row")
    if pool.numel() < pool_slots * bytes_per_token(layout):
        raise ValueError("pool is smaller than pool_slots tokens")
    if norm_weight is not None:
        _cuda(norm_weight, "norm_weight", (torch.float32,))
        if norm_weight.numel() != HEAD_DIM or not norm_weight.is_contiguous():
            raise ValueError("norm_weight must be contiguous [512]")
    rows = 0
    if cos_sin is not None:
        _cuda(cos_sin, "cos_sin", (torch.float32,))
        if cos_sin.dim() != 2 or cos_sin.shape[1] != 64 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be contiguous [rows, 64]")
        rows = cos_sin.shape[0]
    if pos is not None:
        _cuda(pos, "pos", (torch.int32,))
        _contig1d(pos, "pos")
        if pos.numel() != x.shape[0]:
            raise ValueError("pos must hold one position per row")
    st = lib().kvq_store(layout, page_bits, flags, _ptr(x), BF16 if x.dtype == torch.bfloat16 else F32,
                         x.shape[0], x.stride(0), _ptr(loc), _idx_dtype(loc, "loc"),
                         _ptr(norm_weight), float(eps), _ptr(cos_sin), rows, _ptr(pos), _ptr(pool),
                         int(pool_slots), _ptr(err), _stream(stream))
    _check(st, "kvq_store")


def kvq_compress(layout, page_bits, ratio, flags, values, scores, loc, pool, pool_slots, *,
                 cos_sin=None, group_pos=None, err=None, stream=None):
    """Softmax-pool groups of `ratio` rows of values/scores [n*ratio, 512] fp32
    and store the result of group g into slot loc[g]."""
    _cuda(values, "values", (torch.float32,))
    _cuda(scores, "scores", (torch.float32,))
    _cuda(loc, "loc", (torch.int32,))
    _cuda(pool, "pool", (torch.uint8,))
    if values.shape != scores.shape or values.dim() != 2 or values.shape[1] != HEAD_DIM:
        raise ValueError("values and scores must both be [n*ratio, 512]")
    if not values.is_contiguous() or not scores.is_contiguous():
        raise ValueError("values and scores must be contiguous")
    if values.shape[0] % ratio:
        raise ValueError("rows must be a multiple of ratio")
    n_groups = values.shape[0] // ratio
    _contig1d(loc, "loc")
    if loc.numel() != n_groups:
        raise ValueError("loc must hold one slot per group")
    if pool.numel() < pool_slots * bytes_per_token(layout):
        raise ValueError("pool is smaller than pool_slots tokens")
    rows = 0
    if cos_sin is not None:
        _cuda(cos_sin, "cos_sin", (torch.float32,))
        if cos_sin.dim() != 2 or cos_sin.shape[1] != 64 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be contiguous [rows, 64]")
        rows = cos_sin.shape[0]
    if group_pos is not None:
        _cuda(group_pos, "group_pos", (torch.int32,))
        _contig1d(group_pos, "group_pos")
        if group_pos.numel() != n_groups:
            raise ValueError("group_pos must hold one position per group")
    st = lib().kvq_compress(layout, page_bits, ratio, flags, _ptr(values), _ptr(scores), n_groups,
                            _ptr(cos_sin), rows, _ptr(group_pos), _ptr(loc), _ptr(pool),
                            int(pool_slots), _ptr(err), _stream(stream))
    _check(st, "kvq_compress")


def kvq_dequant(layout, page_bits, pool, pool_pages, page_table, out, err=None, stream=None):
    """out [n_tokens, >=512] bf16 <- pages page_table[t >> page_bits] of pool."""
    _cuda(pool, "pool", (torch.uint8,))
    _cuda(page_table, "page_table", (torch.int32,))
    _cuda(out, "out", (torch.bfloat16,))
    _contig1d(page_table, "page_table")
    if out.dim() != 2 or out.shape[1] < HEAD_DIM or out.stride(1) != 1:
        raise ValueError("out must be [n_tokens, >=512] bf16 with unit inner stride")
    n_tokens = out.shape[0]
    if page_table.numel() * (1 << page_bits) != n_tokens:
        raise ValueError("out must have page_table.numel() * 2^page_bits rows")
    if pool.numel() < pool_pages * page_bytes(layout, page_bits):
        raise ValueError("pool is smaller than pool_pages pages")
    st = lib().kvq_dequant(layout, page_bits, _ptr(pool), int(pool_pages), _ptr(page_table),
                           n_tokens, _ptr(out), out.stride(0), _ptr(err), _stream(stream))
    _check(st, "kvq_dequant")


def kvq_dequant_slots(layout, page_bits, pool, pool_slots, slots, out, err=None, stream=None):
    """out [n, >=512] bf16 <- the tokens in slots [n] (int32/int64); slot -1 gives a zero row."""
    _cuda(pool, "pool", (torch.uint8,))
    _cuda(slots, "slots")
    _cuda(out, "out", (torch.bfloat16,))
    _contig1d(slots, "slots")
    if out.dim() != 2 or out.shape[1] < HEAD_DIM or out.stride(1) != 1 or out.shape[0] != slots.numel():
        raise ValueError("out must be [slots.numel(), >=512] bf16 with unit inner stride")
    if pool.numel() < pool_slots * bytes_per_token(layout):
        raise ValueError("pool is smaller than pool_slots tokens")
    st = lib().kvq_dequant_slots(layout, page_bits, _ptr(pool), int(pool_slots), _ptr(slots),
                                 _idx_dtype(slots, "slots"), slots.numel(), _ptr(out), out.stride(0),
                                 _ptr(err), _stream(stream))
    _check(st, "kvq_dequant_slots")


def kvq_compress_decode(layout, page_bits, ratio, flags, values, scores, state, count, loc, pool,
                        pool_slots, *, req=None, cos_sin=None, group_pos=None, err=None, stream=None):
    """One decode step of the ratio-r compressor: request i appends row
    (values[i], scores[i]) to the open group held in state[req[i]] /
    count[req[i]]; a group's ratio-th row pools, quantises and stores it into
    slot loc[i]."""
    _cuda(values, "values", (torch.float32,))
    _cuda(scores, "scores", (torch.float32,))
    _cuda(state, "state", (torch.float32,))
    _cuda(count, "count", (torch.int32,))
    _cuda(loc, "loc", (torch.int32,))
    _cuda(pool, "pool", (torch.uint8,))
    if values.shape != scores.shape or values.dim() != 2 or values.shape[1] != HEAD_DIM:
        raise ValueError("values and scores must both be [n, 512]")
    if not values.is_contiguous() or not scores.is_contiguous():
        raise ValueError("values and scores must be contiguous")
    n = values.shape[0]
    if state.dim() != 3 or state.shape[1:] != (3, HEAD_DIM) or not state.is_contiguous():
        raise ValueError("state must be contiguous [n_state, 3, 512]")
    _contig1d(count, "count")
    if count.numel() != state.shape[0]:
        raise ValueError("count must hold one entry per state row")
    _contig1d(loc, "loc")
    if loc.numel() != n:
        raise ValueError("loc must hold one slot per request")
    if req is not None:
        _cuda(req, "req", (torch.int32,))
        _contig1d(req, "req")
        if req.numel() != n:
            raise ValueError("req must hold one state index per request")
    if pool.numel() < pool_slots * bytes_per_token(layout):
        raise ValueError("pool is smaller than pool_slots tokens")
    rows = 0
    if cos_sin is not None:
        _cuda(cos_sin, "cos_sin", (torch.float32,))
        if cos_sin.dim() != 2 or cos_sin.shape[1] != 64 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be contiguous [rows, 64]")
        rows = cos_sin.shape[0]
    if group_pos is not None:
        _cuda(group_pos, "group_pos", (torch.int32,))
        _contig1d(group_pos, "group_pos")
        if group_pos.numel() != n:
            raise ValueError("group_pos must hold one position per request")
    st = lib().kvq_compress_decode(layout, page_bits, ratio, flags, _ptr(values), _ptr(scores), n,
                                   _ptr(state), _ptr(count), _ptr(req), state.shape[0], _ptr(cos_sin),
                                   rows, _ptr(group_pos), _ptr(loc), _ptr(pool), int(pool_slots),
                                   _ptr(err), _stream(stream))
    _check(st, "kvq_compress_decode")


def attend_workspace(rows):
    """Bytes of workspace for kvq_attend (rows = q_len * heads) or kvq_attend_slots (rows = heads)."""
    return int(lib().kvq_attend_workspace(int(rows)))


def attend_wait_limit(tries):
    """Sets how often a wait inside the attention kernels tries before a later call gives up with DEVERR_WAIT
    (2^20 by default, at most 2^24; 0: every call gives up) and returns the limit before."""
    if not 0 <= tries < 1 << 32:
        raise ValueError("tries must be a 32-bit count")
    return int(lib().kvq_attend_wait_limit(int(tries)))


def _attend_rows(q, out, lse, workspace, err):
    """Checks what both attention calls share; returns (tokens, heads, strides of q and out, device, out dtype)."""
    dev = _at(q, "q", torch.bfloat16)
    bf16 = isinstance(out, torch.Tensor) and out.dtype is torch.bfloat16
    _at(out, "out", torch.bfloat16 if bf16 else torch.float32, dev)
    _at(workspace, "workspace", torch.uint8, dev)
    shape, qs, outs = q.shape, q.stride(), out.stride()
    if len(shape) != 3 or shape[2] != HEAD_DIM or qs[2] != 1:
        raise ValueError("q must be [tokens, heads, 512] with unit inner stride")
    if out.shape != shape or outs[2] != 1:
        raise ValueError("out must have q's shape and unit inner stride")
    n, h, _ = shape
    if n and h:
        lo, hi = ((outs[0], n), (outs[1], h)) if outs[0] <= outs[1] else ((outs[1], h), (outs[0], n))
        if (lo[1] > 1 and lo[0] < HEAD_DIM) or (hi[1] > 1 and hi[0] < (lo[1] - 1) * lo[0] + HEAD_DIM):
            raise ValueError("rows of out must not overlap")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if lse is not None:
        _at(lse, "lse", torch.float32, dev)
        if lse.shape != (n, h) or not lse.is_contiguous():
            raise ValueError("lse must be contiguous [tokens, heads]")
    _err(err, dev)
    return n, h, qs, outs, dev, BF16 if bf16 else F32


def _paged(layout, page_bits, dev, n, q_len, pool, pool_pages, page_table, kv_len, req):
    """Checks what the calls over pages share; returns the addresses of pool, table, req and kv_len, the table's rows, width
    and row stride, and the sequences."""
    _at(pool, "pool", torch.uint8, dev)
    table, rows, width, stride = _mat(page_table, "page_table", torch.int32, dev)
    _at(kv_len, "kv_len", torch.int32, dev)
    if len(kv_len.shape) != 1 or not kv_len.is_contiguous():
        raise ValueError("kv_len must be a contiguous 1-D tensor")
    n_seq = kv_len.shape[0]
    if q_len < 1 or n != n_seq * q_len:
        raise ValueError("q must hold q_len rows per entry of kv_len")
    req = _vec(req, "req", torch.int32, dev, n_seq)
    if req is None and rows < n_seq:
        raise ValueError("page_table must hold one row per sequence")
    if not pool.is_contiguous() or pool.numel() < pool_pages * page_bytes(layout, page_bits):
        raise ValueError("pool must be contiguous and hold pool_pages pages")
    return pool.data_ptr(), table, req, kv_len.data_ptr(), rows, width, stride, n_seq


def kvq_attend(layout, page_bits, q, pool, pool_pages, page_table, kv_len, out, workspace, *, scale, q_len=1,
               req=None, lse=None, err=None, stream=None):
    """Latent attention of q [n_seq * q_len, heads, 512] bf16 over the paged pool: out (bf16 or fp32) of q's
    shape and, if lse [n_seq * q_len, heads] fp32 is given, the natural-log sums.  page_table [rows, width]
    int32, row req[i] (req None: row i) for sequence i; kv_len [n_seq] int32 cached tokens; query token j of a
    sequence sees the first kv_len - (q_len - 1 - j).  workspace: attend_workspace(q_len * heads) bytes."""
    n, heads, qs, outs, dev, out_dtype = _attend_rows(q, out, lse, workspace, err)
    pool, table, req, kv_len, rows, width, ts, n_seq = _paged(layout, page_bits, dev, n, q_len, pool, pool_pages, page_table,
                                                              kv_len, req)
    _run("kvq_attend", dev, stream, layout, page_bits, q.data_ptr(), qs[0], qs[1], n_seq, q_len, heads, pool, int(pool_pages),
         table, rows, width, ts, req, kv_len, float(scale), out.data_ptr(), out_dtype, outs[0], outs[1], _ptr(lse),
         workspace.data_ptr(), workspace.numel(), _ptr(err))
    return out


def kvq_tree_mask(parent, mask, *, kv_len=None, pos=None, err=None, stream=None):
    """mask [n_seq, q_len, ceil(q_len / 64)] int64 <- which drafted tokens each one sees (itself and its ancestors), from
    parent [n_seq, q_len] int32 (-1: the last token before the tree); pos [n_seq, q_len] int32 <- kv_len - q_len + depth, with
    the kv_len that a sequence has, or had it not been cut (kvq_evict_move) would have: positions go on where they were."""
    dev = _at(parent, "parent", torch.int32)
    parent_ptr, n_seq, q_len, stride = _mat(parent, "parent", torch.int32, dev)
    _at(mask, "mask", torch.int64, dev)
    if mask.shape != (n_seq, q_len, (q_len + 63) // 64) or not mask.is_contiguous():
        raise ValueError("mask must be contiguous [n_seq, q_len, ceil(q_len / 64)]")
    if pos is not None:
        _at(pos, "pos", torch.int32, dev)
        if pos.shape != (n_seq, q_len) or not pos.is_contiguous():
            raise ValueError("pos must be contiguous [n_seq, q_len]")
    _run("kvq_tree_mask", dev, stream, parent_ptr, n_seq, q_len, stride, _vec(kv_len, "kv_len", torch.int32, dev, n_seq),
         mask.data_ptr(), _ptr(pos), _err(err, dev))
    return mask


def _tree_words(mask, dev):
    """Checks a tree's masks; returns the drafted tokens of a sequence."""
    _at(mask, "mask", torch.int64, dev)
    shape = mask.shape
    if len(shape) != 3 or shape[2] != (shape[1] + 63) // 64 or not mask.is_contiguous():
        raise ValueError("mask must be contiguous [n_seq, q_len, ceil(q_len / 64)]")
    return shape[1]


def kvq_attend_tree(layout, page_bits, q, pool, pool_pages, page_table, kv_len, mask, out, workspace, *, scale, req=None,
                    lse=None, err=None, stream=None):
    """kvq_attend of a tree of drafted tokens, the last q_len of a sequence's cached tokens: query token j sees all tokens
    before them and those of them whose bits are set in mask[i, j] ([n_seq, q_len, ceil(q_len / 64)] int64)."""
    n, heads, qs, outs, dev, out_dtype = _attend_rows(q, out, lse, workspace, err)
    q_len = _tree_words(mask, dev)
    pool, table, req, kv_len, rows, width, ts, n_seq = _paged(layout, page_bits, dev, n, q_len, pool, pool_pages, page_table,
                                                              kv_len, req)
    if mask.shape[0] != n_seq:
        raise ValueError("mask must hold one tree per sequence")
    _run("kvq_attend_tree", dev, stream, layout, page_bits, q.data_ptr(), qs[0], qs[1], n_seq, q_len, heads, pool,
         int(pool_pages), table, rows, width, ts, req, kv_len, mask.data_ptr(), float(scale), out.data_ptr(), out_dtype, outs[0],
         outs[1], _ptr(lse), workspace.data_ptr(), workspace.numel(), _ptr(err))
    return out


def kvq_attend_slots(layout, page_bits, q, pool, pool_slots, slots, out, workspace, *, scale, lse=None, err=None,
                     stream=None):
    """kvq_attend of query token i over the tokens in slots[i] ([tokens, n_sel] int32 / int64; -1 is padding).
    workspace: attend_workspace(heads) bytes."""
    n, heads, qs, outs, dev, out_dtype = _attend_rows(q, out, lse, workspace, err)
    _cuda(pool, "pool", (torch.uint8,))
    _cuda(slots, "slots")
    dt = _idx_dtype(slots, "slots")
    if slots.dim() != 2 or slots.shape[0] != n or (slots.numel() and slots.stride(1) != 1 and slots.shape[1] > 1):
        raise ValueError("slots must be [tokens, n_sel] with unit inner stride")
    if not pool.is_contiguous() or pool.numel() < pool_slots * bytes_per_token(layout):
        raise ValueError("pool must be contiguous and hold pool_slots tokens")
    _same_device(q, pool, slots)
    st = _on(dev, stream, lambda s: lib().kvq_attend_slots(
        layout, page_bits, _ptr(q), qs[0], qs[1], n, heads, _ptr(pool), int(pool_slots), _ptr(slots),
        dt, slots.shape[1], slots.stride(0), float(scale), _ptr(out), out_dtype, outs[0], outs[1],
        _ptr(lse), _ptr(workspace), workspace.numel(), _ptr(err), s))
    _check(st, "kvq_attend_slots")
    return out


def _rows2d(t, name, n, width):
    if t.dim() != 2 or t.shape[0] != n or t.shape[1] < width or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [{n}, >={width}] with unit inner stride")


def kvq_norm_quant(x, weight, codes, scales, *, eps=1e-6, residual=None, residual_out=None, stream=None):
    """codes [n, dim] e4m3 bytes and scales [n, dim / 32] ue8m0 bytes of RMSNorm(x + residual) * weight;
    residual_out (which may be residual or x) gets the sum in x's type.  dim is weight.numel()."""
    _cuda(x, "x", (torch.float32, torch.bfloat16))
    _cuda(weight, "weight", (torch.float32,))
    _cuda(codes, "codes", (torch.uint8,))
    _cuda(scales, "scales", (torch.uint8,))
    _contig1d(weight, "weight")
    dim = weight.numel()
    if x.dim() != 2:
        raise ValueError("x must be [n, >=dim]")
    n = x.shape[0]
    _rows2d(x, "x", n, dim)
    _rows2d(codes, "codes", n, dim)
    _rows2d(scales, "scales", n, dim // 32)
    if (residual is None) != (residual_out is None):
        raise ValueError("residual and residual_out come together")
    if residual is not None:
        _cuda(residual, "residual", (x.dtype,))
        _cuda(residual_out, "residual_out", (x.dtype,))
        _rows2d(residual, "residual", n, dim)
        _rows2d(residual_out, "residual_out", n, dim)
    dev = _same_device(x, weight, codes, scales, residual, residual_out)
    st = _on(dev, stream, lambda s: lib().kvq_norm_quant(
        _ptr(x), BF16 if x.dtype == torch.bfloat16 else F32, n, dim, x.stride(0), _ptr(residual),
        residual.stride(0) if residual is not None else 0, _ptr(residual_out),
        residual_out.stride(0) if residual is not None else 0, _ptr(weight), float(eps), _ptr(codes),
        codes.stride(0), _ptr(scales), scales.stride(0), s))
    _check(st, "kvq_norm_quant")


def kvq_rope_table(freq, table, *, first=0, amplitude=1.0, stream=None):
    """table [rows, rot] fp32 <- amplitude * cosines, then sines, of (first + row) * freq (freq [rot / 2] fp64)."""
    dev = _at(freq, "freq", torch.float64)
    to, rows, rot, stride = _mat(table, "table", torch.float32, dev)
    if stride != rot:
        raise ValueError("table must be contiguous [rows, rot]")
    _run("kvq_rope_table", dev, stream, _vec(freq, "freq", torch.float64, dev, rot // 2), rot, int(first), rows,
         float(amplitude), to)
    return table


def kvq_rope(x, pos, cos_sin, out, *, start, half=False, inverse=False, err=None, stream=None):
    """out <- x [tokens, heads, dim] (fp32 / bf16) with dims start .. start + rot - 1 rotated by row pos[token] of cos_sin
    [rows, rot], interleaved pairs or halves; with `inverse` by the transpose, which turns back what a table of amplitude 1
    turned (what one of amplitude A turned, a table of 1 / A does: with the same one A * A stays).  out may be x itself."""
    bf16 = isinstance(x, torch.Tensor) and x.dtype is torch.bfloat16
    dtype = torch.bfloat16 if bf16 else torch.float32
    dev = _at(x, "x", dtype)
    _at(out, "out", dtype, dev)
    shape, xs, outs = x.shape, x.stride(), out.stride()
    if len(shape) != 3 or (shape[2] > 1 and xs[2] != 1):
        raise ValueError("x must be [tokens, heads, dim] with unit inner stride")
    if out.shape != shape or (shape[2] > 1 and outs[2] != 1):
        raise ValueError("out must have x's shape and unit inner stride")
    table, rows, rot, stride = _mat(cos_sin, "cos_sin", torch.float32, dev)
    if stride != rot:
        raise ValueError("cos_sin must be contiguous [rows, rot]")
    flags = (ROPE_HALF if half else 0) | (ROPE_INVERSE if inverse else 0)
    _run("kvq_rope", dev, stream, x.data_ptr(), BF16 if bf16 else F32, shape[0], shape[1], shape[2], xs[0], xs[1], int(start),
         rot, flags, table, rows, _vec(pos, "pos", torch.int32, dev, shape[0]), out.data_ptr(), outs[0], outs[1],
         _err(err, dev))
    return out


def mass_workspace(n_seq, rows, max_len):
    """Bytes of workspace for kvq_attend_mass: n_seq sequences, rows = q_len * heads, max_len tokens a row of the table (or of
    the weights, where that is less) can have."""
    return int(lib().kvq_mass_workspace(int(n_seq), int(rows), int(max_len)))


def kvq_attend_mass(layout, page_bits, q, lse, pool, pool_pages, page_table, kv_len, mass, workspace=None, *, scale, q_len=1,
                    mask=None, req=None, rows=None, prev=None, decay=1.0, err=None, stream=None):
    """mass [rows, width] fp32 (row rows[i], or i) <- decay * prev + the weight of each of a sequence's cached tokens in
    kvq_attend, or with mask in kvq_attend_tree, summed over heads and query tokens; q, pool, page_table, kv_len, scale, q_len
    (with mask: mask.shape[1]), req and lse as in that call.  prev may be mass itself, or None: no weights from before.
    workspace: mass_workspace(n_seq, q_len * heads, max_len)."""
    dev = _at(q, "q", torch.bfloat16)
    shape, qs = q.shape, q.stride()
    if len(shape) != 3 or shape[2] != HEAD_DIM or qs[2] != 1:
        raise ValueError("q must be [tokens, heads, 512] with unit inner stride")
    n, heads, _ = shape
    _at(lse, "lse", torch.float32, dev)
    if lse.shape != (n, heads) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous [tokens, heads]")
    if mask is not None:
        q_len = _tree_words(mask, dev)
    pool, table, req, kv_len, t_rows, width, ts, n_seq = _paged(layout, page_bits, dev, n, q_len, pool, pool_pages, page_table,
                                                                kv_len, req)
    if mask is not None and mask.shape[0] != n_seq:
        raise ValueError("mask must hold one tree per sequence")
    to, m_rows, m_width, m_stride = _mat(mass, "mass", torch.float32, dev)
    rows = _vec(rows, "rows", torch.int32, dev, n_seq)
    if rows is None and m_rows < n_seq:
        raise ValueError("mass must hold one row per sequence")
    before = p_stride = None
    if prev is not None:
        before, p_rows, p_width, p_stride = _mat(prev, "prev", torch.float32, dev)
        if p_rows != m_rows or p_width != m_width:
            raise ValueError("prev must have mass's shape")
    ws = size = 0
    if workspace is not None:
        _at(workspace, "workspace", torch.uint8, dev)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        ws, size = workspace.data_ptr(), workspace.numel()
    _run("kvq_attend_mass", dev, stream, layout, page_bits, q.data_ptr(), qs[0], qs[1], n_seq, q_len, heads, lse.data_ptr(), pool,
         int(pool_pages), table, t_rows, width, ts, req, kv_len, _ptr(mask), float(scale), to, m_rows, m_width, m_stride, rows,
         before, p_stride or 0, float(decay), ws, size, _err(err, dev))
    return mass


def kvq_evict_select(mass, kv_len, kept, count, *, first=0, last=0, rows=None, err=None, stream=None):
    """kept [n_seq, keep] int32 <- the tokens that stay of each sequence, ascending, then -1: the first and last few and,
    of the others, those of most weight in mass [rows, width] fp32 (row rows[i], or i); count [n_seq] int32 of them."""
    dev = _at(mass, "mass", torch.float32)
    of, m_rows, m_width, m_stride = _mat(mass, "mass", torch.float32, dev)
    to, n_seq, keep, k_stride = _mat(kept, "kept", torch.int32, dev)
    rows = _vec(rows, "rows", torch.int32, dev, n_seq)
    if rows is None and m_rows < n_seq:
        raise ValueError("mass must hold one row per sequence")
    _run("kvq_evict_select", dev, stream, of, m_rows, m_width, m_stride, rows, _vec(kv_len, "kv_len", torch.int32, dev, n_seq),
         n_seq, keep, int(first), int(last), to, k_stride, _vec(count, "count", torch.int32, dev, n_seq), _err(err, dev))
    return kept, count


def kvq_evict_move(layout, page_bits, pool, pool_pages, page_table, new_table, kept, *, req=None, mass=None, rows=None,
                   mass_out=None, err=None, stream=None):
    """Moves token kept[i, k] of sequence i (page_table row req[i], or i) to token k of the pages new_table[i], and its
    weight to mass_out[i, k] where mass and mass_out are given.  Rows keep the rotation of the positions that they had: later
    tokens' positions go on from the length without the cut, the calls over pages take the cut one."""
    dev = _at(pool, "pool", torch.uint8)
    table, t_rows, t_width, t_stride = _mat(page_table, "page_table", torch.int32, dev)
    new, n_rows, n_width, n_stride = _mat(new_table, "new_table", torch.int32, dev)
    of, n_seq, keep, k_stride = _mat(kept, "kept", torch.int32, dev)
    if n_rows != n_seq:
        raise ValueError("new_table must hold one row per sequence")
    req = _vec(req, "req", torch.int32, dev, n_seq)
    if req is None and t_rows < n_seq:
        raise ValueError("page_table must hold one row per sequence")
    if (mass is None) != (mass_out is None):
        raise ValueError("mass and mass_out come together")
    weights, m_rows, m_width, m_stride, w_out, o_stride = None, 0, 0, 0, None, 0
    rows = _vec(rows, "rows", torch.int32, dev, n_seq)
    if mass is not None:
        weights, m_rows, m_width, m_stride = _mat(mass, "mass", torch.float32, dev)
        w_out, o_rows, o_width, o_stride = _mat(mass_out, "mass_out", torch.float32, dev)
        if o_rows != n_seq or o_width < keep:
            raise ValueError("mass_out must hold one row of kept weights per sequence")
        if rows is None and m_rows < n_seq:
            raise ValueError("mass must hold one row per sequence")
    elif rows is not None:
        raise ValueError("rows are of mass")
    if not pool.is_contiguous() or pool.numel() < pool_pages * page_bytes(layout, page_bits):
        raise ValueError("pool must be contiguous and hold pool_pages pages")
    _run("kvq_evict_move", dev, stream, layout, page_bits, pool.data_ptr(), int(pool_pages), table, t_rows, t_width, t_stride, req,
         new, n_width, n_stride, of, n_seq, keep, k_stride, weights, m_rows, m_width, m_stride, rows, w_out, o_stride,
         _err(err, dev))
