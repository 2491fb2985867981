"""Python binding of libpa: the C-ABI calls with the same names, taking torch
tensors.  Argument marshalling only: every step of the computation runs in
the library's CUDA kernels.  If libpa.so is missing the calls raise; there is
no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpa.so")

PA_OK, PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_ERR_CUDA = 0, 1, 2, 3
PA_F32, PA_BF16, PA_FP8_E4M3, PA_INT4 = 0, 1, 2, 3
PA_INT4_LIMIT = 16384  # |x / scale| saturates here in a 4-bit cache
PA_DEV_SLOT_RANGE, PA_DEV_BLOCK_RANGE, PA_DEV_QSL, PA_DEV_LENGTHS, PA_DEV_CAPACITY = 1, 2, 4, 8, 16
PA_DEV_TIMEOUT = 32
PA_DEV_POSITION = 64
PA_ROPE_HALVES, PA_ROPE_PAIRS = 0, 1

_DTYPES = {torch.float32: PA_F32, torch.bfloat16: PA_BF16}
_ELEM_BYTES = {PA_F32: 4, PA_BF16: 2}


class pa_layout(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_size", ctypes.c_int), ("block_size", ctypes.c_int),
                ("num_blocks", ctypes.c_int), ("dtype", ctypes.c_int),
                ("cache_dtype", ctypes.c_int), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


class pa_rope(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("cos_sin", ctypes.c_void_p),
                ("max_position", ctypes.c_int), ("rope_size", ctypes.c_int), ("style", ctypes.c_int)]


class pa_latent_layout(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int), ("latent_size", ctypes.c_int),
                ("rope_size", ctypes.c_int), ("block_size", ctypes.c_int),
                ("num_blocks", ctypes.c_int), ("dtype", ctypes.c_int)]


class pa_expanded_layout(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int), ("head_size", ctypes.c_int),
                ("rope_size", ctypes.c_int), ("dtype", ctypes.c_int)] + [
                    (n, ctypes.c_int64) for n in ("q_stride", "q_head_stride", "k_stride", "k_head_stride",
                                                  "kr_stride", "v_stride", "v_head_stride")]


class PaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libpa error {code}: {msg}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Load libpa.so (built in-tree by paged_kv_attention_04_gb300.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m paged_kv_attention_04_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lp = ctypes.POINTER(pa_layout)
        L.pa_cache_write.argtypes = [vp, vp, vp, i32, vp, vp, lp, vp, vp]
        L.pa_cache_write.restype = i32
        L.pa_cache_read.argtypes = [vp, vp, vp, i32, vp, vp, lp, vp, vp]
        L.pa_cache_read.restype = i32
        i64, f32, rp = ctypes.c_int64, ctypes.c_float, ctypes.POINTER(pa_rope)
        llp, elp = ctypes.POINTER(pa_latent_layout), ctypes.POINTER(pa_expanded_layout)
        L.pa_rope_cache_write.argtypes = [vp, i64, vp, i64, vp, i64, rp, vp, i32, vp, vp, vp, lp, vp, vp]
        L.pa_rope_cache_write.restype = i32
        L.pa_latent_write.argtypes = [vp, i64, vp, i64, vp, f32, vp, i64, i64, rp, vp, i32, vp, i64, i64,
                                      vp, llp, vp, vp]
        L.pa_latent_write.restype = i32
        L.pa_latent_read.argtypes = [vp, vp, i32, vp, vp, llp, vp, vp]
        L.pa_latent_read.restype = i32
        L.pa_latent_workspace_size.argtypes = [llp, i32, i32, i32, i32]
        L.pa_latent_workspace_size.restype = sz
        L.pa_latent_forward.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, f32, vp, vp, sz, llp,
                                        vp, vp]
        L.pa_latent_forward.restype = i32
        L.pa_expanded_forward.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, vp, sz,
                                          elp, vp, vp]
        L.pa_expanded_workspace_size.argtypes = [elp, i32, i32]
        L.pa_expanded_workspace_size.restype = sz
        L.pa_expanded_forward.restype = i32
        L.pa_forward_workspace_size.argtypes = [lp, i32, i32, i32]
        L.pa_forward_workspace_size.restype = sz
        L.pa_forward.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, ctypes.c_float,
                                 vp, vp, sz, lp, vp, vp]
        L.pa_forward.restype = i32
        L.pa_last_error.argtypes = []
        L.pa_last_error.restype = ctypes.c_char_p
        L.pa_forward_noalloc.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32,
                                         ctypes.c_float, vp, lp, vp, vp]
        L.pa_forward_noalloc.restype = i32
        L.pa_set_profile_events.argtypes = [vp, vp]
        L.pa_set_profile_events.restype = i32
        L.pa_set_prefill_profile_events.argtypes = [vp, vp]
        L.pa_set_prefill_profile_events.restype = i32
        L.pa_set_prefill_overlap.argtypes = [i32]
        L.pa_set_prefill_overlap.restype = i32
        L.pa_version.argtypes = []
        L.pa_version.restype = i32
        _lib = L
    return _lib


def last_error() -> str:
    return lib().pa_last_error().decode()


def _check(rc: int):
    if rc != PA_OK:
        raise PaError(rc, last_error())


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _on_one_device(**tensors) -> int:
    """Every tensor argument must be a contiguous CUDA tensor, all on one
    device (a host pointer would reach the kernels unchecked).  Returns the
    device's index."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise PaError(PA_ERR_INVALID, f"{name} is not a CUDA tensor")
        if not t.is_contiguous():
            raise PaError(PA_ERR_INVALID, f"{name} is not contiguous")
        d = t.get_device()
        if dev is None:
            dev = d
        elif d != dev:
            raise PaError(PA_ERR_INVALID, f"{name} is on cuda:{d}, expected cuda:{dev}")
    return dev


def _int4_pages(layout: pa_layout, *caches) -> None:
    """The caches of a 4-bit layout must have its pages (their size is not the
    rows' size that the other types share)."""
    if layout.cache_dtype != PA_INT4:
        return
    n = layout.num_blocks * layout.num_kv_heads * layout.head_size * 10
    for c in caches:
        if c.dtype != torch.uint8 or c.numel() != n:
            raise PaError(PA_ERR_INVALID, f"a 4-bit cache is uint8 {cache_shape(layout)}, got {c.dtype} "
                                          f"{tuple(c.shape)}")


def _int64_slots(slot_mapping) -> None:
    if slot_mapping.dtype != torch.int64:
        raise PaError(PA_ERR_INVALID, f"slot_mapping is {slot_mapping.dtype}, expected torch.int64")


def _rows_message(name: str, t, n: int, layout: pa_layout) -> str:
    return (f"{name} is {t.dtype} {tuple(t.shape)}, expected {n} rows of {layout.num_kv_heads} x "
            f"{layout.head_size} of the layout's dtype")


# the current stream's handle without building a Stream object (about a microsecond a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream, dev: int) -> int | None:
    if stream is None:
        return _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _launch(fn, dev: int, stream, *args) -> None:
    """Call fn(*args, stream) with the tensors' device current: the library
    launches on the current device."""
    s = _stream(stream, dev)
    if dev == _current_device():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc != PA_OK:
        raise PaError(rc, last_error())


def make_layout(num_q_heads: int, num_kv_heads: int, head_size: int, num_blocks: int,
                dtype, block_size: int = 16, cache_dtype=None, k_scale: float = 1.0,
                v_scale: float = 1.0) -> pa_layout:
    """Layout of a step; cache_dtype defaults to dtype (PA_FP8_E4M3 for an 8-bit cache,
    PA_INT4 for a 4-bit one)."""
    code = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    if cache_dtype is None:
        ccode = code
    elif isinstance(cache_dtype, torch.dtype):
        ccode = PA_FP8_E4M3 if cache_dtype == torch.uint8 else _DTYPES[cache_dtype]
    else:
        ccode = int(cache_dtype)
    return pa_layout(num_q_heads, num_kv_heads, head_size, block_size, num_blocks, code, ccode,
                     float(k_scale), float(v_scale))


def layout_of(k_cache: torch.Tensor, num_q_heads: int, dtype=None, k_scale: float = 1.0,
              v_scale: float = 1.0) -> pa_layout:
    """Layout of a cache tensor [num_blocks][block_size][num_kv_heads][head_size].  A
    uint8 cache of that shape holds FP8 (E4M3) codes, one of shape
    [num_blocks][num_kv_heads][10 * head_size] the pages of a 4-bit cache; then
    `dtype` (of q/out, default bf16) and the scales apply."""
    if k_cache.dtype == torch.uint8 and k_cache.dim() == 3:
        nb, hkv, page = k_cache.shape
        if page % 10:
            raise PaError(PA_ERR_INVALID, f"a 4-bit page of {page} bytes is not 10 * head_size")
        return make_layout(num_q_heads, hkv, page // 10, nb, dtype or torch.bfloat16, 16, PA_INT4,
                           k_scale, v_scale)
    nb, bs, hkv, d = k_cache.shape
    if k_cache.dtype == torch.uint8:
        return make_layout(num_q_heads, hkv, d, nb, dtype or torch.bfloat16, bs, PA_FP8_E4M3,
                           k_scale, v_scale)
    return make_layout(num_q_heads, hkv, d, nb, k_cache.dtype, bs)


def pa_cache_write(k, v, slot_mapping, k_cache, v_cache, layout: pa_layout,
                   status: torch.Tensor | None = None, stream=None) -> None:
    """Write k[t], v[t] into slot slot_mapping[t] (int64) of the caches (in place); k's
    first dimension counts the tokens."""
    dev = _on_one_device(k=k, v=v, slot_mapping=slot_mapping, k_cache=k_cache, v_cache=v_cache,
                         status=status)
    _int4_pages(layout, k_cache, v_cache)
    _int64_slots(slot_mapping)
    n = k.shape[0]
    if slot_mapping.numel() < n:
        raise PaError(PA_ERR_INVALID, f"{slot_mapping.numel()} slots for {n} tokens")
    elems = n * layout.num_kv_heads * layout.head_size
    for name, t in (("k", k), ("v", v)):
        # (an unquantised cache takes the rows' bits: any type of the same size will do)
        typed = _DTYPES.get(t.dtype) == layout.dtype or (
            layout.cache_dtype == layout.dtype and t.element_size() == _ELEM_BYTES.get(layout.dtype))
        if not typed or t.numel() < elems or (t is k and t.numel() != elems):
            raise PaError(PA_ERR_INVALID, _rows_message(name, t, n, layout))
    _launch(lib().pa_cache_write, dev, stream, _ptr(k), _ptr(v), _ptr(slot_mapping), n,
            _ptr(k_cache), _ptr(v_cache), ctypes.byref(layout), _ptr(status))


def cache_shape(layout: pa_layout) -> tuple:
    """Shape of the k_cache / v_cache tensors of a layout (uint8 for FP8 and 4-bit caches)."""
    if layout.cache_dtype == PA_INT4:
        return (layout.num_blocks, layout.num_kv_heads, 10 * layout.head_size)
    return (layout.num_blocks, layout.block_size, layout.num_kv_heads, layout.head_size)


def pa_cache_read(k_cache, v_cache, slot_mapping, k, v, layout: pa_layout,
                  status: torch.Tensor | None = None, stream=None) -> None:
    """Read slot slot_mapping[t] of the caches into k[t], v[t] (in place); the
    values of a quantised cache come rounded to layout.dtype."""
    dev = _on_one_device(k_cache=k_cache, v_cache=v_cache, slot_mapping=slot_mapping, k=k, v=v,
                         status=status)
    _int4_pages(layout, k_cache, v_cache)
    _int64_slots(slot_mapping)
    n = slot_mapping.shape[0]
    elems = n * layout.num_kv_heads * layout.head_size
    for name, t in (("k", k), ("v", v)):
        if t.numel() != elems or _DTYPES.get(t.dtype) != layout.dtype:
            raise PaError(PA_ERR_INVALID, _rows_message(name, t, n, layout))
    _launch(lib().pa_cache_read, dev, stream, _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping), n,
            _ptr(k), _ptr(v), ctypes.byref(layout), _ptr(status))


def pa_forward_workspace_size(layout: pa_layout, num_seqs: int, num_tokens: int,
                              max_seq_len: int) -> int:
    n = lib().pa_forward_workspace_size(ctypes.byref(layout), int(num_seqs), int(num_tokens),
                                        int(max_seq_len))
    if n == 0:
        raise PaError(PA_ERR_INVALID, last_error())
    return int(n)


def pa_forward(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc,
               max_query_len: int, max_seq_len: int, scale: float, out, workspace,
               layout: pa_layout, status: torch.Tensor | None = None, stream=None) -> None:
    """Attention for every row of the flattened step, written into `out`."""
    dev = _on_one_device(q=q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
                         seq_lens=seq_lens, query_start_loc=query_start_loc, out=out,
                         workspace=workspace, status=status)
    _int4_pages(layout, k_cache, v_cache)
    _launch(lib().pa_forward, dev, stream, _ptr(q), _ptr(k_cache), _ptr(v_cache),
            _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), _ptr(query_start_loc),
            seq_lens.shape[0], q.shape[0], int(max_query_len), int(max_seq_len), float(scale),
            _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
            ctypes.byref(layout), _ptr(status))


def pa_forward_noalloc(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc,
                       max_query_len: int, max_seq_len: int, scale: float, out,
                       layout: pa_layout, status: torch.Tensor | None = None, stream=None) -> None:
    """pa_forward using the library's built-in device scratch instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    dev = _on_one_device(q=q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
                         seq_lens=seq_lens, query_start_loc=query_start_loc, out=out, status=status)
    _int4_pages(layout, k_cache, v_cache)
    _launch(lib().pa_forward_noalloc, dev, stream, _ptr(q), _ptr(k_cache), _ptr(v_cache),
            _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), _ptr(query_start_loc),
            seq_lens.shape[0], q.shape[0], int(max_query_len), int(max_seq_len), float(scale),
            _ptr(out), ctypes.byref(layout), _ptr(status))


def _event_handles(start, stop) -> list:
    """CUDA handles of two torch events (None stays None).  torch creates an
    event's handle on its first record, so unrecorded events are recorded once
    here first."""
    handles = []
    for ev in (start, stop):
        if ev is None:
            handles.append(None)
            continue
        if not ev.cuda_event:
            ev.record()
        handles.append(ev.cuda_event)
    return handles


def pa_set_profile_events(start: "torch.cuda.Event | None", stop: "torch.cuda.Event | None") -> None:
    """Record `start`/`stop` around the decode-attention kernel of later
    pa_forward calls on this thread (None, None turns it off)."""
    _check(lib().pa_set_profile_events(*_event_handles(start, stop)))


def pa_set_prefill_profile_events(start: "torch.cuda.Event | None",
                                  stop: "torch.cuda.Event | None") -> None:
    """Record `start`/`stop` around the tensor-core prefill kernel of later
    pa_forward calls on this thread, on the stream it runs on (None, None
    turns it off)."""
    _check(lib().pa_set_prefill_profile_events(*_event_handles(start, stop)))


def pa_set_prefill_overlap(on: bool) -> None:
    """True (the default): the prefill kernel runs on a side stream beside the
    decode kernel; False: on the caller's stream before it."""
    _check(lib().pa_set_prefill_overlap(1 if on else 0))


def alloc_workspace(layout: pa_layout, num_seqs: int, num_tokens: int, max_seq_len: int,
                    device="cuda") -> torch.Tensor:
    """Caller-owned workspace for pa_forward (torch's allocator aligns to >= 256 bytes)."""
    n = pa_forward_workspace_size(layout, num_seqs, num_tokens, max_seq_len)
    return torch.empty(n, dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- rotation and latent attention

# Small calls are bound by their host time, so what passes is checked by few comparisons a
# tensor, and only what does not is looked into (_explain).

def _explain(name: str, t, dev: int, dtype, shape, inner: int | None) -> None:
    d = t.get_device()
    if d != dev:
        raise PaError(PA_ERR_INVALID, f"{name} is on cuda:{d}, expected cuda:{dev}" if d >= 0 else
                      f"{name} is not a CUDA tensor")
    if t.dtype is not dtype or t.shape != shape:
        raise PaError(PA_ERR_INVALID, f"{name} is {t.dtype} {tuple(t.shape)}, expected {dtype} {tuple(shape)}")
    if inner is None:
        raise PaError(PA_ERR_INVALID, f"{name} is not contiguous")
    raise PaError(PA_ERR_INVALID, f"{name}: its last {inner} dimensions must be contiguous, strides {t.stride()}")


def _device(name: str, t) -> int:
    dev = t.get_device()
    if dev < 0:
        raise PaError(PA_ERR_INVALID, f"{name} is not a CUDA tensor")
    return dev


def _whole(name: str, t, dev: int, dtype, shape) -> int:
    """Pointer of a contiguous tensor of this device, type and shape."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _explain(name, t, dev, dtype, shape, None)
    return t.data_ptr()


def _rows(name: str, t, dev: int, dtype, shape, inner: int, step: int) -> int:
    """Token stride of a tensor [tokens, ...] whose last `inner` dimensions lie side by side, `step`
    elements in all (a single token's is never stepped over)."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _explain(name, t, dev, dtype, shape, inner)
    st = t.stride()
    if shape[-1] > 1 and st[-1] != 1 or inner == 2 and shape[-2] > 1 and st[-2] != shape[-1]:
        _explain(name, t, dev, dtype, shape, inner)
    return st[0] if shape[0] > 1 else step


def _heads(name: str, t, dev: int, dtype, shape) -> tuple:
    """Token and head strides of a tensor [tokens, heads, size] whose last dimension is contiguous."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _explain(name, t, dev, dtype, shape, 1)
    s0, s1, s2 = t.stride()
    if s2 != 1 and shape[2] > 1:
        _explain(name, t, dev, dtype, shape, 1)
    if shape[1] <= 1:
        s1 = shape[2]
    return (s0 if shape[0] > 1 else s1 * shape[1]), s1


def _list_of(name: str, t, dev: int, dtype, least: int, what: str) -> int:
    """Pointer of a contiguous array of at least `least` numbers."""
    if t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous():
        _explain(name, t, dev, dtype, t.shape, None)
    if t.numel() < least:
        raise PaError(PA_ERR_INVALID, f"{t.numel()} {what} for {least} tokens")
    return t.data_ptr()


def _status(status, dev: int) -> int | None:
    if status is None:
        return None
    if status.get_device() != dev or status.dtype is not torch.int32 or status.numel() < 1:
        _explain("status", status, dev, torch.int32, (1,), None)
    return status.data_ptr()


_TORCH = {PA_F32: torch.float32, PA_BF16: torch.bfloat16}


def _torch_dtype(code: int):
    return _TORCH[code] if code in _TORCH else torch.bfloat16  # (a bad code is refused by the library)


def _rope(positions, cos_sin, dev: int, tokens: int, pairs: bool) -> pa_rope:
    at = _list_of("positions", positions, dev, torch.int64, tokens, "positions")
    if cos_sin.dim() != 2:
        raise PaError(PA_ERR_INVALID, f"cos_sin is {tuple(cos_sin.shape)}, expected [max_position, rope_size]")
    rows, size = cos_sin.shape
    return pa_rope(at, _whole("cos_sin", cos_sin, dev, torch.float32, (rows, size)), rows, size,
                   PA_ROPE_PAIRS if pairs else PA_ROPE_HALVES)


def _both(q, q_out) -> None:
    if (q is None) != (q_out is None):
        raise PaError(PA_ERR_INVALID, "q and q_out must both be given, or neither")


def pa_rope_cache_write(q, k, v, positions, cos_sin, slot_mapping, q_out, k_cache, v_cache,
                        layout: pa_layout, pairs: bool = False, status: torch.Tensor | None = None,
                        stream=None) -> None:
    """Rotate q [T, Hq, D] into q_out and k [T, Hkv, D] on its way into the caches, with v
    as it is, at slot_mapping's slots (int64).  The first n = cos_sin.shape[1] dims
    of a head are rotated by row positions[t] (int64) of cos_sin [max_position, n]
    (float32: n / 2 cosines, then n / 2 sines), in pairs (x_i, x_(i + n/2)), or with
    `pairs` (x_2i, x_(2i+1)).  q, k and v may be slices of one projection (any token
    stride, heads contiguous); q_out may be q.  q and q_out None: only k and v."""
    dev, hq, hkv, d = _device("k_cache", k_cache), layout.num_q_heads, layout.num_kv_heads, layout.head_size
    dt, n = _torch_dtype(layout.dtype), k.shape[0]
    held, shape = dt if layout.cache_dtype == layout.dtype else torch.uint8, cache_shape(layout)
    kc = _whole("k_cache", k_cache, dev, held, shape)
    vc = _whole("v_cache", v_cache, dev, held, shape)
    ks = _rows("k", k, dev, dt, (n, hkv, d), 2, hkv * d)
    vs = _rows("v", v, dev, dt, (n, hkv, d), 2, hkv * d)
    _both(q, q_out)
    qp, qs, qo = None, 0, None
    if q is not None:
        qs = _rows("q", q, dev, dt, (n, hq, d), 2, hq * d)
        qp, qo = q.data_ptr(), _whole("q_out", q_out, dev, dt, (n, hq, d))
    slots = _list_of("slot_mapping", slot_mapping, dev, torch.int64, n, "slots")
    rope = _rope(positions, cos_sin, dev, n, pairs)
    _launch(lib().pa_rope_cache_write, dev, stream, qp, qs, k.data_ptr(), ks, v.data_ptr(), vs, rope, slots, n,
            qo, kc, vc, layout, _status(status, dev))


def make_latent_layout(num_heads: int, latent_size: int, num_blocks: int, dtype=torch.bfloat16,
                       rope_size: int = 64, block_size: int = 16) -> pa_latent_layout:
    """Layout of a latent cache and the heads that attend over it."""
    code = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return pa_latent_layout(num_heads, latent_size, rope_size, block_size, num_blocks, code)


def latent_cache_shape(layout: pa_latent_layout) -> tuple:
    """Shape of a latent cache: [num_blocks, block_size, latent_size + rope_size]."""
    return (layout.num_blocks, layout.block_size, layout.latent_size + layout.rope_size)


def latent_layout_of(cache: torch.Tensor, num_heads: int, rope_size: int = 64) -> pa_latent_layout:
    """Layout of a latent cache tensor [num_blocks][block_size][latent_size + rope_size]."""
    nb, bs, row = cache.shape
    return make_latent_layout(num_heads, row - rope_size, nb, cache.dtype, rope_size, bs)


def pa_latent_write(c, k_rope, q, positions, cos_sin, slot_mapping, q_out, cache,
                    layout: pa_latent_layout, norm_weight=None, eps: float = 1e-6,
                    pairs: bool = False, status: torch.Tensor | None = None, stream=None) -> None:
    """Write [c[t], rotated k_rope[t]] into slot slot_mapping[t] (int64) of the latent cache and the
    rotated q[t] (the heads' parts [T, H, rope_size] that meet the key part) into q_out.  With
    norm_weight [latent_size], c is divided by its root mean square (eps inside the root) and
    weighted first.  positions, cos_sin and pairs as for pa_rope_cache_write.  c [T, latent_size],
    k_rope [T, rope_size], q and q_out may be slices (last dimension contiguous); q_out may be
    q.  q and q_out None: only the cache is written."""
    dev, h, size, rs = _device("cache", cache), layout.num_heads, layout.latent_size, layout.rope_size
    dt, n = _torch_dtype(layout.dtype), c.shape[0]
    held = _whole("cache", cache, dev, dt, latent_cache_shape(layout))
    cs = _rows("c", c, dev, dt, (n, size), 1, size)
    ks = _rows("k_rope", k_rope, dev, dt, (n, rs), 1, rs)
    weight = None if norm_weight is None else _whole("norm_weight", norm_weight, dev, dt, (size,))
    _both(q, q_out)
    qp, qs, qh, qo, os, oh = None, 0, 0, None, 0, 0
    if q is not None:
        qs, qh = _heads("q", q, dev, dt, (n, h, rs))
        os, oh = _heads("q_out", q_out, dev, dt, (n, h, rs))
        qp, qo = q.data_ptr(), q_out.data_ptr()
    slots = _list_of("slot_mapping", slot_mapping, dev, torch.int64, n, "slots")
    rope = _rope(positions, cos_sin, dev, n, pairs)
    _launch(lib().pa_latent_write, dev, stream, c.data_ptr(), cs, k_rope.data_ptr(), ks, weight, eps, qp, qs, qh,
            rope, slots, n, qo, os, oh, held, layout, _status(status, dev))


def pa_latent_read(cache, slot_mapping, c, k_rope, layout: pa_latent_layout,
                   status: torch.Tensor | None = None, stream=None) -> None:
    """Read slot slot_mapping[t] of the latent cache into c[t], k_rope[t] (in place)."""
    dev, dt, n = _device("cache", cache), _torch_dtype(layout.dtype), slot_mapping.numel()
    _launch(lib().pa_latent_read, dev, stream, _whole("cache", cache, dev, dt, latent_cache_shape(layout)),
            _list_of("slot_mapping", slot_mapping, dev, torch.int64, n, "slots"), n,
            _whole("c", c, dev, dt, (n, layout.latent_size)),
            _whole("k_rope", k_rope, dev, dt, (n, layout.rope_size)), layout, _status(status, dev))


def pa_latent_workspace_size(layout: pa_latent_layout, num_seqs: int, num_tokens: int,
                             max_query_len: int, max_seq_len: int) -> int:
    n = lib().pa_latent_workspace_size(ctypes.byref(layout), int(num_seqs), int(num_tokens),
                                       int(max_query_len), int(max_seq_len))
    if n == 0:
        raise PaError(PA_ERR_INVALID, last_error())
    return int(n)


def alloc_latent_workspace(layout: pa_latent_layout, num_seqs: int, num_tokens: int,
                           max_query_len: int, max_seq_len: int, device="cuda") -> torch.Tensor:
    """Caller-owned workspace for pa_latent_forward."""
    n = pa_latent_workspace_size(layout, num_seqs, num_tokens, max_query_len, max_seq_len)
    return torch.empty(n, dtype=torch.uint8, device=device)


_CUT_KEYS = 1024  # pa_expanded_forward cuts no shorter requests


def _workspace(workspace, dev: int) -> tuple:
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _explain("workspace", workspace, dev, workspace.dtype, workspace.shape, None)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def pa_latent_forward(q, cache, block_tables, seq_lens, query_start_loc, max_query_len: int,
                      max_seq_len: int, scale: float, out, workspace, layout: pa_latent_layout,
                      status: torch.Tensor | None = None, stream=None) -> None:
    """Attention over a latent cache (absorbed form): q [T, H, latent_size + rope_size], out
    [T, H, latent_size], the rest as for pa_forward."""
    dev, dt, n, b = _device("cache", cache), _torch_dtype(layout.dtype), q.shape[0], seq_lens.shape[0]
    h, size = layout.num_heads, layout.latent_size
    if block_tables.dim() != 2:
        raise PaError(PA_ERR_INVALID, f"block_tables is {tuple(block_tables.shape)}, expected [requests, blocks]")
    width = block_tables.shape[1]
    ws, nbytes = _workspace(workspace, dev)
    _launch(lib().pa_latent_forward, dev, stream, _whole("q", q, dev, dt, (n, h, size + layout.rope_size)),
            _whole("cache", cache, dev, dt, latent_cache_shape(layout)),
            _whole("block_tables", block_tables, dev, torch.int32, (b, width)), width,
            _whole("seq_lens", seq_lens, dev, torch.int32, (b,)),
            _whole("query_start_loc", query_start_loc, dev, torch.int32, (b + 1,)), b, n, max_query_len,
            max_seq_len, scale, _whole("out", out, dev, dt, (n, h, size)), ws, nbytes, layout,
            _status(status, dev))


def pa_expanded_forward(q, k_nope, k_rope, v, query_start_loc, kv_start_loc, max_query_len: int,
                        max_kv_len: int, scale: float, out, workspace: torch.Tensor | None = None,
                        status: torch.Tensor | None = None, stream=None) -> None:
    """Attention in the expanded form: q [T, H, D + 64] against the keys [k_nope [Tk, H, D], k_rope
    [Tk, 64] (shared by the heads)] and values v [Tk, H, D] of ragged requests, causal
    from the bottom right; out [T, H, D].  q, k_nope, k_rope and v may be slices (last
    dimension contiguous).  A workspace of pa_expanded_workspace_size bytes is taken from torch's
    allocator for the call where none is given and it is of use."""
    dev, dt = _device("q", q), q.dtype
    if q.dim() != 3 or k_nope.dim() != 3 or k_rope.dim() != 2 or dt not in _DTYPES:
        raise PaError(PA_ERR_INVALID, f"q is {dt} {tuple(q.shape)}, k_nope {tuple(k_nope.shape)}, k_rope "
                                      f"{tuple(k_rope.shape)}: expected [tokens, heads, size] of float32 or "
                                      "bfloat16 and [tokens, size]")
    (n, h, _), (tk, _, d), rs, b = q.shape, k_nope.shape, k_rope.shape[1], query_start_loc.numel() - 1
    if b < 0:
        raise PaError(PA_ERR_INVALID, "query_start_loc is empty")
    layout = pa_expanded_layout(h, d, rs, _DTYPES[dt], *_heads("q", q, dev, dt, (n, h, d + rs)),
                                *_heads("k_nope", k_nope, dev, dt, (tk, h, d)),
                                _rows("k_rope", k_rope, dev, dt, (tk, rs), 1, rs),
                                *_heads("v", v, dev, dt, (tk, h, d)))
    ws, nbytes = None, 0
    if workspace is not None:
        ws, nbytes = _workspace(workspace, dev)
    elif max_kv_len >= _CUT_KEYS:
        nbytes = lib().pa_expanded_workspace_size(layout, n, max_kv_len)
        if nbytes:
            if stream is None:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
            else:  # of that stream: behind what it still runs, and before what it gets next
                with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                                       else torch.cuda.ExternalStream(int(stream), device=q.device)):
                    workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
            ws = workspace.data_ptr()
    _launch(lib().pa_expanded_forward, dev, stream, q.data_ptr(), k_nope.data_ptr(), k_rope.data_ptr(),
            v.data_ptr(), _whole("query_start_loc", query_start_loc, dev, torch.int32, (b + 1,)),
            _whole("kv_start_loc", kv_start_loc, dev, torch.int32, (b + 1,)), b, n, tk, max_query_len, max_kv_len,
            scale, _whole("out", out, dev, dt, (n, h, d)), ws, nbytes, layout, _status(status, dev))


def pa_expanded_workspace_size(num_heads: int, head_size: int, num_tokens: int, max_kv_len: int,
                               dtype=torch.bfloat16, rope_size: int = 64) -> int:
    """Bytes of workspace that are of use to a pa_expanded_forward of num_tokens tokens (0: none); that of one
    token serves steps of any number."""
    layout = pa_expanded_layout(num_heads, head_size, rope_size, _DTYPES[dtype])
    n = lib().pa_expanded_workspace_size(layout, num_tokens, max_kv_len)
    if n == 0 and last_error():
        raise PaError(PA_ERR_INVALID, last_error())
    return int(n)
