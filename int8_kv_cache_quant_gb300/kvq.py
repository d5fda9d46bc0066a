"""Python binding of libkvq (include/kvq.h): argument marshalling only.

Every function here has the name of the C entry point it calls.  torch supplies device
memory and the current stream; all arithmetic runs in libkvq's CUDA kernels.  There is no
CPU fallback: if libkvq.so is missing or the call fails, an exception is raised.

A call runs on the current stream, or on `stream` where one is given.  What it allocates (a workspace, a result
that was not passed in) belongs to that stream; tensors that are passed in are ordered before and after the call
by the caller, as with torch's own operators.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")

BLOCK_SIZE = 16
PV_TILE = 128

_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape or option",
           3: "device pointer not 16-byte aligned", 4: "workspace missing or too small",
           5: "CUDA launch or runtime error"}

DEV_BAD_BLOCK, DEV_BAD_POS, DEV_TIMEOUT, DEV_BAD_CELL, DEV_BAD_SEQ, DEV_BAD_SCALE = 0x1, 0x2, 0x4, 0x8, 0x10, 0x20


class KvqError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__("%s failed: %s (status %d)" % (fn, _STATUS.get(status, "?"), status))
        self.status = status


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _Int32:
    """An int32 argument of the calls that answer a size, checked as it is converted."""

    @classmethod
    def from_param(cls, v):
        _fit("kvq", v)
        return ctypes.c_int32(int(v))


class _DecodeOpts(ctypes.Structure):
    _fields_ = [("split_rows", ctypes.c_int32), ("route_threshold", ctypes.c_int32),
                ("force_route", ctypes.c_int32), ("stage1_event_begin", ctypes.c_void_p),
                ("stage1_event_end", ctypes.c_void_p), ("launches", ctypes.POINTER(ctypes.c_int32))]


class _RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double), ("original_len", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("divisors", ctypes.POINTER(ctypes.c_double))]


ROPE_HALF, ROPE_INTERLEAVED = 0, 1
_ROPE_ORDERS, _ROPE_LADDERS = {"chunked": 0, "turns": 1}, {"shared": 0, "per_axis": 1}
_ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4, "divisors": 5}

_lib = None


def lib():
    """The loaded libkvq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libkvq.so is not built (%s); run int8_kv_cache_quant_gb300.build.build()"
                               % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        cp = ctypes.POINTER(_Cache)
        L.kvq_version.restype = ctypes.c_int
        L.kvq_status_string.restype = ctypes.c_char_p
        L.kvq_status_string.argtypes = [ctypes.c_int]
        L.kvq_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), vp]
        L.kvq_quant_write.argtypes = [cp, vp, vp, i32, vp, vp, vp, i32, i32, vp]
        L.kvq_rope_quant_write.argtypes = [cp, vp, i32, vp, vp, i32, vp, vp, vp, i32, i32, vp, i32, i32,
                                           vp, vp, vp, vp]
        L.kvq_attn_prefill_int8_qcodes.argtypes = [cp, vp, vp, i32, i32, i32, vp, i32, f32, vp, vp, sz, vp]
        L.kvq_decode_workspace_bytes.restype = sz
        L.kvq_decode_auto_split_rows.restype = i32
        L.kvq_decode_auto_split_rows.argtypes = [_Int32, _Int32, _Int32, _Int32, _Int32]
        L.kvq_prefill_split_tiles.restype = i32
        L.kvq_device_accessible.restype = i32
        L.kvq_device_accessible.argtypes = [ctypes.c_void_p]
        L.kvq_prefill_split_tiles.argtypes = [_Int32, _Int32, _Int32, _Int32]
        L.kvq_decode_workspace_bytes.argtypes = [_Int32, _Int32, _Int32, _Int32, ctypes.POINTER(_DecodeOpts)]
        L.kvq_attn_decode_int8kv.argtypes = [cp, vp, i32, i32, vp, i32, vp, i32, f32, vp, vp, sz,
                                             ctypes.POINTER(_DecodeOpts), vp]
        L.kvq_attn_decode_int8kv_noalloc.argtypes = [cp, vp, i32, i32, vp, i32, vp, i32, f32, vp,
                                                     ctypes.POINTER(_DecodeOpts), vp]
        L.kvq_verify_workspace_bytes.restype = sz
        L.kvq_verify_workspace_bytes.argtypes = [_Int32, _Int32, _Int32, _Int32, _Int32, ctypes.POINTER(_DecodeOpts)]
        L.kvq_attn_verify_int8kv.argtypes = [cp, vp, i32, i32, i32, vp, i32, vp, i32, f32, vp, vp, sz,
                                             ctypes.POINTER(_DecodeOpts), vp]
        L.kvq_decode_step_int8kv.argtypes = [cp, vp, vp, vp, i32, i32, i32, vp, i32, vp, i32, f32, vp, vp, sz,
                                             ctypes.POINTER(_DecodeOpts), vp]
        i64 = ctypes.c_int64
        L.kvq_step_accum_workspace_bytes.restype = sz
        L.kvq_step_accum_workspace_bytes.argtypes = [_Int32, _Int32, _Int32, _Int32, _Int32, ctypes.POINTER(_DecodeOpts)]
        L.kvq_decode_step_accum_int8kv.argtypes = [cp, vp, vp, vp, i32, i32, i32, vp, i32, vp, i32, f32, vp, vp, i64,
                                                   vp, vp, vp, sz, ctypes.POINTER(_DecodeOpts), vp]
        L.kvq_step_window_workspace_bytes.restype = sz
        L.kvq_step_window_workspace_bytes.argtypes = [_Int32] * 8 + [ctypes.POINTER(_DecodeOpts)]
        L.kvq_decode_step_window_int8kv.argtypes = [cp, vp, vp, vp, i32, i32, i32, vp, i32, vp, i32, f32, i32, i32, vp, vp, sz,
                                                    ctypes.POINTER(_DecodeOpts), vp]
        L.kvq_chunk_weights_workspace_bytes.restype = sz
        L.kvq_chunk_weights_workspace_bytes.argtypes = [_Int32, _Int32, _Int32, _Int32, _Int32]
        L.kvq_attn_chunk_weights_int8kv.argtypes = [cp, vp, i32, i32, i32, vp, i32, f32, vp, i64, vp, sz, vp]
        L.kvq_evict_workspace_bytes.restype = sz
        L.kvq_evict_workspace_bytes.argtypes = [_Int32, _Int32, _Int32, _Int32]
        L.kvq_cache_evict.argtypes = [cp, i32, vp, i32, vp, i32, i32, i32, i32, vp, vp, i64, vp, vp, i64, vp, vp, sz, vp]
        L.kvq_rope_phases.argtypes = [i32, ctypes.c_double, ctypes.POINTER(_RopeScaling),
                                      ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_float)]
        L.kvq_rope_bf16.argtypes = [vp, vp, i64, i64, i32, vp, vp, i64, i64, i32, i32, i32, vp, vp, i32, i32, i32, f32, vp]
        L.kvq_rope_axes_phases.argtypes = [i32, ctypes.POINTER(i32), i32, i32, ctypes.c_double, ctypes.POINTER(_RopeScaling),
                                           ctypes.POINTER(ctypes.c_uint64), vp, ctypes.POINTER(ctypes.c_float)]
        L.kvq_rope_axes_bf16.argtypes = [vp, vp, i64, i64, i32, vp, vp, i64, i64, i32, i32, i32, vp, i64, i32, vp, vp, i32,
                                         i32, i32, f32, i32, vp]
        L.kvq_rope_append_int8kv.argtypes = [cp, vp, vp, i64, i64, i32, vp, i64, vp, i64, i32, vp, vp, vp, i32, i32, vp, i64,
                                             i32, vp, vp, i32, i32, i32, f32, vp]
        L.kvq_prefill_window_workspace_bytes.restype = sz
        L.kvq_prefill_window_workspace_bytes.argtypes = [_Int32] * 7
        L.kvq_attn_prefill_window_int8kv.argtypes = [cp, vp, i32, i32, i32, vp, i32, f32, i32, i32, vp, i32, vp, sz, vp]
        L.kvq_prefill_first_workspace_bytes.restype = sz
        L.kvq_prefill_first_workspace_bytes.argtypes = [_Int32, _Int32, _Int32, _Int32]
        L.kvq_attn_prefill_first_bf16.argtypes = [cp, vp, vp, vp, i32, i32, vp, i32, f32, vp, vp, sz, vp]
        L.kvq_prefill_workspace_bytes.restype = sz
        L.kvq_prefill_workspace_bytes.argtypes = [_Int32, _Int32, _Int32, _Int32, _Int32]
        L.kvq_attn_prefill_int8.argtypes = [cp, vp, i32, i32, i32, vp, i32, f32, vp, vp, sz, vp]
        L.kvq_attn_sparse_int8kv.argtypes = [cp, vp, i32, i32, vp, vp, vp, i32, f32, vp, vp, sz, vp]
        L.kvq_sparse_workspace_bytes.restype = sz
        L.kvq_sparse_workspace_bytes.argtypes = [_Int32, _Int32, _Int32]
        L.kvq_debug_prefill_q_codes.argtypes = [vp, i32, i32, i32, vp, vp, vp]
        L.kvq_debug_fault_inject.argtypes = [i32, ctypes.c_int64]
        L.kvq_debug_stream_floor.argtypes = [cp, i32, vp, i32, vp, i32, i32, vp]
        L.kvq_debug_prefill_qk_int32.argtypes = [cp, vp, vp, i32, i32, i32, vp, i32, f32, i32, i32, i32, i32, i32,
                                                 vp, vp, vp, sz, vp]
        _lib = L
    return _lib


# A call's host time is a few microseconds of the kernel's at decode sizes, so the marshalling below
# stays on attribute reads that cost under 0.1 us each (a torch.cuda.Stream object alone is 3 us).
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _stream(stream):
    """cudaStream_t of the stream, or of the current device's current stream."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(_current_device())


def _p(t):
    """Device pointer of a CUDA tensor.  Anything else is refused before any launch: a kernel
    handed a host pointer would fault."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("the library takes CUDA tensors here (got a %s tensor)" % t.device.type)
    return t.data_ptr()


def _hp(t):
    """Pointer for the decode calls' zero-copy arguments (q, k_new, v_new, out): a CUDA tensor,
    or page-locked host memory mapped into the device's address space."""
    if t is None:
        return None
    if not t.is_cuda and not kvq_device_accessible(t):
        raise ValueError("a host tensor must be page-locked memory mapped into the device's address space "
                         "(e.g. tensor.pin_memory())")
    return t.data_ptr()


def _fit(fn, *values):
    """Refuses whole numbers that ctypes would cut to their low 32 bits: a budget of 2^32 + 1 would evict all but one."""
    for v in values:
        if (int(v) + 0x80000000) >> 32:
            raise ValueError("%s: %d does not fit in 32 bits" % (fn, v))


def _check(fn, status):
    if status != 0:
        raise KvqError(fn, status)


def kvq_device_accessible(t):
    """True when the kernels can dereference tensor t's storage (device memory, or page-locked
    host memory mapped into the device's address space)."""
    return bool(lib().kvq_device_accessible(ctypes.c_void_p(t.data_ptr())))


def _host_ok(fn, *tensors):
    """Host tensors passed to a decode call must be mapped page-locked memory (zero-copy): the
    kernels read and write them across the host link.  Anything else is refused before launch."""
    for t in tensors:
        if t is not None and not t.is_cuda and not kvq_device_accessible(t):
            raise ValueError(fn + ": a host tensor must be page-locked memory mapped into the device's "
                             "address space (e.g. tensor.pin_memory())")


def _empty(shape, dtype, device, stream):
    """A tensor for a call on `stream` (None: the current one).  The allocator hands a block that one stream has
    freed to that stream's next tensor at once, so a block that the call's kernels use has to be the call's stream's."""
    if stream is None or stream.cuda_stream == _stream(None):
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):  # another library's, known by its handle
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _result(shape, dtype, device, stream):
    """_empty, for what the caller gets and will read on the current stream (after waiting for the call): the block
    is not given away before that stream's work on it is done."""
    t = _empty(shape, dtype, device, stream)
    if stream is not None and t.is_cuda and stream.cuda_stream != _stream(None):
        t.record_stream(torch.cuda.current_stream())
    return t


def _new_out(shape, q, stream):
    # a host q (zero-copy) gets its result in page-locked host memory too
    if q.device.type == "cpu":
        return torch.empty(shape, dtype=torch.float32, pin_memory=True)
    return _result(shape, torch.float32, q.device, stream)


class KVCache:
    """A paged int8 K/V cache on the GPU in the library's layout:
    k [num_blocks][n_kv_heads][head_dim/16][16][16] int8, v [num_blocks][n_kv_heads][head_dim][16]
    int8, k_scale / v_scale [num_blocks][n_kv_heads][16] fp32."""

    def __init__(self, num_blocks, n_kv_heads, head_dim, device="cuda"):
        self.num_blocks, self.n_kv_heads, self.head_dim = num_blocks, n_kv_heads, head_dim
        self.k = torch.zeros((num_blocks, n_kv_heads, head_dim // 16, BLOCK_SIZE, 16),
                             dtype=torch.int8, device=device)
        self.v = torch.zeros((num_blocks, n_kv_heads, head_dim, BLOCK_SIZE), dtype=torch.int8,
                             device=device)
        self.k_scale = torch.zeros((num_blocks, n_kv_heads, BLOCK_SIZE), dtype=torch.float32,
                                   device=device)
        self.v_scale = torch.zeros_like(self.k_scale)

    @classmethod
    def wrap(cls, k, v, k_scale, v_scale):
        """A cache over tensors that exist already, in the layout above (nothing is copied)."""
        nb, hkv, chunks = k.shape[:3]
        want = (("k", k, torch.int8, (nb, hkv, chunks, BLOCK_SIZE, 16)),
                ("v", v, torch.int8, (nb, hkv, chunks * 16, BLOCK_SIZE)),
                ("k_scale", k_scale, torch.float32, (nb, hkv, BLOCK_SIZE)),
                ("v_scale", v_scale, torch.float32, (nb, hkv, BLOCK_SIZE)))
        for name, t, dtype, shape in want:
            if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError("KVCache.wrap: %s must be a contiguous %s tensor of shape %s" % (name, dtype, shape))
            if t.device != k.device:  # the calls look at k's device alone
                raise ValueError("KVCache.wrap: %s is on %s, k on %s" % (name, t.device, k.device))
        c = cls.__new__(cls)
        c.num_blocks, c.n_kv_heads, c.head_dim = int(nb), int(hkv), int(chunks) * 16
        c.k, c.v, c.k_scale, c.v_scale = k, v, k_scale, v_scale
        return c

    def struct(self):
        # every cache tensor goes through _p: a cache left in host memory is refused before any
        # launch (a kernel handed its pageable pointers would fault)
        return _Cache(_p(self.k), _p(self.v), _p(self.k_scale), _p(self.v_scale), self.num_blocks, BLOCK_SIZE,
                      self.n_kv_heads, self.head_dim)


def kvq_version():
    return lib().kvq_version()


def kvq_device_status(stream=None):
    flags = ctypes.c_uint32(0)
    _check("kvq_device_status", lib().kvq_device_status(ctypes.byref(flags), _stream(stream)))
    return flags.value


def kvq_quant_write(cache, k_new, v_new, seq_idx, pos, block_table, stream=None):
    """k_new, v_new: bf16 [T][Hkv][D]; seq_idx, pos: int32 [T]; block_table: int32 [S][M]."""
    bt = block_table if block_table.dim() == 2 else block_table.view(1, -1)
    c = cache.struct()
    _check("kvq_quant_write", lib().kvq_quant_write(
        ctypes.byref(c), _p(k_new), _p(v_new), int(seq_idx.numel()), _p(seq_idx), _p(pos), _p(bt),
        int(bt.shape[0]), int(bt.shape[1]), _stream(stream)))


def kvq_rope_quant_write(cache, q, k_new, v_new, seq_idx, pos, block_table, cos_sin, rotary_dim,
                         q_codes=None, q_scales=None, q_rot=None, stream=None):
    """Fused producer: RoPE on Q and K (cos_sin fp32 [max_pos][rotary_dim]), the quantisation
    rule on Q, K and V; K/V into the cache.  q: bf16 [T][Hq][D] or None.  Returns
    (q_codes int8 [T][Hq][D], q_scales fp32 [T][Hq], q_rot bf16 [T][Hq][D]), allocated when not
    given (None when q is None)."""
    _fit("kvq_rope_quant_write", rotary_dim)
    bt = block_table if block_table.dim() == 2 else block_table.view(1, -1)
    T = int(seq_idx.numel())
    Hq = int(q.shape[1]) if q is not None else 0
    D = cache.head_dim
    if q is not None:
        dev = q.device
        if q_codes is None:
            q_codes = _result((T, Hq, D), torch.int8, dev, stream)
        if q_scales is None:
            q_scales = _result((T, Hq), torch.float32, dev, stream)
        if q_rot is None:
            q_rot = _result((T, Hq, D), torch.bfloat16, dev, stream)
    c = cache.struct()
    _check("kvq_rope_quant_write", lib().kvq_rope_quant_write(
        ctypes.byref(c), _p(q) if q is not None else None, Hq, _p(k_new), _p(v_new), T, _p(seq_idx), _p(pos),
        _p(bt), int(bt.shape[0]), int(bt.shape[1]), _p(cos_sin), int(cos_sin.shape[0]), int(rotary_dim),
        _p(q_codes) if q_codes is not None else None, _p(q_scales) if q_scales is not None else None,
        _p(q_rot) if q_rot is not None else None, _stream(stream)))
    return q_codes, q_scales, q_rot


def _decode_opts(split_rows, route_threshold, force_route, events=None, launches=None):
    if split_rows or route_threshold or force_route:
        _fit("split_rows, route_threshold, force_route", split_rows, route_threshold, force_route)
    ev0 = ev1 = None
    if events is not None:
        ev0, ev1 = (ctypes.c_void_p(e.cuda_event) for e in events)
    return _DecodeOpts(int(split_rows), int(route_threshold), int(force_route), ev0, ev1,
                       ctypes.pointer(launches) if launches is not None else None)


def kvq_decode_auto_split_rows(batch, n_kv_heads, head_dim, max_ctx, n_sms):
    return int(lib().kvq_decode_auto_split_rows(batch, n_kv_heads, head_dim, max_ctx, n_sms))


def kvq_prefill_split_tiles(n_tokens, n_q_heads, history_len, n_sms):
    return int(lib().kvq_prefill_split_tiles(n_tokens, n_q_heads, history_len, n_sms))


def kvq_decode_workspace_bytes(batch, n_q_heads, max_ctx, head_dim, split_rows=0,
                               route_threshold=0, force_route=0):
    o = _decode_opts(split_rows, route_threshold, force_route)
    return int(lib().kvq_decode_workspace_bytes(batch, n_q_heads, max_ctx, head_dim, ctypes.byref(o)))


def kvq_verify_workspace_bytes(batch, n_rows, n_q_heads, max_ctx, head_dim, split_rows=0,
                               route_threshold=0, force_route=0):
    o = _decode_opts(split_rows, route_threshold, force_route)
    return int(lib().kvq_verify_workspace_bytes(batch, n_rows, n_q_heads, max_ctx, head_dim, ctypes.byref(o)))


def kvq_attn_decode_int8kv(cache, q, block_table, ctx_lens, max_ctx, softmax_scale, out=None,
                           workspace=None, split_rows=0, route_threshold=0, force_route=0,
                           stream=None, stage1_events=None):
    """q: bf16 [B][Hq][D]; block_table int32 [B][M]; ctx_lens int32 [B] (device);
    max_ctx: host bound of ctx_lens.  Returns out fp32 [B][Hq][D].  stage1_events: optional
    pair of torch.cuda.Event recorded around the stage-1 kernel (profiling)."""
    _fit("kvq_attn_decode_int8kv", max_ctx)
    B, Hq, D = q.shape
    if out is None:
        out = _new_out((B, Hq, D), q, stream)
    _host_ok("kvq_attn_decode_int8kv", q, out)
    o = _decode_opts(split_rows, route_threshold, force_route, stage1_events)
    need = int(lib().kvq_decode_workspace_bytes(B, Hq, max(1, int(max_ctx)), D, ctypes.byref(o)))
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, cache.k.device, stream)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    c = cache.struct()
    _check("kvq_attn_decode_int8kv", lib().kvq_attn_decode_int8kv(
        ctypes.byref(c), _hp(q), B, Hq, _p(block_table), int(block_table.shape[1]), _p(ctx_lens),
        int(max_ctx), float(softmax_scale), _hp(out), _p(workspace), wbytes, ctypes.byref(o),
        _stream(stream)))
    return out


def kvq_attn_verify_int8kv(cache, q, block_table, ctx_lens, max_ctx, softmax_scale, out=None,
                           workspace=None, split_rows=0, route_threshold=0, force_route=0,
                           stream=None, stage1_events=None):
    """q: bf16 [B][nq][Hq][D], the nq newest tokens of each sequence; row i of sequence b sees
    keys t < ctx_lens[b] - nq + 1 + i.  Returns out fp32 [B][nq][Hq][D]."""
    _fit("kvq_attn_verify_int8kv", max_ctx)
    B, nq, Hq, D = q.shape
    if out is None:
        out = _new_out((B, nq, Hq, D), q, stream)
    _host_ok("kvq_attn_verify_int8kv", q, out)
    o = _decode_opts(split_rows, route_threshold, force_route, stage1_events)
    need = int(lib().kvq_verify_workspace_bytes(B, nq, Hq, max(1, int(max_ctx)), D, ctypes.byref(o)))
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, cache.k.device, stream)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    c = cache.struct()
    _check("kvq_attn_verify_int8kv", lib().kvq_attn_verify_int8kv(
        ctypes.byref(c), _hp(q), B, nq, Hq, _p(block_table), int(block_table.shape[1]), _p(ctx_lens),
        int(max_ctx), float(softmax_scale), _hp(out), _p(workspace), wbytes, ctypes.byref(o),
        _stream(stream)))
    return out


def kvq_decode_step_int8kv(cache, k_new, v_new, q, block_table, ctx_lens, max_ctx, softmax_scale, out=None,
                           workspace=None, split_rows=0, route_threshold=0, force_route=0,
                           stream=None, stage1_events=None, launches=None):
    """One decode step: write each sequence's nq newest tokens (k_new / v_new bf16
    [B][nq][Hkv][D], positions ctx_lens[b] - nq + j) into the cache, then attend with their
    query rows q bf16 [B][nq][Hq][D].  A 3-D q ([B][Hq][D]) with 3-D k_new / v_new
    ([B][Hkv][D]) is the one-token step.  Returns out fp32 shaped like q."""
    _fit("kvq_decode_step_int8kv", max_ctx)
    squeeze = q.dim() == 3
    if squeeze:
        q, k_new, v_new = q[:, None], k_new[:, None], v_new[:, None]
    B, nq, Hq, D = q.shape
    if out is None:
        out = _new_out((B, nq, Hq, D), q, stream)
        ret = out[:, 0] if squeeze else out
    else:
        ret = out  # the caller's buffer, in the caller's shape ([B][Hq][D] for the one-token step)
    _host_ok("kvq_decode_step_int8kv", q, k_new, v_new, out)
    o = _decode_opts(split_rows, route_threshold, force_route, stage1_events, launches)
    need = int(lib().kvq_verify_workspace_bytes(B, nq, Hq, max(1, int(max_ctx)), D, ctypes.byref(o)))
    if workspace is None and need > 0:
        workspace = _empty(need, torch.uint8, cache.k.device, stream)
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    c = cache.struct()
    _check("kvq_decode_step_int8kv", lib().kvq_decode_step_int8kv(
        ctypes.byref(c), _hp(k_new), _hp(v_new), _hp(q), B, nq, Hq, _p(block_table), int(block_table.shape[1]),
        _p(ctx_lens), int(max_ctx), float(softmax_scale), _hp(out), _p(workspace), wbytes, ctypes.byref(o),
        _stream(stream)))
    return ret


NOALLOC_SCRATCH_BYTES = 16 << 20


def kvq_attn_decode_int8kv_noalloc(cache, q, block_table, ctx_lens, max_ctx, softmax_scale, out,
                                   split_rows=0, route_threshold=0, force_route=0, stream=None):
    """kvq_attn_decode_int8kv without a workspace argument, for callers that cannot allocate:
    the split-K partials live in a fixed scratch array inside the library.  `out` (fp32
    [B][Hq][D]) must be provided by the caller; nothing is allocated here."""
    _fit("kvq_attn_decode_int8kv_noalloc", max_ctx)
    B, Hq, D = q.shape
    _host_ok("kvq_attn_decode_int8kv_noalloc", q, out)
    o = _decode_opts(split_rows, route_threshold, force_route)
    c = cache.struct()
    _check("kvq_attn_decode_int8kv_noalloc", lib().kvq_attn_decode_int8kv_noalloc(
        ctypes.byref(c), _hp(q), B, Hq, _p(block_table), int(block_table.shape[1]), _p(ctx_lens),
        int(max_ctx), float(softmax_scale), _hp(out), ctypes.byref(o), _stream(stream)))
    return out


def kvq_debug_fault_inject(mode, wait_budget_cycles=0):
    """Test entry point of the failure path (see kvq.h): mode 0 none, 1 a decode stage-1 copy left
    un-issued, 2 a prefill piece left un-issued, 3 a sparse chunk left un-issued, 4 a key tile of the chunk
    weights not announced, 5 a tile of the windowed prefill left un-issued; every bounded wait gives up after wait_budget_cycles (<= 0: the default)."""
    _fit("kvq_debug_fault_inject", mode)
    _check("kvq_debug_fault_inject", lib().kvq_debug_fault_inject(int(mode), int(wait_budget_cycles)))


def kvq_prefill_workspace_bytes(n_tokens, n_q_heads, n_kv_heads, history_len, head_dim):
    return int(lib().kvq_prefill_workspace_bytes(n_tokens, n_q_heads, n_kv_heads, history_len, head_dim))


def kvq_prefill_first_workspace_bytes(n_tokens, n_q_heads, n_kv_heads, head_dim):
    return int(lib().kvq_prefill_first_workspace_bytes(n_tokens, n_q_heads, n_kv_heads, head_dim))


def kvq_attn_prefill_first_bf16(cache, q, k_new, v_new, block_table_row, softmax_scale, out=None, workspace=None,
                                stream=None):
    """The first prefill chunk: q bf16 [T][Hq][D], k_new / v_new bf16 [T][Hkv][D] (positions 0..T-1,
    written into the cache as int8); returns the high-precision causal attention, fp32 [T][Hq][D]."""
    T, Hq, D = q.shape
    if out is None:
        out = _result((T, Hq, D), torch.float32, q.device, stream)
    if workspace is None:
        workspace = _empty(kvq_prefill_first_workspace_bytes(T, Hq, cache.n_kv_heads, D), torch.uint8, q.device, stream)
    c = cache.struct()
    _check("kvq_attn_prefill_first_bf16", lib().kvq_attn_prefill_first_bf16(
        ctypes.byref(c), _p(q), _p(k_new), _p(v_new), T, Hq, _p(block_table_row), int(block_table_row.numel()),
        float(softmax_scale), _p(out), _p(workspace), workspace.numel(), _stream(stream)))
    return out


def kvq_attn_prefill_int8(cache, q, history_len, block_table_row, softmax_scale, out=None,
                          workspace=None, stream=None):
    """q: bf16 [T][Hq][D]; block_table_row int32 [n]; returns out fp32 [T][Hq][D]."""
    _fit("kvq_attn_prefill_int8", history_len)
    T, Hq, D = q.shape
    if out is None:
        out = _result((T, Hq, D), torch.float32, q.device, stream)
    need = kvq_prefill_workspace_bytes(T, Hq, cache.n_kv_heads, int(history_len), D)
    if workspace is None:
        workspace = _empty(need, torch.uint8, q.device, stream)
    wbytes = workspace.numel() * workspace.element_size()
    c = cache.struct()
    _check("kvq_attn_prefill_int8", lib().kvq_attn_prefill_int8(
        ctypes.byref(c), _p(q), T, Hq, int(history_len), _p(block_table_row),
        int(block_table_row.numel()), float(softmax_scale), _p(out), _p(workspace), wbytes,
        _stream(stream)))
    return out


def kvq_attn_prefill_int8_qcodes(cache, q_codes, q_scales, history_len, block_table_row, softmax_scale,
                                 out=None, workspace=None, stream=None):
    """q_codes int8 [T][Hq][D], q_scales fp32 [T][Hq] (from kvq_rope_quant_write); returns fp32 [T][Hq][D]."""
    _fit("kvq_attn_prefill_int8_qcodes", history_len)
    T, Hq, D = q_codes.shape
    if out is None:
        out = _result((T, Hq, D), torch.float32, q_codes.device, stream)
    need = kvq_prefill_workspace_bytes(T, Hq, cache.n_kv_heads, int(history_len), D)
    if workspace is None:
        workspace = _empty(need, torch.uint8, q_codes.device, stream)
    wbytes = workspace.numel() * workspace.element_size()
    c = cache.struct()
    _check("kvq_attn_prefill_int8_qcodes", lib().kvq_attn_prefill_int8_qcodes(
        ctypes.byref(c), _p(q_codes), _p(q_scales), T, Hq, int(history_len), _p(block_table_row),
        int(block_table_row.numel()), float(softmax_scale), _p(out), _p(workspace), wbytes, _stream(stream)))
    return out


def kvq_prefill_window_workspace_bytes(n_tokens, n_q_heads, n_kv_heads, history_len, window, n_sink, head_dim):
    return int(lib().kvq_prefill_window_workspace_bytes(n_tokens, n_q_heads, n_kv_heads, history_len, window, n_sink, head_dim))


_OUT_TYPES = {torch.float32: 0, torch.bfloat16: 1}


def kvq_attn_prefill_window_int8kv(cache, q, history_len, block_table_row, softmax_scale, window, n_sink=0, out=None,
                                   out_dtype=torch.bfloat16, workspace=None, stream=None):
    """A chunk of prompt queries with a sliding window: q bf16 [T][Hq][D] at slots history_len .. sees keys t <= its slot p with
    t > p - window or t < n_sink.  block_table_row int32 [n].  Returns out [T][Hq][D], bf16 or fp32 (out's type, or out_dtype)."""
    fn = "kvq_attn_prefill_window_int8kv"
    _fit(fn, history_len, window, n_sink)
    T, Hq, D = q.shape
    dev, n_blocks = _current_device(), block_table_row.numel()
    q_p = _need(fn, "q", q, torch.bfloat16, (T, Hq, cache.head_dim), dev)
    table_p = _need(fn, "block_table_row", block_table_row, torch.int32, (n_blocks,), dev)
    kind = out_dtype if out is None else out.dtype
    if kind not in _OUT_TYPES:
        raise ValueError("%s: the output is bf16 or fp32 (got %s)" % (fn, kind))
    if out is None:
        out = _result((T, Hq, D), kind, q.device, stream)
    out_p = _need(fn, "out", out, kind, (T, Hq, D), dev)
    n = T * Hq * D
    if out_p < q_p + 2 * n and q_p < out_p + (4 if kind is torch.float32 else 2) * n:
        raise ValueError("%s: out overlaps q" % fn)
    need = 0
    if workspace is None:
        need = kvq_prefill_window_workspace_bytes(T, Hq, cache.n_kv_heads, int(history_len), int(window), int(n_sink), D)
    workspace, wbytes = _ws(workspace, need, q.device, stream)
    if workspace.get_device() != dev:
        _elsewhere(fn, "the workspace", workspace)
    c = _cache_struct(fn, cache, dev)
    _check(fn, lib().kvq_attn_prefill_window_int8kv(
        ctypes.byref(c), q_p, T, Hq, int(history_len), table_p, n_blocks, float(softmax_scale), int(window), int(n_sink), out_p,
        _OUT_TYPES[kind], _p(workspace), wbytes, _stream(stream)))
    return out


def kvq_sparse_workspace_bytes(n_blocks_row, n_kv_heads, head_dim):
    return int(lib().kvq_sparse_workspace_bytes(n_blocks_row, n_kv_heads, head_dim))


def kvq_attn_sparse_int8kv(cache, q, cell_offsets, cells, block_table_row, softmax_scale,
                           out=None, workspace=None, stream=None):
    """q: bf16 [N][Hq][D]; cell_offsets int32 [N+1]; cells int32; returns fp32 [N][Hq][D]."""
    N, Hq, D = q.shape
    if out is None:
        out = _result((N, Hq, D), torch.float32, q.device, stream)
    nb = int(block_table_row.numel())
    if workspace is None:
        workspace = _empty(kvq_sparse_workspace_bytes(nb, cache.n_kv_heads, D), torch.uint8, q.device, stream)
    c = cache.struct()
    _check("kvq_attn_sparse_int8kv", lib().kvq_attn_sparse_int8kv(
        ctypes.byref(c), _p(q), N, Hq, _p(cell_offsets), _p(cells), _p(block_table_row),
        nb, float(softmax_scale), _p(out), _p(workspace), workspace.numel(), _stream(stream)))
    return out


def _need(fn, name, t, dtype, shape, dev):
    """Pointer of t, a contiguous tensor of this type and shape on the current CUDA device, number dev."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s: %s must be a contiguous %s tensor of shape %s (got %s %s)"
                         % (fn, name, dtype, tuple(shape), t.dtype, tuple(t.shape)))
    if t.get_device() != dev:
        _elsewhere(fn, name, t)
    return t.data_ptr()


def _elsewhere(fn, name, t):
    raise ValueError("%s: %s must be on the current CUDA device (it is on %s)" % (fn, name, t.device))


def _cache_struct(fn, cache, dev):
    """The cache's C struct; its tensors are on the current device."""
    if cache.k.get_device() != dev:
        _elsewhere(fn, "the cache", cache.k)
    return cache.struct()


def _ws(workspace, need, device, stream):
    """(workspace tensor, its bytes): the caller's, or one of `need` bytes on the device."""
    if workspace is None:
        workspace = _empty(max(need, 16), torch.uint8, device, stream)
    return workspace, workspace.numel() * workspace.element_size()


def _row_stride(fn, name, t, dtype, B, H, dev):
    """(elements from one (sequence, KV head) row of a [B][H][slots] tensor to the next, slots, pointer): rows
    contiguous and evenly spaced (a view of wider rows will do), on the current device."""
    shape, st = t.shape, t.stride()
    if t.dtype is not dtype or len(shape) != 3 or shape[0] != B or shape[1] != H or (st[2] != 1 and shape[2] > 1):
        raise ValueError("%s: %s must be a %s tensor [%d][%d][slots] with contiguous rows" % (fn, name, dtype, B, H))
    slots = shape[2]
    stride = st[1] if H > 1 else st[0] if B > 1 else slots
    if stride < slots or (B > 1 and st[0] != H * stride):
        raise ValueError("%s: the rows of %s must be evenly spaced" % (fn, name))
    if t.get_device() != dev:
        _elsewhere(fn, name, t)
    return stride, slots, t.data_ptr()


def kvq_step_accum_workspace_bytes(batch, n_new, n_q_heads, max_ctx, head_dim, split_rows=0):
    o = _decode_opts(split_rows, 0, 0)
    return int(lib().kvq_step_accum_workspace_bytes(batch, n_new, n_q_heads, max_ctx, head_dim, ctypes.byref(o)))


def kvq_decode_step_accum_int8kv(cache, k_new, v_new, q, block_table, ctx_lens, max_ctx, softmax_scale, acc,
                                 slot_pos=None, pos=None, out=None, workspace=None, split_rows=0, stream=None,
                                 stage1_events=None, launches=None):
    """kvq_decode_step_int8kv (k_new = v_new = None: kvq_attn_verify_int8kv) that also adds to
    acc (fp32 [B][Hkv][>= max_ctx]) the attention weight each key was given, summed over the rows and
    over the query heads of its KV head; the new tokens' entries start from zero.  slot_pos (int32,
    shaped like acc) receives the new tokens' positions pos[b] + j (pos: int32 [B]).  Returns out
    fp32 shaped like q."""
    _fit("kvq_decode_step_accum_int8kv", max_ctx)
    fn = "kvq_decode_step_accum_int8kv"
    shape, H, dev = q.shape, cache.n_kv_heads, _current_device()
    if len(shape) == 3:  # one token
        (B, Hq, D), nq = shape, 1
        rows = B, H, D
    else:
        B, nq, Hq, D = shape
        rows = B, nq, H, D
    if out is None:
        out = _new_out(shape, q, stream)
    q_p = _step_rows(fn, "q", q, torch.bfloat16, None, dev)
    out_p = _step_rows(fn, "out", out, torch.float32, shape, dev)
    k_p = v_p = None
    if k_new is not None:
        k_p = _step_rows(fn, "k_new", k_new, torch.bfloat16, rows, dev)
    if v_new is not None:
        v_p = _step_rows(fn, "v_new", v_new, torch.bfloat16, rows, dev)
    if D != cache.head_dim:
        raise ValueError("%s: q has head_dim %d, the cache %d" % (fn, D, cache.head_dim))
    ctx_p = _need(fn, "ctx_lens", ctx_lens, torch.int32, (B,), dev)
    n_blocks = block_table.shape[-1]
    table_p = _need(fn, "block_table", block_table, torch.int32, (B, n_blocks), dev)
    stride, slots, acc_p = _row_stride(fn, "acc", acc, torch.float32, B, H, dev)
    slot_pos_p = pos_p = None
    if slots < max_ctx:
        raise ValueError("%s: acc has %d slots, max_ctx is %d" % (fn, slots, max_ctx))
    if slot_pos is not None:
        pstride, slots, slot_pos_p = _row_stride(fn, "slot_pos", slot_pos, torch.int32, B, H, dev)
        if pstride != stride or slots < max_ctx:
            raise ValueError("%s: slot_pos must be shaped and laid out like acc" % fn)
        if pos is None:
            raise ValueError("%s: slot_pos needs pos" % fn)
        pos_p = _need(fn, "pos", pos, torch.int32, (B,), dev)
    o = _decode_opts(split_rows, 0, 0, stage1_events, launches)
    need = 0
    if workspace is None:
        need = int(lib().kvq_step_accum_workspace_bytes(B, nq, Hq, int(max_ctx), D, ctypes.byref(o)))
    workspace, wbytes = _ws(workspace, need, cache.k.device, stream)
    c = _cache_struct(fn, cache, dev)
    _check(fn, lib().kvq_decode_step_accum_int8kv(
        ctypes.byref(c), k_p, v_p, q_p, B, nq, Hq, table_p, n_blocks, ctx_p, int(max_ctx), float(softmax_scale), out_p, acc_p,
        stride, slot_pos_p, pos_p, _p(workspace), wbytes, ctypes.byref(o), _stream(stream)))
    return out


def kvq_step_window_workspace_bytes(batch, n_new, n_q_heads, n_kv_heads, max_ctx, window, n_sink, head_dim, split_rows=0,
                                    force_route=0):
    o = _decode_opts(split_rows, 0, force_route)
    return int(lib().kvq_step_window_workspace_bytes(batch, n_new, n_q_heads, n_kv_heads, max_ctx, window, n_sink, head_dim,
                                                     ctypes.byref(o)))


def kvq_decode_step_window_int8kv(cache, k_new, v_new, q, block_table, ctx_lens, max_ctx, softmax_scale, window, n_sink=0,
                                  out=None, workspace=None, split_rows=0, force_route=0, stream=None, stage1_events=None,
                                  launches=None):
    """kvq_decode_step_int8kv (k_new = v_new = None: kvq_attn_verify_int8kv) with a sliding window: the row at position p
    sees keys t <= p with t > p - window or t < n_sink.  Returns out fp32 shaped like q."""
    fn = "kvq_decode_step_window_int8kv"
    _fit(fn, max_ctx, window, n_sink)
    shape, H, dev = q.shape, cache.n_kv_heads, _current_device()
    if len(shape) == 3:  # one token
        (B, Hq, D), nq = shape, 1
        rows = B, H, D
    else:
        B, nq, Hq, D = shape
        rows = B, nq, H, D
    if out is None:
        out = _new_out(shape, q, stream)
    q_p = _step_rows(fn, "q", q, torch.bfloat16, None, dev)
    out_p = _step_rows(fn, "out", out, torch.float32, shape, dev)
    k_p = v_p = None
    if k_new is not None or v_new is not None:
        if k_new is None or v_new is None:
            raise ValueError("%s: k_new and v_new go together" % fn)
        k_p = _step_rows(fn, "k_new", k_new, torch.bfloat16, rows, dev)
        v_p = _step_rows(fn, "v_new", v_new, torch.bfloat16, rows, dev)
    if D != cache.head_dim:
        raise ValueError("%s: q has head_dim %d, the cache %d" % (fn, D, cache.head_dim))
    ctx_p = _need(fn, "ctx_lens", ctx_lens, torch.int32, (B,), dev)
    n_blocks = block_table.shape[-1]
    table_p = _need(fn, "block_table", block_table, torch.int32, (B, n_blocks), dev)
    plain = not (split_rows or force_route or stage1_events or launches is not None)
    o = None if plain else ctypes.byref(_decode_opts(split_rows, 0, force_route, stage1_events, launches))
    ws_p, wbytes = None, 0
    if workspace is None:
        need = int(lib().kvq_step_window_workspace_bytes(B, nq, Hq, H, int(max_ctx), int(window), int(n_sink), D, o))
        if need:
            workspace = _empty(need, torch.uint8, cache.k.device, stream)
    if workspace is not None:
        if workspace.get_device() != dev:
            _elsewhere(fn, "the workspace", workspace)
        ws_p, wbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    c = _cache_struct(fn, cache, dev)
    _check(fn, lib().kvq_decode_step_window_int8kv(
        ctypes.byref(c), k_p, v_p, q_p, B, nq, Hq, table_p, n_blocks, ctx_p, int(max_ctx), float(softmax_scale), int(window),
        int(n_sink), out_p, ws_p, wbytes, o, _stream(stream)))
    return out


def _step_rows(fn, name, t, dtype, shape, dev):
    """Pointer of contiguous rows in the order of `shape` (its dims may be merged; None: any) on the current device, or in
    mapped page-locked host memory (zero-copy)."""
    if t.dtype is not dtype or not t.is_contiguous() or (shape is not None and t.shape != shape and not _merged(t.shape, shape)):
        raise ValueError("%s: %s must be a contiguous %s tensor of shape %s (got %s %s)" %
                         (fn, name, dtype, list(shape or t.shape), t.dtype, list(t.shape)))
    if t.get_device() != dev:
        if t.is_cuda:
            _elsewhere(fn, name, t)
        return _hp(t)
    return t.data_ptr()


def kvq_chunk_weights_workspace_bytes(n_tokens, n_q_heads, n_kv_heads, history_len, head_dim):
    return int(lib().kvq_chunk_weights_workspace_bytes(n_tokens, n_q_heads, n_kv_heads, history_len, head_dim))


def kvq_attn_chunk_weights_int8kv(cache, q, history_len, block_table_row, softmax_scale, acc, workspace=None,
                                  stream=None):
    """Adds to acc (fp32 [Hkv][>= history_len + T]) the attention weights that the causal queries q (bf16
    [T][Hq][D], at slots history_len ..) give to every key of the sequence, summed over the queries and
    over the query heads of each KV head.  block_table_row int32 [n].  Returns acc."""
    _fit("kvq_attn_chunk_weights_int8kv", history_len)
    fn = "kvq_attn_chunk_weights_int8kv"
    T, Hq, D = q.shape
    dev, n_blocks = _current_device(), block_table_row.numel()
    _need(fn, "q", q, torch.bfloat16, (T, Hq, cache.head_dim), dev)
    _need(fn, "block_table_row", block_table_row, torch.int32, (n_blocks,), dev)
    if acc.dim() != 2 or acc.shape[1] < history_len + T:
        raise ValueError("%s: acc must be [%d][>= %d]" % (fn, cache.n_kv_heads, history_len + T))
    stride, _, _ = _row_stride(fn, "acc", acc[None], torch.float32, 1, cache.n_kv_heads, dev)
    need = 0
    if workspace is None:
        need = kvq_chunk_weights_workspace_bytes(T, Hq, cache.n_kv_heads, int(history_len), D)
    workspace, wbytes = _ws(workspace, need, q.device, stream)
    c = _cache_struct(fn, cache, dev)
    _check(fn, lib().kvq_attn_chunk_weights_int8kv(
        ctypes.byref(c), _p(q), T, Hq, int(history_len), _p(block_table_row), n_blocks,
        float(softmax_scale), _p(acc), stride, _p(workspace), wbytes, _stream(stream)))
    return acc


def kvq_evict_workspace_bytes(batch, n_kv_heads, max_ctx, keep):
    return int(lib().kvq_evict_workspace_bytes(batch, n_kv_heads, max_ctx, keep))


def kvq_cache_evict(cache, block_table, ctx_lens, max_ctx, keep, acc, slot_pos, n_sink=0, n_recent=0, acc_out=None,
                    slot_pos_out=None, new_lens=None, workspace=None, stream=None):
    """Brings every (sequence, KV head) down to `keep` tokens: those at positions below n_sink, the
    n_recent newest, then those of the largest acc (ties to the lowest slot); kept tokens past the
    budget move into the slots given up below it.  acc fp32 / slot_pos int32 [B][Hkv][>= max_ctx];
    acc_out / slot_pos_out: None for in place, or tensors [B][Hkv][>= min(keep, max_ctx)].  Returns
    (acc_out, slot_pos_out, new_lens int32 [B])."""
    _fit("kvq_cache_evict", max_ctx, keep, n_sink, n_recent)
    fn = "kvq_cache_evict"
    B, H = int(ctx_lens.shape[0]), cache.n_kv_heads
    if (acc_out is None) != (slot_pos_out is None):
        raise ValueError("%s: acc_out and slot_pos_out go together" % fn)
    in_place = acc_out is None
    if in_place:
        acc_out, slot_pos_out = acc, slot_pos
    if new_lens is None:
        new_lens = _result(ctx_lens.shape, torch.int32, ctx_lens.device, stream)
    dev, n_blocks = _current_device(), block_table.shape[-1]
    ctx_p = _need(fn, "ctx_lens", ctx_lens, torch.int32, (B,), dev)
    new_p = _need(fn, "new_lens", new_lens, torch.int32, (B,), dev)
    table_p = _need(fn, "block_table", block_table, torch.int32, (B, n_blocks), dev)
    stride, slots, acc_p = _row_stride(fn, "acc", acc, torch.float32, B, H, dev)
    pstride, pslots, pos_p = _row_stride(fn, "slot_pos", slot_pos, torch.int32, B, H, dev)
    ostride, oslots, acc_out_p, qstride, qslots, pos_out_p = stride, slots, acc_p, pstride, pslots, pos_p
    if not in_place:
        ostride, oslots, acc_out_p = _row_stride(fn, "acc_out", acc_out, torch.float32, B, H, dev)
        qstride, qslots, pos_out_p = _row_stride(fn, "slot_pos_out", slot_pos_out, torch.int32, B, H, dev)
    if pstride != stride or qstride != ostride:
        raise ValueError("%s: slot_pos must be laid out like acc, slot_pos_out like acc_out" % fn)
    if min(slots, pslots) < max_ctx or min(oslots, qslots) < min(keep, max_ctx):
        raise ValueError("%s: acc and slot_pos need max_ctx slots, the outputs min(keep, max_ctx)" % fn)
    need = kvq_evict_workspace_bytes(B, H, int(max_ctx), int(keep)) if workspace is None else 0
    workspace, wbytes = _ws(workspace, need, cache.k.device, stream)
    c = _cache_struct(fn, cache, dev)
    _check(fn, lib().kvq_cache_evict(
        ctypes.byref(c), B, table_p, n_blocks, ctx_p, int(max_ctx), int(keep), int(n_sink), int(n_recent), acc_p, pos_p,
        stride, acc_out_p, pos_out_p, ostride, new_p, _p(workspace), wbytes, _stream(stream)))
    return acc_out, slot_pos_out, new_lens


def _rope_scaling(fn, n, scaling, factor, original_len, low, high, divisors):
    """The C struct of a scaling of n frequencies."""
    if scaling not in _ROPE_SCALINGS:
        raise ValueError("%s: unknown scaling %r" % (fn, scaling))
    div = None
    if divisors is not None:
        if len(divisors) != n:
            raise ValueError("%s: %d divisors for %d frequencies" % (fn, len(divisors), n))
        div = (ctypes.c_double * n)(*[float(x) for x in divisors])
    z = _RopeScaling(_ROPE_SCALINGS[scaling], float(factor), float(original_len), float(low), float(high),
                     ctypes.cast(div, ctypes.POINTER(ctypes.c_double)) if div is not None else None)
    z.keep = div  # the struct holds its address alone
    return z


def kvq_rope_phases(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0,
                    divisors=None, device="cuda"):
    """The plan of kvq_rope_bf16: (phases, attn_factor), phases int64 [rotary_dim / 2] (the bits of the
    64-bit fractions of a turn per position).  scaling: "none", "linear", "ntk", "yarn", "bands" or
    "divisors"."""
    _fit("kvq_rope_phases", rotary_dim)
    n = max(int(rotary_dim), 0) // 2
    z = _rope_scaling("kvq_rope_phases", n, scaling, factor, original_len, low, high, divisors)
    host = torch.empty(n, dtype=torch.int64)
    af = ctypes.c_float(1.0)
    _check("kvq_rope_phases", lib().kvq_rope_phases(
        int(rotary_dim), float(base), ctypes.byref(z), ctypes.cast(host.data_ptr(), ctypes.POINTER(ctypes.c_uint64)),
        ctypes.byref(af)))
    return host.to(device), af.value


def kvq_rope_bf16(q, k, pos, phases, layout=ROPE_HALF, rotary_offset=0, attn_factor=1.0, q_out=None, k_out=None,
                  stream=None):
    """Rotates q bf16 [T][Hq][D] and k bf16 [T][Hkv][D] (either may be None) by pos int32 [T]; rows may be
    views of a packed projection (token stride free, heads and dims contiguous).  q_out / k_out:
    None for new tensors, or tensors like the inputs, the inputs themselves among them.  Returns
    (q_out, k_out)."""
    _fit("kvq_rope_bf16", rotary_offset, layout)
    fn = "kvq_rope_bf16"
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("%s: q and k are both None" % fn)
    T, _, D = ref.shape
    dev = _current_device()
    q_p = qo_p = k_p = ko_p = None
    hq = qs = qos = hk = ks = kos = 0
    if q is not None:
        if q_out is None:
            q_out = _result(q.shape, torch.bfloat16, q.device, stream)
        hq, qs, q_p = _heads(fn, "q", q, T, D, dev)
        ho, qos, qo_p = _heads(fn, "q_out", q_out, T, D, dev)
        if ho != hq:
            raise ValueError("%s: q_out has %d heads, q %d" % (fn, ho, hq))
    if k is not None:
        if k_out is None:
            k_out = _result(k.shape, torch.bfloat16, k.device, stream)
        hk, ks, k_p = _heads(fn, "k", k, T, D, dev)
        ho, kos, ko_p = _heads(fn, "k_out", k_out, T, D, dev)
        if ho != hk:
            raise ValueError("%s: k_out has %d heads, k %d" % (fn, ho, hk))
    n = phases.numel()
    pos_p = _need(fn, "pos", pos, torch.int32, (T,), dev)
    phases_p = _need(fn, "phases", phases, torch.int64, (n,), dev)
    _check(fn, lib().kvq_rope_bf16(q_p, qo_p, qs, qos, hq, k_p, ko_p, ks, kos, hk, D, T, pos_p, phases_p, 2 * n,
                                   int(rotary_offset), int(layout), float(attn_factor), _stream(stream)))
    return (q_out if q is not None else None), (k_out if k is not None else None)


class RopeAxes:
    """A plan of kvq_rope_axes_bf16 and kvq_rope_append_int8kv: phases (int64 [rotary_dim / 2] on the device, the bits of
    the 64-bit fractions of a turn per position), the axis of each frequency, and the factor on cos and sin."""

    __slots__ = ("phases", "axis_of", "attn_factor", "n_axes", "rotary_dim")

    def __init__(self, phases, axis_of, attn_factor=1.0):
        self.phases, self.axis_of, self.attn_factor = phases, bytes(list(axis_of)), float(attn_factor)
        self.n_axes, self.rotary_dim = max(self.axis_of, default=0) + 1, 2 * len(self.axis_of)
        if phases.dtype is not torch.int64 or tuple(phases.shape) != (len(self.axis_of),) or not phases.is_contiguous():
            raise ValueError("RopeAxes: phases must be a contiguous int64 tensor [%d]" % len(self.axis_of))
        if self.n_axes > 4:
            raise ValueError("RopeAxes: %d axes, at most 4" % self.n_axes)


def kvq_rope_axes_phases(sections, base=10000.0, order="chunked", ladder="shared", scaling="none", factor=1.0,
                         original_len=0.0, low=1.0, high=32.0, divisors=None, device="cuda"):
    """A RopeAxes plan: sections[a] frequencies for axis a, "chunked" (one axis after the other) or in "turns"; one "shared"
    ladder of frequencies, or a ladder "per_axis".  Scalings as in kvq_rope_phases."""
    fn = "kvq_rope_axes_phases"
    if order not in _ROPE_ORDERS or ladder not in _ROPE_LADDERS:
        raise ValueError("%s: unknown order or ladder (%r, %r)" % (fn, order, ladder))
    _fit(fn, *sections)
    sections = [int(n) for n in sections]
    n = max(sum(sections), 0)
    z = _rope_scaling(fn, n, scaling, factor, original_len, low, high, divisors)
    host, axis_of, af = torch.empty(n, dtype=torch.int64), ctypes.create_string_buffer(max(n, 1)), ctypes.c_float(1.0)
    _check(fn, lib().kvq_rope_axes_phases(
        len(sections), (ctypes.c_int32 * max(len(sections), 1))(*sections), _ROPE_ORDERS[order], _ROPE_LADDERS[ladder],
        float(base), ctypes.byref(z), ctypes.cast(host.data_ptr(), ctypes.POINTER(ctypes.c_uint64)), axis_of, ctypes.byref(af)))
    return RopeAxes(host.to(device), axis_of.raw[:n], af.value)


def _axes(fn, pos, plan, T, dev):
    """(pointer, stride, axes) of pos int32 [axes][T] (or [T] with one axis); the plan's phases are on the device."""
    n = plan.n_axes
    shape = pos.shape
    if len(shape) == 1:
        shape = (1,) + tuple(shape)
    if pos.dtype is not torch.int32 or len(shape) != 2 or shape[0] < n or shape[1] != T or (T > 1 and pos.stride(-1) != 1):
        raise ValueError("%s: pos must be int32 [%d][%d] with contiguous rows (got %s %s)" % (fn, n, T, pos.dtype, tuple(pos.shape)))
    stride = pos.stride(0) if n > 1 else T
    if pos.get_device() != dev:
        _elsewhere(fn, "pos", pos)
    if plan.phases.get_device() != dev:
        _elsewhere(fn, "the plan", plan.phases)
    if stride < T:
        raise ValueError("%s: the rows of pos overlap" % fn)
    return pos.data_ptr(), stride, n


def kvq_rope_axes_bf16(q, k, pos, plan, layout=ROPE_HALF, rotary_offset=0, inverse=False, q_out=None, k_out=None, stream=None):
    """kvq_rope_bf16 with positions on several axes: pos int32 [axes][T] ([T] with one axis), plan a RopeAxes.  inverse turns
    the other way: the gradient of the rotation.  Returns (q_out, k_out)."""
    fn = "kvq_rope_axes_bf16"
    _fit(fn, rotary_offset, layout)
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("%s: q and k are both None" % fn)
    T, _, D = ref.shape
    dev = _current_device()
    q_p = qo_p = k_p = ko_p = None
    hq = qs = qos = hk = ks = kos = 0
    if q is not None:
        if q_out is None:
            q_out = _result(q.shape, torch.bfloat16, q.device, stream)
        hq, qs, q_p = _heads(fn, "q", q, T, D, dev)
        ho, qos, qo_p = _heads(fn, "q_out", q_out, T, D, dev)
        if ho != hq:
            raise ValueError("%s: q_out has %d heads, q %d" % (fn, ho, hq))
    if k is not None:
        if k_out is None:
            k_out = _result(k.shape, torch.bfloat16, k.device, stream)
        hk, ks, k_p = _heads(fn, "k", k, T, D, dev)
        ho, kos, ko_p = _heads(fn, "k_out", k_out, T, D, dev)
        if ho != hk:
            raise ValueError("%s: k_out has %d heads, k %d" % (fn, ho, hk))
    pos_p, pos_stride, n_axes = _axes(fn, pos, plan, T, dev)
    _check(fn, lib().kvq_rope_axes_bf16(q_p, qo_p, qs, qos, hq, k_p, ko_p, ks, kos, hk, D, T, pos_p, pos_stride, n_axes,
                                        plan.phases.data_ptr(), plan.axis_of, plan.rotary_dim, int(rotary_offset), int(layout),
                                        plan.attn_factor, 1 if inverse else 0, _stream(stream)))
    return (q_out if q is not None else None), (k_out if k is not None else None)


def kvq_rope_append_int8kv(cache, q, k_new, v_new, pos, plan, seq_idx, slot, block_table, layout=ROPE_HALF, rotary_offset=0,
                           q_out=None, stream=None):
    """New tokens into the cache: q bf16 [T][Hq][D] (or None) rotated by pos (int32 [axes][T]) and plan into q_out, k_new
    rotated and k_new, v_new bf16 [T][Hkv][D] quantised into slot[i] of sequence seq_idx[i] (int32 [T]; slot -1: a padding
    token, nothing of it is written).  Rows may be views of a packed projection.  block_table int32 [S][M].  Returns q_out."""
    fn = "kvq_rope_append_int8kv"
    _fit(fn, rotary_offset, layout)
    T, H, D = k_new.shape
    dev = _current_device()
    if H != cache.n_kv_heads or D != cache.head_dim:
        raise ValueError("%s: k_new has %d heads of %d, the cache %d of %d" % (fn, H, D, cache.n_kv_heads, cache.head_dim))
    _, ks, k_p = _heads(fn, "k_new", k_new, T, D, dev)
    hv, vs, v_p = _heads(fn, "v_new", v_new, T, D, dev)
    if hv != H:
        raise ValueError("%s: v_new has %d heads, the cache %d" % (fn, hv, H))
    q_p = qo_p = None
    hq = qs = qos = 0
    if q is not None:
        if q_out is None:
            q_out = _result(q.shape, torch.bfloat16, q.device, stream)
        hq, qs, q_p = _heads(fn, "q", q, T, D, dev)
        ho, qos, qo_p = _heads(fn, "q_out", q_out, T, D, dev)
        if ho != hq:
            raise ValueError("%s: q_out has %d heads, q %d" % (fn, ho, hq))
    pos_p, pos_stride, n_axes = _axes(fn, pos, plan, T, dev)
    seq_p = _need(fn, "seq_idx", seq_idx, torch.int32, (T,), dev)
    slot_p = _need(fn, "slot", slot, torch.int32, (T,), dev)
    n_seqs, n_blocks = block_table.shape
    table_p = _need(fn, "block_table", block_table, torch.int32, (n_seqs, n_blocks), dev)
    c = _cache_struct(fn, cache, dev)
    _check(fn, lib().kvq_rope_append_int8kv(
        ctypes.byref(c), q_p, qo_p, qs, qos, hq, k_p, ks, v_p, vs, T, seq_p, slot_p, table_p, n_seqs, n_blocks, pos_p, pos_stride,
        n_axes, plan.phases.data_ptr(), plan.axis_of, plan.rotary_dim, int(rotary_offset), int(layout), plan.attn_factor,
        _stream(stream)))
    return q_out if q is not None else None


def _merged(got, shape):
    """Whether a shape is `shape` with neighbouring dims merged, or dims of 1 put in: the same elements in the same order."""
    places, n = {1}, 1
    for x in reversed(shape):
        n *= x
        places.add(n)
    m = 1
    for x in reversed(got):
        m *= x
        if m not in places:
            return False
    return m == n


def _heads(fn, name, t, T, D, dev):
    """(heads, token stride, pointer) of bf16 rows [T][heads][D] on the current device: heads and dims contiguous,
    tokens any stride apart."""
    shape = t.shape
    if t.dtype is not torch.bfloat16 or len(shape) != 3 or shape[0] != T or shape[2] != D:
        _not_heads(fn, name, T, D)
    H, (st, sh, sd) = shape[1], t.stride()
    if (sh != D and H > 1) or (sd != 1 and D > 1):
        _not_heads(fn, name, T, D)
    if t.get_device() != dev:
        _elsewhere(fn, name, t)
    return H, st, t.data_ptr()


def _not_heads(fn, name, T, D):
    raise ValueError("%s: %s must be bf16 [%d][heads][%d] with contiguous heads" % (fn, name, T, D))


def kvq_debug_prefill_q_codes(q, stream=None):
    """Q quantisation step alone: returns (int8 codes [T][Hq][D], fp32 scales [T][Hq])."""
    T, Hq, D = q.shape
    codes = _result((T, Hq, D), torch.int8, q.device, stream)
    scales = _result((T, Hq), torch.float32, q.device, stream)
    _check("kvq_debug_prefill_q_codes", lib().kvq_debug_prefill_q_codes(
        _p(q), T, Hq, D, _p(codes), _p(scales), _stream(stream)))
    return codes, scales


def kvq_debug_prefill_qk_int32(cache, q_codes, q_scales, history_len, block_table_row, softmax_scale, q_head, q0,
                               k0, nk, split_tiles=-1, out=None, workspace=None, stream=None):
    """The production prefill (kvq_attn_prefill_int8_qcodes) that also exports the integer QK scores
    of one unit: returns (S int32 [128][nk] for query rows q0..q0+127 of q_head and keys
    k0..k0+nk-1, out fp32 [T][Hq][D]).  split_tiles: -1 the call's own key-range split, 0 none,
    r > 0 a forced tail of r key tiles."""
    _fit("kvq_debug_prefill_qk_int32", history_len, split_tiles, q_head, q0, k0, nk)
    T, Hq, D = q_codes.shape
    s = _result((128, nk), torch.int32, q_codes.device, stream)
    if out is None:
        out = _result((T, Hq, D), torch.float32, q_codes.device, stream)
    need = kvq_prefill_workspace_bytes(T, Hq, cache.n_kv_heads, int(history_len), D)
    if workspace is None:
        workspace = _empty(need, torch.uint8, q_codes.device, stream)
    c = cache.struct()
    _check("kvq_debug_prefill_qk_int32", lib().kvq_debug_prefill_qk_int32(
        ctypes.byref(c), _p(q_codes), _p(q_scales), T, Hq, int(history_len), _p(block_table_row),
        int(block_table_row.numel()), float(softmax_scale), int(split_tiles), int(q_head), int(q0), int(k0), int(nk),
        _p(s), _p(out), _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return s, out


def kvq_debug_stream_floor(cache, block_table, ctx_lens, max_ctx, split_rows=0, stream=None):
    """The K/V stream of decode stage 1 alone (same grid, rings and copies, no arithmetic)."""
    _fit("kvq_debug_stream_floor", max_ctx, split_rows)
    c = cache.struct()
    _check("kvq_debug_stream_floor", lib().kvq_debug_stream_floor(
        ctypes.byref(c), int(block_table.shape[0]), _p(block_table), int(block_table.shape[1]), _p(ctx_lens),
        int(max_ctx), int(split_rows), _stream(stream)))
