"""ctypes binding of libkvq.so (argument marshalling only).

Every function here forwards to the C entry point of the same name declared in
include/kvq.h; torch tensors are passed as raw device pointers and the current
torch CUDA stream is used unless one is given.  Nothing is computed here, and
there is no fallback: if the shared library is missing the import fails.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_char_p, c_double, c_float, c_int32, c_int64, c_size_t, c_uint32, c_void_p

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvq.so")

KVQ_OK = 0
KVQ_ERR_INVALID_ARG = 1
KVQ_ERR_UNSUPPORTED = 2
KVQ_ERR_ALIGNMENT = 3
KVQ_ERR_WORKSPACE = 4
KVQ_ERR_CUDA = 5

KVQ_DEVERR_BLOCK_ID = 1
KVQ_DEVERR_SEQ_LEN = 2
KVQ_DEVERR_TIMEOUT = 4
KVQ_DEVERR_RANGE = 8
KVQ_DEVERR_POSITION = 16
KVQ_DEVERR_NO_BLOCKS = 32

APPEND_QUANT = 0
APPEND_RING = 1
APPEND_STEP = 2
PREFILL_TILES = -1  # kvq_prefill stream_ctas: the query-tile path
PREFILL_UNITS = -2  # kvq_prefill_sinks stream_ctas: units of 256 query vectors
ROPE_PLAIN = 0
ROPE_LINEAR = 1
ROPE_NTK = 2
ROPE_BANDS = 3
DECODE_GEOMETRY_READY = 1  # kvq_decode_ex flag: lengths and block table final before the previous kernel ends


class KvqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class CacheDesc(ctypes.Structure):
    """Mirror of kvq_cache_desc."""
    _fields_ = [
        ("num_kv_heads", c_int32), ("head_dim", c_int32), ("block_size", c_int32), ("num_blocks", c_int32),
        ("k_bits", c_int32), ("v_bits", c_int32),
        ("k_codes", c_void_p), ("v_codes", c_void_p), ("meta", c_void_p), ("asym", c_int32),
        ("k_channel_factor", c_void_p),
        ("window", c_int32), ("window_batch", c_int32),
        ("k_window", c_void_p), ("v_window", c_void_p),
        ("q_bits", c_int32), ("k_per_channel", c_int32),
    ]


class RopeFreqs(ctypes.Structure):
    """Mirror of kvq_rope_freqs."""
    _fields_ = [("base", c_double), ("scaling", c_int32), ("factor", c_double), ("original_len", c_double),
                ("low_turns", c_double), ("high_turns", c_double), ("amplitude", c_double)]


class RopeDesc(ctypes.Structure):
    """Mirror of kvq_rope_desc."""
    _fields_ = [("rotary_dim", c_int32), ("interleaved", c_int32), ("max_pos", c_int32), ("table", c_void_p)]


class NormDesc(ctypes.Structure):
    """Mirror of kvq_norm_desc."""
    _fields_ = [("eps", c_float), ("per_head", c_int32), ("q_weight", c_void_p), ("k_weight", c_void_p)]


class DecodePlan(ctypes.Structure):
    """Mirror of kvq_decode_plan."""
    _fields_ = [("stream_ctas", c_int32), ("window_ctas", c_int32), ("units", c_int32),
                ("partial_slots", c_int32), ("workspace_bytes", c_size_t)]


class CacheList:
    """The caches of a model's layers as one argument (kvq_copy_blocks, kvq_fork_windows); made once."""

    def __init__(self, descs):
        self.held = list(descs)  # with the tensors that they keep
        self.array = (CacheDesc * len(self.held))(*self.held)


_lib = None

# Exported symbol -> (restype, argtypes)
SIGNATURES = {
    "kvq_status_string": (c_char_p, [c_int32]),
    "kvq_block_bytes": (c_int32, [c_int32, POINTER(c_size_t)]),
    "kvq_append": (c_int32, [POINTER(CacheDesc), c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32,
                             c_void_p, c_int32, c_int32, c_void_p, c_void_p]),
    "kvq_rope_table": (c_int32, [POINTER(RopeFreqs), c_int32, c_int32, c_void_p, c_void_p]),
    "kvq_rope_append": (c_int32, [POINTER(CacheDesc), POINTER(RopeDesc), c_void_p, c_int32, c_int64, c_void_p,
                                  c_void_p, c_int64, c_void_p, c_int64, c_int32, c_void_p, c_void_p, c_void_p,
                                  c_int32, c_void_p, c_int32, c_int32, c_void_p, c_void_p]),
    "kvq_norm_rope_append": (c_int32, [POINTER(CacheDesc), POINTER(RopeDesc), POINTER(NormDesc), c_void_p, c_int32, c_int64,
                                       c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_int32, c_void_p, c_void_p,
                                       c_void_p, c_int32, c_void_p, c_int32, c_int32, c_void_p, c_void_p]),
    "kvq_decode_shared": (c_int32, [POINTER(CacheDesc), c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_int32, c_int32,
                                    c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_size_t, c_void_p,
                                    c_void_p]),
    "kvq_decode_shared_workspace_size": (c_int32, [POINTER(CacheDesc), c_int32, c_int32, c_int32, POINTER(c_size_t)]),
    "kvq_decode_sinks": (c_int32, [POINTER(CacheDesc), c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_int32, c_int32,
                                   c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_size_t, c_int32, c_void_p,
                                   c_void_p]),
    "kvq_prefill_sinks": (c_int32, [POINTER(CacheDesc), c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32, c_void_p, c_int32, c_void_p,
                                    c_void_p, c_size_t, c_int32, c_void_p, c_void_p]),
    "kvq_attn_mass": (c_int32, [POINTER(CacheDesc), c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_int32,
                                c_void_p, c_int32, c_float, c_void_p, c_void_p]),
    "kvq_evict": (c_int32, [POINTER(CacheDesc), c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_int32,
                            c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p,
                            c_void_p]),
    "kvq_pages_update": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32,
                                   c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                   c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "kvq_pages_compact": (c_int32, [c_void_p, c_int32, c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "kvq_pages_workspace_size": (c_int32, [c_int32, POINTER(c_size_t)]),
    "kvq_copy_blocks": (c_int32, [POINTER(CacheDesc), c_int32, c_void_p, c_void_p, c_int32, c_void_p, c_void_p]),
    "kvq_fork_windows": (c_int32, [POINTER(CacheDesc), c_int32, c_void_p, c_int32, c_void_p, c_void_p]),
    "kvq_make_decode_plan": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_int32, c_int32, c_int32,
                                       POINTER(DecodePlan)]),
    "kvq_decode_device_plan": (c_int32, [POINTER(CacheDesc), c_int32, c_int32, c_int32, POINTER(DecodePlan)]),
    "kvq_decode_workspace_size": (c_int32, [POINTER(CacheDesc), c_int32, c_int32, c_int32, POINTER(c_size_t)]),
    "kvq_workspace_init": (c_int32, [c_void_p, c_size_t, c_void_p]),
    "kvq_decode": (c_int32, [POINTER(CacheDesc), c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_int32,
                             c_void_p, c_int32, c_void_p, c_void_p, c_size_t, c_int32, c_void_p, c_void_p]),
    "kvq_decode_ex": (c_int32, [POINTER(CacheDesc), c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_int32,
                                c_void_p, c_int32, c_void_p, c_void_p, c_size_t, c_int32, c_uint32, c_void_p,
                                c_void_p]),
    "kvq_dequant": (c_int32, [POINTER(CacheDesc), c_void_p, c_int32, c_void_p, c_void_p, c_void_p]),
    "kvq_prefill": (c_int32, [POINTER(CacheDesc), c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                              c_void_p, c_int32, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_size_t, c_int32,
                              c_void_p, c_void_p]),
    "kvq_prefill_workspace_size": (c_int32, [POINTER(CacheDesc), c_int32, c_int32, c_int32, POINTER(c_size_t)]),
    "kvq_decode_static_scratch": (c_int32, [POINTER(CacheDesc), c_void_p, c_int32, c_int32, c_void_p, c_void_p,
                                            c_int32, c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_void_p]),
}

STATIC_SCRATCH_BYTES = 8 << 20


def load() -> ctypes.CDLL:
    """Load libkvq.so (built in-tree by build.py); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libkvq.so not built ({LIB_PATH}); run quantized_kv_cache_07_gb300.build.build()")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().kvq_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != KVQ_OK:
        raise KvqError(status, where)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_torch = _current_device = _raw_stream = None


def _first_device() -> int:
    """The current device; later calls take it without torch's look at whether CUDA has been started."""
    global _current_device
    device = _torch.cuda.current_device()
    _current_device = getattr(_torch._C, "_cuda_getDevice", _torch.cuda.current_device)
    return device


def _need_torch():
    """torch, imported by the first call that needs it."""
    global _torch, _current_device, _raw_stream
    if _torch is None:
        import torch
        _current_device = _first_device
        # the raw handle without a Stream object per call, where this torch has it
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
        _torch = torch
    return _torch


def _stream(stream, device: int | None = None) -> int | None:
    if stream is None:
        if _torch is None:
            _need_torch()
        return _raw_stream(_current_device() if device is None else device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def block_bytes(bits: int) -> int:
    out = c_size_t(0)
    _check(load().kvq_block_bytes(bits, ctypes.byref(out)), "kvq_block_bytes")
    return out.value


def kvq_append(desc: CacheDesc, k_new, v_new, seq_idx, pos, mode: int, block_table, batch: int,
               max_blocks_per_seq: int, err_word=None, stream=None, n: int | None = None):
    n = int(seq_idx.shape[0]) if n is None else n
    _check(load().kvq_append(ctypes.byref(desc), _ptr(k_new), _ptr(v_new), n, _ptr(seq_idx), _ptr(pos), mode,
                             _ptr(block_table), batch, max_blocks_per_seq, _ptr(err_word),
                             _stream(stream) if n else None), "kvq_append")


class _Args:
    """Pointers of one call's tensor arguments; None and raw pointers pass through.  The library cannot see a
    tensor's type, layout or device: they are checked here, and a mismatch is an invalid argument."""

    __slots__ = ("where", "device")
    bf16 = f32 = i32 = u8 = None  # torch's, from the first call on

    def __init__(self, where: str):
        if _torch is None or _Args.u8 is None:
            torch = _need_torch()
            _Args.bf16, _Args.f32, _Args.i32, _Args.u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
        self.where, self.device = where, _current_device()

    def stream(self, stream):
        return _stream(stream, self.device)

    def __call__(self, t, dtype, shape=None):
        if t is None or isinstance(t, int):
            return t
        if (t.dtype is not dtype or t.get_device() != self.device or not t.is_contiguous()
                or (shape is not None and t.shape != shape)):
            raise KvqError(KVQ_ERR_INVALID_ARG, self.where)
        return t.data_ptr()

    def room(self, t, dtype, count: int):
        """The pointer of a contiguous tensor of any shape that holds `count` elements, or more."""
        if t is None or isinstance(t, int):
            return t
        if t.dtype is not dtype or t.get_device() != self.device or not t.is_contiguous() or t.numel() < count:
            raise KvqError(KVQ_ERR_INVALID_ARG, self.where)
        return t.data_ptr()

    def word(self, t):
        """The pointer of an error word: 4 bytes or more of the device."""
        if t is None or isinstance(t, int):
            return t
        if t.get_device() != self.device or t.nbytes < 4:
            raise KvqError(KVQ_ERR_INVALID_ARG, self.where)
        return t.data_ptr()

    def rows(self, t, heads: int, n: int):
        """(pointer, row stride) of bf16 rows [n, heads * 128] or [n, heads, 128] whose heads are contiguous and whose
        rows do not overlap (an expanded row has stride 0, which the library takes for heads * 128)."""
        if t is None or isinstance(t, int):
            return t, 0
        shape, stride = t.shape, t.stride()
        ok = t.dtype is self.bf16 and t.get_device() == self.device
        if ok and len(shape) == 2:
            ok = shape[0] == n and shape[1] == heads * 128 and (n == 0 or stride[1] == 1)
        elif ok:
            ok = shape == (n, heads, 128) and (n == 0 or stride[1:] == (128, 1))
        if not ok or (n > 1 and stride[0] < heads * 128):
            raise KvqError(KVQ_ERR_INVALID_ARG, self.where)
        return t.data_ptr(), stride[0] if n > 1 else 0


def kvq_rope_table(freqs: RopeFreqs, rotary_dim: int, max_pos: int, table, stream=None):
    arg = _Args("kvq_rope_table")
    _check(load().kvq_rope_table(ctypes.byref(freqs), rotary_dim, max_pos,
                                 arg.room(table, arg.f32, max_pos * rotary_dim), arg.stream(stream)), arg.where)


def kvq_rope_append(desc: CacheDesc, rope: RopeDesc, q, q_heads: int, q_out, k_new, v_new, pos, seq_idx, slot,
                    mode: int, block_table, batch: int, max_blocks_per_seq: int, err_word=None, stream=None):
    """kvq_rope_append: ``pos`` are the rope positions (int32 [n], None to use ``slot``) and ``slot`` the cache
    positions (the C argument pos).  q, k_new and v_new may be slices of one projection [n, heads * 128]: their row
    strides are taken from the tensors.  q and q_out, or k_new and v_new, may be None."""
    _rope_append(_Args("kvq_rope_append"), desc, rope, (), q, q_heads, q_out, k_new, v_new, pos, seq_idx, slot, mode,
                 block_table, batch, max_blocks_per_seq, err_word, stream)


def kvq_norm_rope_append(desc: CacheDesc, rope: RopeDesc, norm: NormDesc, q, q_heads: int, q_out, k_new, v_new, pos,
                         seq_idx, slot, mode: int, block_table, batch: int, max_blocks_per_seq: int, err_word=None,
                         stream=None):
    """kvq_norm_rope_append; ``norm`` as cache.HeadNorm makes it, the other arguments as kvq_rope_append's."""
    arg = _Args("kvq_norm_rope_append")
    for held, heads in zip(getattr(norm, "heads", ()), (q_heads, desc.num_kv_heads)):
        if held is not None and held < heads:  # weights of fewer heads than there are
            raise KvqError(KVQ_ERR_INVALID_ARG, arg.where)
    _rope_append(arg, desc, rope, (ctypes.byref(norm),), q, q_heads, q_out, k_new, v_new, pos,
                 seq_idx, slot, mode, block_table, batch, max_blocks_per_seq, err_word, stream)


def _rope_append(arg, desc, rope, norm, q, q_heads, q_out, k_new, v_new, pos, seq_idx, slot, mode, block_table, batch,
                 max_blocks_per_seq, err_word, stream):
    ref = pos if pos is not None else slot
    n = int(ref.shape[0])
    qp, qs = arg.rows(q, q_heads, n)
    kp, ks = arg.rows(k_new, desc.num_kv_heads, n)
    vp, vs = arg.rows(v_new, desc.num_kv_heads, n)
    places = batch * max_blocks_per_seq if k_new is not None and mode != APPEND_RING else 0  # read by the write alone
    entry = getattr(load(), arg.where)
    _check(entry(ctypes.byref(desc), ctypes.byref(rope), *norm, qp, q_heads, qs,
                 arg.room(q_out, arg.bf16, n * q_heads * 128), kp, ks, vp, vs, n, arg(pos, arg.i32, (n,)),
                 arg(seq_idx, arg.i32, (n,)), arg(slot, arg.i32, (n,)), mode, arg.room(block_table, arg.i32, places), batch,
                 max_blocks_per_seq, arg.word(err_word), arg.stream(stream) if n else None), arg.where)


def kvq_decode_shared_workspace_size(desc: CacheDesc, batch: int, q_heads: int, num_groups: int) -> int:
    out = c_size_t(0)
    _check(load().kvq_decode_shared_workspace_size(ctypes.byref(desc), batch, q_heads, num_groups, ctypes.byref(out)),
           "kvq_decode_shared_workspace_size")
    return out.value


def kvq_decode_shared(desc: CacheDesc, q, batch: int, q_heads: int, seq_lens, block_table, max_blocks_per_seq: int,
                      num_groups: int, group_start, prefix_blocks, out, lse=None, workspace=None,
                      workspace_bytes: int = 0, err_word=None, stream=None, out_fp32: bool | None = None):
    arg = _Args("kvq_decode_shared")
    if out_fp32 is None:
        out_fp32 = out.dtype is arg.f32
    rows = (batch, q_heads, 128)
    _check(load().kvq_decode_shared(ctypes.byref(desc), arg(q, arg.bf16, rows), batch, q_heads,
                                    arg(seq_lens, arg.i32, (batch,)), arg(block_table, arg.i32, (batch, max_blocks_per_seq)),
                                    max_blocks_per_seq, num_groups, arg(group_start, arg.i32, (num_groups + 1,)),
                                    arg(prefix_blocks, arg.i32, (num_groups,)),
                                    arg(out, arg.f32 if out_fp32 else arg.bf16, rows), int(bool(out_fp32)),
                                    arg(lse, arg.f32, (batch, q_heads)),
                                    arg.room(workspace, arg.u8, workspace_bytes), workspace_bytes,
                                    arg.word(err_word), arg.stream(stream)), arg.where)


def kvq_decode_sinks(desc: CacheDesc, q, batch: int, q_heads: int, seq_lens, block_table, max_blocks_per_seq: int,
                     sinks: int, span: int, out, lse=None, workspace=None, workspace_bytes: int = 0,
                     stream_ctas: int = 0, err_word=None, stream=None, out_fp32: bool | None = None):
    arg = _Args("kvq_decode_sinks")
    if out_fp32 is None:
        out_fp32 = out.dtype is arg.f32
    rows = (batch, q_heads, 128)
    _check(load().kvq_decode_sinks(ctypes.byref(desc), arg(q, arg.bf16, rows), batch, q_heads,
                                   arg(seq_lens, arg.i32, (batch,)), arg(block_table, arg.i32, (batch, max_blocks_per_seq)),
                                   max_blocks_per_seq, sinks, span, arg(out, arg.f32 if out_fp32 else arg.bf16, rows),
                                   int(bool(out_fp32)), arg(lse, arg.f32, (batch, q_heads)),
                                   arg.room(workspace, arg.u8, workspace_bytes), workspace_bytes, stream_ctas,
                                   arg.word(err_word), arg.stream(stream)), arg.where)


def kvq_prefill_sinks(desc: CacheDesc, q, q_heads: int, seq_idx, pos, block_table, batch: int, max_blocks_per_seq: int,
                      sinks: int, span: int, out, k_new=None, v_new=None, lse=None, workspace=None,
                      workspace_bytes: int = 0, stream_ctas: int = 0, err_word=None, stream=None,
                      out_fp32: bool | None = None):
    arg = _Args("kvq_prefill_sinks")
    n = int(pos.shape[0])
    if out_fp32 is None:
        out_fp32 = out.dtype is arg.f32
    rows, new = (n, q_heads, 128), (n, desc.num_kv_heads, 128)
    _check(load().kvq_prefill_sinks(ctypes.byref(desc), arg(q, arg.bf16, rows), n, q_heads, arg(seq_idx, arg.i32, (n,)),
                                    arg(pos, arg.i32, (n,)), arg(k_new, arg.bf16, new), arg(v_new, arg.bf16, new),
                                    arg(block_table, arg.i32, (batch, max_blocks_per_seq)), batch, max_blocks_per_seq,
                                    sinks, span, arg(out, arg.f32 if out_fp32 else arg.bf16, rows), int(bool(out_fp32)),
                                    arg(lse, arg.f32, (n, q_heads)), arg.room(workspace, arg.u8, workspace_bytes),
                                    workspace_bytes, stream_ctas, arg.word(err_word), arg.stream(stream)), arg.where)


def kvq_attn_mass(desc: CacheDesc, q, batch: int, q_heads: int, lse, seq_lens, block_table, max_blocks_per_seq: int,
                  mass, decay: float = 1.0, err_word=None, stream=None, mass_stride: int | None = None):
    """kvq_attn_mass; ``mass`` is float32 [batch, kv_heads, mass_stride]."""
    arg = _Args("kvq_attn_mass")
    if mass_stride is None:
        mass_stride = int(mass.shape[-1])
    _check(load().kvq_attn_mass(ctypes.byref(desc), arg(q, arg.bf16, (batch, q_heads, 128)), batch, q_heads,
                                arg(lse, arg.f32, (batch, q_heads)), arg(seq_lens, arg.i32, (batch,)),
                                arg(block_table, arg.i32, (batch, max_blocks_per_seq)), max_blocks_per_seq,
                                arg(mass, arg.f32, (batch, desc.num_kv_heads, mass_stride)), mass_stride, decay,
                                arg.word(err_word), arg.stream(stream)), arg.where)


def kvq_evict(desc: CacheDesc, mass, mass_out, seq_lens, keep, block_table, batch: int, max_blocks_per_seq: int,
              source, new_lens, protect_first: int = 0, protect_recent: int = 0, token_pos=None, token_pos_out=None,
              next_pos=None, err_word=None, stream=None, mass_stride: int | None = None):
    """kvq_evict; mass, mass_out, source, token_pos and token_pos_out are [batch, kv_heads, mass_stride]."""
    arg = _Args("kvq_evict")
    if mass_stride is None:
        mass_stride = int(mass.shape[-1])
    rows, each = (batch, desc.num_kv_heads, mass_stride), (batch,)
    _check(load().kvq_evict(ctypes.byref(desc), arg(mass, arg.f32, rows), arg(mass_out, arg.f32, rows), mass_stride,
                            arg(seq_lens, arg.i32, each), arg(keep, arg.i32, each), protect_first, protect_recent,
                            arg(token_pos, arg.i32, rows), arg(token_pos_out, arg.i32, rows),
                            arg(next_pos, arg.i32, each), arg(block_table, arg.i32, (batch, max_blocks_per_seq)), batch,
                            max_blocks_per_seq, arg(new_lens, arg.i32, each), arg(source, arg.i32, rows),
                            arg.word(err_word), arg.stream(stream)), arg.where)


def kvq_pages_workspace_size(num_blocks: int) -> int:
    out = c_size_t(0)
    _check(load().kvq_pages_workspace_size(num_blocks, ctypes.byref(out)), "kvq_pages_workspace_size")
    return out.value


def kvq_pages_update(refs, block_table, seq_lens, refs_out, table_out, lens_out, copies, num_copies, parent=None,
                     room=0, window: int = 0, sinks: int = 0, span: int = 0, parent_out=None, workspace=None,
                     err_word=None, stream=None):
    """kvq_pages_update; refs are int32 [num_blocks], tables [batch, max_blocks_per_seq], copies [batch, 2]; room is a
    number for all rows or an int32 tensor [batch] (the C argument rooms)."""
    arg = _Args("kvq_pages_update")
    n, (batch, width) = int(refs.shape[0]), block_table.shape
    rooms = None
    if not isinstance(room, int):
        room, rooms = 0, arg(room, arg.i32, (batch,))
    _check(load().kvq_pages_update(arg(refs, arg.i32, (n,)), n, arg(block_table, arg.i32, (batch, width)),
                                   arg(seq_lens, arg.i32, (batch,)), arg(parent, arg.i32, (batch,)), batch, width, window,
                                   room, rooms, sinks, span, arg(refs_out, arg.i32, (n,)),
                                   arg(table_out, arg.i32, (batch, width)), arg(lens_out, arg.i32, (batch,)),
                                   arg(parent_out, arg.i32, (batch,)), arg.room(copies, arg.i32, 2 * batch),
                                   arg.room(num_copies, arg.i32, 1), arg.room(workspace, arg.u8, 0),
                                   0 if workspace is None else workspace.numel(), arg.word(err_word),
                                   arg.stream(stream)), arg.where)


def kvq_pages_compact(refs, block_table, refs_out, table_out, moves, counts, workspace=None, err_word=None, stream=None):
    """kvq_pages_compact; moves are int32 [num_blocks / 2, 2] (one pair at least), counts [2]; without a table, None
    twice."""
    arg = _Args("kvq_pages_compact")
    n = int(refs.shape[0])
    batch, width = (0, 0) if block_table is None else block_table.shape
    _check(load().kvq_pages_compact(arg(refs, arg.i32, (n,)), n, arg(block_table, arg.i32, (batch, width)), batch, width,
                                    arg(refs_out, arg.i32, (n,)), arg(table_out, arg.i32, (batch, width)),
                                    arg.room(moves, arg.i32, 2 * max(n // 2, 1)), arg.room(counts, arg.i32, 2),
                                    arg.room(workspace, arg.u8, 0), 0 if workspace is None else workspace.numel(),
                                    arg.word(err_word), arg.stream(stream)), arg.where)


def kvq_copy_blocks(caches: CacheList, copies, num_copies, err_word=None, stream=None):
    """kvq_copy_blocks of the first num_copies[0] pairs of copies (int32 [.., 2])."""
    arg = _Args("kvq_copy_blocks")
    pairs = copies.numel() // 2
    _check(load().kvq_copy_blocks(caches.array, len(caches.held), arg.room(copies, arg.i32, 2 * pairs),
                                  arg.room(num_copies, arg.i32, 1), pairs, arg.word(err_word), arg.stream(stream)),
           arg.where)


def kvq_fork_windows(caches: CacheList, parent, batch: int, err_word=None, stream=None):
    arg = _Args("kvq_fork_windows")
    _check(load().kvq_fork_windows(caches.array, len(caches.held), arg(parent, arg.i32, (batch,)), batch,
                                   arg.word(err_word), arg.stream(stream)), arg.where)


def kvq_make_decode_plan(batch: int, q_heads: int, kv_heads: int, window: int, num_sms: int, ctas_per_sm: int,
                         stream_ctas: int = 0) -> DecodePlan:
    plan = DecodePlan()
    _check(load().kvq_make_decode_plan(batch, q_heads, kv_heads, window, num_sms, ctas_per_sm, stream_ctas,
                                       ctypes.byref(plan)), "kvq_make_decode_plan")
    return plan


def kvq_decode_device_plan(desc: CacheDesc, batch: int, q_heads: int, stream_ctas: int = 0) -> DecodePlan:
    plan = DecodePlan()
    _check(load().kvq_decode_device_plan(ctypes.byref(desc), batch, q_heads, stream_ctas, ctypes.byref(plan)),
           "kvq_decode_device_plan")
    return plan


def kvq_decode_workspace_size(desc: CacheDesc, batch: int, q_heads: int, stream_ctas: int = 0) -> int:
    out = c_size_t(0)
    _check(load().kvq_decode_workspace_size(ctypes.byref(desc), batch, q_heads, stream_ctas, ctypes.byref(out)),
           "kvq_decode_workspace_size")
    return out.value


def kvq_workspace_init(workspace, nbytes: int, stream=None):
    _check(load().kvq_workspace_init(_ptr(workspace), nbytes, _stream(stream)), "kvq_workspace_init")


def kvq_decode(desc: CacheDesc, q, batch: int, q_heads: int, seq_lens, block_table, max_blocks_per_seq: int, out,
               lse=None, workspace=None, workspace_bytes: int = 0, stream_ctas: int = 0, err_word=None,
               stream=None, out_fp32: bool | None = None, flags: int = 0):
    """kvq_decode (flags 0) or kvq_decode_ex with flags (DECODE_GEOMETRY_READY)."""
    if out_fp32 is None:
        import torch
        out_fp32 = out.dtype == torch.float32
    if flags:
        _check(load().kvq_decode_ex(ctypes.byref(desc), _ptr(q), batch, q_heads, _ptr(seq_lens), _ptr(block_table),
                                    max_blocks_per_seq, _ptr(out), int(bool(out_fp32)), _ptr(lse), _ptr(workspace),
                                    workspace_bytes, stream_ctas, flags, _ptr(err_word), _stream(stream)),
               "kvq_decode_ex")
        return
    _check(load().kvq_decode(ctypes.byref(desc), _ptr(q), batch, q_heads, _ptr(seq_lens), _ptr(block_table),
                             max_blocks_per_seq, _ptr(out), int(bool(out_fp32)), _ptr(lse), _ptr(workspace),
                             workspace_bytes, stream_ctas, _ptr(err_word), _stream(stream)), "kvq_decode")


def kvq_prefill_workspace_size(desc: CacheDesc, n: int, q_heads: int, stream_ctas: int = 0) -> int:
    out = c_size_t(0)
    _check(load().kvq_prefill_workspace_size(ctypes.byref(desc), n, q_heads, stream_ctas, ctypes.byref(out)),
           "kvq_prefill_workspace_size")
    return out.value


def kvq_prefill(desc: CacheDesc, q, q_heads: int, seq_idx, pos, block_table, batch: int, max_blocks_per_seq: int,
                out, k_new=None, v_new=None, lse=None, workspace=None, workspace_bytes: int = 0, stream_ctas: int = 0,
                err_word=None, stream=None, out_fp32: bool | None = None, n: int | None = None):
    n = int(seq_idx.shape[0]) if n is None else n
    if out_fp32 is None:
        import torch
        out_fp32 = out.dtype == torch.float32
    _check(load().kvq_prefill(ctypes.byref(desc), _ptr(q), n, q_heads, _ptr(seq_idx), _ptr(pos), _ptr(k_new),
                              _ptr(v_new), _ptr(block_table), batch, max_blocks_per_seq, _ptr(out),
                              int(bool(out_fp32)), _ptr(lse), _ptr(workspace), workspace_bytes, stream_ctas,
                              _ptr(err_word), _stream(stream)), "kvq_prefill")


def kvq_dequant(desc: CacheDesc, slots, k_out, v_out, stream=None, n: int | None = None):
    n = int(slots.shape[0]) if n is None else n
    _check(load().kvq_dequant(ctypes.byref(desc), _ptr(slots), n, _ptr(k_out), _ptr(v_out), _stream(stream)),
           "kvq_dequant")


def kvq_decode_static_scratch(desc: CacheDesc, q, batch: int, q_heads: int, seq_lens, block_table,
                              max_blocks_per_seq: int, out, lse=None, stream_ctas: int = 0, err_word=None,
                              stream=None, out_fp32: bool | None = None):
    """kvq_decode without a caller workspace (fixed device scratch inside the
    library; see include/kvq.h for the size limit and the sharing rules)."""
    if out_fp32 is None:
        import torch
        out_fp32 = out.dtype == torch.float32
    _check(load().kvq_decode_static_scratch(ctypes.byref(desc), _ptr(q), batch, q_heads, _ptr(seq_lens),
                                            _ptr(block_table), max_blocks_per_seq, _ptr(out), int(bool(out_fp32)),
                                            _ptr(lse), stream_ctas, _ptr(err_word), _stream(stream)),
           "kvq_decode_static_scratch")
