"""ctypes binding of libgtq (the C ABI in include/gtq.h).

Argument marshalling only: every step of the hot path runs in the CUDA library
(``libgtq.so``, built in-tree by ``decode_attention_13_b200.build``).  There is
no Python or CPU fallback: importing this package raises if the library is
missing, and every wrapper raises ``GtqError`` on a nonzero return code.

The functions mirror the C ABI in ``include/gtq.h``:

    plan = gtq_alloc_bits(cfg, k, T, stream=None)          # energy + greedy
    gtq_quantize_pack(plan, k, v, t0, n, packed, stream=None)
    gtq_decode_attn(plan, packed, T, q, out, stream=None)
    gtq_free(plan)

Tensor arguments may be torch tensors (CUDA memory; their data pointer and
strides are passed through) or raw integer device pointers.
A call runs on `stream` (a torch stream or a raw handle).  stream=None is CUDA's
legacy default stream, not torch's current one: under `torch.cuda.stream(s)` pass
stream=s, or the call is not ordered with what torch does on s.

gtq_rope, gtq_chunk_attn, gtq_attn_weights and gtq_evict refuse (ValueError)
tensors of another type than their kernels read, and tensors that are not on the
plan's GPU (gtq_rope: the current one).
"""

from __future__ import annotations

import ctypes
import math
import os
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgtq.so")

GTQ_OK = 0
GTQ_T0_TAIL = -1  # gtq_quantize_pack_ex: write the last n tokens of every sequence
GTQ_ERR_INVALID = -1
GTQ_ERR_UNSUPPORTED = -2
GTQ_ERR_CUDA = -3
GTQ_ERR_OOM = -4
GTQ_ERR_TIMEOUT = -5
GTQ_ERR_OVERFLOW = -6
GTQ_ERR_STATE = -7
PAIRING_HALF = 0
PAIRING_INTERLEAVED = 1
DTYPE_FP16 = 0
DTYPE_FP32 = 1
ROPE_PLAIN = 0
ROPE_LINEAR = 1
ROPE_LLAMA3 = 2
ROPE_YARN = 3
TILE_TOKENS = 64
TAG_KEY = 0x4B
TAG_VALUE = 0x56

ABI_FUNCTIONS = (
    "gtq_alloc_bits", "gtq_alloc_bits_from_energy", "gtq_quantize_pack", "gtq_decode_attn",
    "gtq_free", "gtq_packed_bytes", "gtq_get_bits", "gtq_get_energy", "gtq_status",
    "gtq_strerror", "gtq_last_error", "gtq_lloyd_max", "gtq_rotation", "gtq_layout_tile_bytes",
    "gtq_block_energy_noalloc", "gtq_plan_device_bytes", "gtq_raise_status",
    "gtq_alloc_bits_ex", "gtq_quantize_pack_ex", "gtq_decode_attn_ex", "gtq_decode_attn_full",
    "gtq_rope", "gtq_chunk_attn", "gtq_chunk_workspace_bytes", "gtq_attn_weights",
    "gtq_weights_workspace_bytes", "gtq_evict", "gtq_evict_workspace_bytes",
)


_I64x4 = ctypes.c_int64 * 4


class GtqError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        detail = ""
        if code in (GTQ_ERR_CUDA, GTQ_ERR_OOM):
            detail = " [%s]" % _lib.gtq_last_error().decode()
        super().__init__("%s failed: %s (%d)%s" % (where, strerror(code), code, detail))


class gtq_config(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("k_bits", ctypes.c_int32), ("v_bits", ctypes.c_int32),
        ("max_bits", ctypes.c_int32), ("rope_pairing", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("seed", ctypes.c_uint64), ("t_capacity", ctypes.c_int64),
    ]


class gtq_seq_layout(ctypes.Structure):
    _fields_ = [
        ("seq_lens_dev", ctypes.c_void_p), ("block_table_dev", ctypes.c_void_p),
        ("max_blocks", ctypes.c_int64),
    ]


def seq_layout(seq_lens=None, block_table=None):
    """A gtq_seq_layout from device int32 tensors: lengths [batch] and a block
    table [batch][max_blocks] (either may be None).  Keep the tensors alive
    while the calls that use the layout run."""
    lay = gtq_seq_layout(None, None, 0)
    if seq_lens is not None:
        lay.seq_lens_dev = _ptr(seq_lens)
    if block_table is not None:
        lay.block_table_dev = _ptr(block_table)
        lay.max_blocks = int(block_table.shape[1])
    return lay


class gtq_fp16_kv(ctypes.Structure):
    _fields_ = [
        ("v_dev", ctypes.c_void_p), ("v_strides", ctypes.c_int64 * 4),
        ("recent_k_dev", ctypes.c_void_p), ("recent_v_dev", ctypes.c_void_p),
        ("recent_strides", ctypes.c_int64 * 4), ("recent_lens_dev", ctypes.c_void_p),
        ("recent_len", ctypes.c_int64),
    ]


def fp16_kv(v=None, recent_k=None, recent_v=None, recent_lens=None, recent_len=None):
    """A gtq_fp16_kv from device fp16 tensors: values [batch, kv_heads, tokens, 128]
    of a K-only plan, and a window of recent keys / values [batch, kv_heads, rows,
    128] (same strides for both) with optional int32 lengths [batch].  Keep the
    tensors alive while the calls that use it run."""
    kv = gtq_fp16_kv()
    if v is not None:
        kv.v_dev = _ptr(v)
        kv.v_strides = (ctypes.c_int64 * 4)(*[int(s) for s in v.stride()])
    if recent_k is not None:
        if tuple(recent_k.stride()) != tuple(recent_v.stride()):
            raise ValueError("recent keys and values must share strides")
        kv.recent_k_dev = _ptr(recent_k)
        kv.recent_v_dev = _ptr(recent_v)
        kv.recent_strides = (ctypes.c_int64 * 4)(*[int(s) for s in recent_k.stride()])
        kv.recent_len = int(recent_k.shape[2]) if recent_len is None else int(recent_len)
    if recent_lens is not None:
        kv.recent_lens_dev = _ptr(recent_lens)
    return kv


class gtq_rope_config(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
        ("rope_pairing", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("scaling", ctypes.c_int32), ("backward", ctypes.c_int32),
        ("theta", ctypes.c_double), ("factor", ctypes.c_double),
        ("original_context", ctypes.c_double), ("low_freq", ctypes.c_double),
        ("high_freq", ctypes.c_double), ("magnitude", ctypes.c_double),
    ]


class gtq_rope_tensor(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("heads", ctypes.c_int32),
        ("reserved", ctypes.c_int32), ("x_strides", ctypes.c_int64 * 4),
        ("y_strides", ctypes.c_int64 * 4),
    ]


class gtq_chunk(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int64), ("chunk_lens_dev", ctypes.c_void_p),
        ("causal", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("q_strides", ctypes.c_int64 * 4), ("out_strides", ctypes.c_int64 * 4),
    ]


class gtq_eviction(ctypes.Structure):
    _fields_ = [
        ("keep", ctypes.c_int64), ("n_first", ctypes.c_int64), ("n_recent", ctypes.c_int64),
        ("weights_dev", ctypes.c_void_p), ("w_strides", ctypes.c_int64 * 2),
        ("weights_out_dev", ctypes.c_void_p), ("w_out_strides", ctypes.c_int64 * 2),
        ("kept_dev", ctypes.c_void_p), ("new_lens_dev", ctypes.c_void_p),
    ]


def make_rope(head_dim, theta, rotary_dim=None, rope_pairing=PAIRING_HALF, dtype=DTYPE_FP16,
              scaling=ROPE_PLAIN, factor=1.0, original_context=0.0, low_freq=1.0, high_freq=None,
              magnitude=None, backward=False) -> gtq_rope_config:
    """A gtq_rope_config.  rotary_dim defaults to the whole head; the ramp's turns and the magnitude to
    what is customary for the scaling: 1 and 4 turns (ROPE_LLAMA3), 1 and 32 turns with the
    magnitude 0.1 ln(factor) + 1 (ROPE_YARN), and else the magnitude 1."""
    yarn = scaling == ROPE_YARN
    if high_freq is None:
        high_freq = 32.0 if yarn else 4.0
    if magnitude is None:
        magnitude = 0.1 * math.log(factor) + 1.0 if yarn and factor > 0 else 1.0
    return gtq_rope_config(head_dim, head_dim if rotary_dim is None else rotary_dim, rope_pairing,
                           dtype, scaling, int(backward), theta, factor, original_context,
                           low_freq, high_freq, magnitude)


def make_config(batch, n_q_heads, n_kv_heads, k_bits, v_bits, t_capacity, head_dim=128,
                max_bits=8, rope_pairing=PAIRING_HALF, in_dtype=DTYPE_FP16, seed=0) -> gtq_config:
    return gtq_config(batch, n_q_heads, n_kv_heads, head_dim, k_bits, v_bits, max_bits,
                      rope_pairing, in_dtype, 0, seed, t_capacity)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libgtq.so not built (run `python -m decode_attention_13_b200.build`); "
                          "there is no fallback implementation")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    I64x4 = ctypes.POINTER(ctypes.c_int64)
    sig = {
        "gtq_alloc_bits": (I32, [ctypes.POINTER(gtq_config), P, I64, I64x4, P, ctypes.POINTER(P)]),
        "gtq_alloc_bits_from_energy": (I32, [ctypes.POINTER(gtq_config), ctypes.POINTER(ctypes.c_double), ctypes.POINTER(P)]),
        "gtq_quantize_pack": (I32, [P, P, P, I64x4, I64, I64, P, SZ, P]),
        "gtq_decode_attn": (I32, [P, P, I64, P, I32, P, P]),
        "gtq_free": (I32, [P]),
        "gtq_packed_bytes": (SZ, [P]),
        "gtq_get_bits": (I32, [P, ctypes.POINTER(ctypes.c_uint8), P]),
        "gtq_get_energy": (I32, [P, ctypes.POINTER(ctypes.c_double), P]),
        "gtq_status": (I32, [P]),
        "gtq_strerror": (ctypes.c_char_p, [I32]),
        "gtq_last_error": (ctypes.c_char_p, []),
        "gtq_lloyd_max": (I32, [I32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]),
        "gtq_rotation": (I32, [ctypes.c_uint64, I32, I32, ctypes.POINTER(ctypes.c_double)]),
        "gtq_layout_tile_bytes": (SZ, [I32, I32]),
        "gtq_block_energy_noalloc": (I32, [ctypes.POINTER(gtq_config), P, I64, I64x4, P, P]),
        "gtq_plan_device_bytes": (SZ, [P]),
        "gtq_raise_status": (I32, [P, I32]),
        "gtq_alloc_bits_ex": (I32, [ctypes.POINTER(gtq_config), P, I64, I64x4,
                                    ctypes.POINTER(gtq_seq_layout), P, ctypes.POINTER(P)]),
        "gtq_quantize_pack_ex": (I32, [P, P, P, I64x4, I64, I64, P, SZ,
                                       ctypes.POINTER(gtq_seq_layout), P]),
        "gtq_decode_attn_ex": (I32, [P, P, I64, ctypes.POINTER(gtq_seq_layout), P, I32, P, P]),
        "gtq_decode_attn_full": (I32, [P, P, I64, ctypes.POINTER(gtq_seq_layout),
                                       ctypes.POINTER(gtq_fp16_kv), P, I32, P, P]),
        "gtq_rope": (I32, [ctypes.POINTER(gtq_rope_config), I64, I64, P, I64, I64,
                           ctypes.POINTER(gtq_rope_tensor), ctypes.POINTER(gtq_rope_tensor), P]),
        "gtq_chunk_attn": (I32, [P, P, I64, ctypes.POINTER(gtq_seq_layout),
                                 ctypes.POINTER(gtq_chunk), P, P, P, SZ, P]),
        "gtq_chunk_workspace_bytes": (SZ, [P, I64, I64]),
        "gtq_attn_weights": (I32, [P, P, I64, ctypes.POINTER(gtq_seq_layout),
                                   ctypes.POINTER(gtq_chunk), P, P, P, I64x4, P, SZ, P]),
        "gtq_weights_workspace_bytes": (SZ, [P, I64, I64]),
        "gtq_evict": (I32, [P, P, I64, ctypes.POINTER(gtq_seq_layout),
                            ctypes.POINTER(gtq_eviction), P, SZ, ctypes.POINTER(gtq_seq_layout),
                            P, SZ, P]),
        "gtq_evict_workspace_bytes": (SZ, [P, I64]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


_lib = _load()


def library():
    """The loaded ctypes library (for ABI checks)."""
    return _lib


def strerror(code: int) -> str:
    return _lib.gtq_strerror(int(code)).decode()


def _check(rc: int, where: str) -> None:
    if rc != GTQ_OK:
        raise GtqError(rc, where)


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream(s) -> int:
    if s is None:
        return 0
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _current_device():
    torch = sys.modules.get("torch")
    return torch.cuda.current_device() if torch is not None and torch.cuda.is_initialized() else None


def _need(x, what: str, device, dtype=None) -> None:
    """Refuses a tensor of another type, or one that is not on the GPU `device` (None: any)."""
    if x is None or isinstance(x, int):  # absent, or a raw device pointer
        return
    if dtype is not None and x.dtype is not dtype:
        raise ValueError("%s must be %s, not %s" % (what, str(dtype)[6:], str(x.dtype)[6:]))
    at = x.get_device()
    if at < 0:
        raise ValueError("%s must be on a GPU, not %s" % (what, x.device))
    if device is not None and at != device:
        raise ValueError("%s must be on cuda:%d, not %s" % (what, device, x.device))


def _strides4(x, strides):
    if strides is not None:
        return (ctypes.c_int64 * 4)(*[int(v) for v in strides])
    st = tuple(int(v) for v in x.stride())
    if len(st) != 4:
        raise ValueError("K/V must be 4-D [batch, kv_heads, tokens, head_dim]")
    return (ctypes.c_int64 * 4)(*st)


class Plan:
    """Owning handle of a gtq_plan (freed by gtq_free or on garbage collection).  device: the index
    of the GPU it was made on, or None where torch does not know it."""

    def __init__(self, handle: int, cfg: gtq_config, device=None):
        self.handle = handle
        self.cfg = cfg
        self.device = _current_device() if device is None else device

    @property
    def packed_bytes(self) -> int:
        return int(_lib.gtq_packed_bytes(self.handle))

    def free(self) -> None:
        if self.handle:
            h, self.handle = self.handle, None
            _check(_lib.gtq_free(h), "gtq_free")

    def __del__(self):
        try:
            if self.handle:
                _lib.gtq_free(self.handle)
        except Exception:
            pass


def gtq_alloc_bits(cfg: gtq_config, k, T: int, stream=None, strides=None) -> Plan:
    out = ctypes.c_void_p()
    rc = _lib.gtq_alloc_bits(ctypes.byref(cfg), _ptr(k), int(T), _strides4(k, strides),
                             _stream(stream), ctypes.byref(out))
    _check(rc, "gtq_alloc_bits")
    return Plan(out.value, cfg)


def gtq_alloc_bits_from_energy(cfg: gtq_config, energy) -> Plan:
    import numpy as np

    e = np.ascontiguousarray(energy, dtype=np.float64)
    out = ctypes.c_void_p()
    rc = _lib.gtq_alloc_bits_from_energy(ctypes.byref(cfg),
                                         e.ctypes.data_as(ctypes.POINTER(ctypes.c_double)),
                                         ctypes.byref(out))
    _check(rc, "gtq_alloc_bits_from_energy")
    return Plan(out.value, cfg)


def gtq_quantize_pack(plan: Plan, k, v, t0: int, n_tokens: int, packed, stream=None,
                      strides=None, packed_bytes=None) -> None:
    nbytes = packed_bytes if packed_bytes is not None else (
        packed.numel() * packed.element_size())
    rc = _lib.gtq_quantize_pack(plan.handle, _ptr(k), _ptr(v), _strides4(k, strides), int(t0),
                                int(n_tokens), _ptr(packed), int(nbytes), _stream(stream))
    _check(rc, "gtq_quantize_pack")


def gtq_decode_attn(plan: Plan, packed, T: int, q, out, stream=None, q_dtype=None) -> None:
    if q_dtype is None:
        import torch

        q_dtype = DTYPE_FP32 if q.dtype == torch.float32 else DTYPE_FP16
    rc = _lib.gtq_decode_attn(plan.handle, _ptr(packed), int(T), _ptr(q), int(q_dtype),
                              _ptr(out), _stream(stream))
    _check(rc, "gtq_decode_attn")


def _lay(layout):
    return None if layout is None else ctypes.byref(layout)


def gtq_alloc_bits_ex(cfg: gtq_config, k, T: int, layout=None, stream=None,
                      strides=None) -> Plan:
    out = ctypes.c_void_p()
    rc = _lib.gtq_alloc_bits_ex(ctypes.byref(cfg), _ptr(k), int(T), _strides4(k, strides),
                                _lay(layout), _stream(stream), ctypes.byref(out))
    _check(rc, "gtq_alloc_bits_ex")
    return Plan(out.value, cfg)


def gtq_quantize_pack_ex(plan: Plan, k, v, t0: int, n_tokens: int, packed, layout=None,
                         stream=None, strides=None, packed_bytes=None) -> None:
    nbytes = packed_bytes if packed_bytes is not None else (
        packed.numel() * packed.element_size())
    rc = _lib.gtq_quantize_pack_ex(plan.handle, _ptr(k), _ptr(v), _strides4(k, strides),
                                   int(t0), int(n_tokens), _ptr(packed), int(nbytes),
                                   _lay(layout), _stream(stream))
    _check(rc, "gtq_quantize_pack_ex")


def gtq_decode_attn_ex(plan: Plan, packed, T: int, q, out, layout=None, stream=None,
                       q_dtype=None) -> None:
    if q_dtype is None:
        import torch

        q_dtype = DTYPE_FP32 if q.dtype == torch.float32 else DTYPE_FP16
    rc = _lib.gtq_decode_attn_ex(plan.handle, _ptr(packed), int(T), _lay(layout), _ptr(q),
                                 int(q_dtype), _ptr(out), _stream(stream))
    _check(rc, "gtq_decode_attn_ex")


def gtq_decode_attn_full(plan: Plan, packed, T: int, q, out, layout=None, kv=None, stream=None,
                         q_dtype=None) -> None:
    if q_dtype is None:
        import torch

        q_dtype = DTYPE_FP32 if q.dtype == torch.float32 else DTYPE_FP16
    rc = _lib.gtq_decode_attn_full(plan.handle, _ptr(packed), int(T), _lay(layout),
                                   None if kv is None else ctypes.byref(kv), _ptr(q),
                                   int(q_dtype), _ptr(out), _stream(stream))
    _check(rc, "gtq_decode_attn_full")


def _rope_tensor(cfg, x, y, batch, tokens, name, dtype, device):
    shape = x.shape
    if x.dtype is not dtype or device < 0 or x.get_device() != device:
        _need(x, name, device, dtype)
    if len(shape) != 4 or shape[3] != cfg.head_dim or shape[0] != batch or shape[2] != tokens:
        raise ValueError("%s must be [%d, heads, %d, %d]" % (name, batch, tokens, cfg.head_dim))
    st = _I64x4(*x.stride())
    if y is None:
        return gtq_rope_tensor(x.data_ptr(), x.data_ptr(), shape[1], 0, st, st)
    if y.dtype is not dtype or y.get_device() != device:
        _need(y, name + "_out", device, dtype)
    if y.shape != shape:
        raise ValueError("%s and its output must have one shape" % name)
    return gtq_rope_tensor(x.data_ptr(), y.data_ptr(), shape[1], 0, st, _I64x4(*y.stride()))


def gtq_rope(cfg: gtq_rope_config, q=None, q_out=None, k=None, k_out=None, positions=None, pos0=0,
             stream=None) -> None:
    """Rotate q and / or k ([batch, heads, tokens, head_dim], any strides with a dense last dim)
    into q_out / k_out (None: in place).  positions: int64 [batch, tokens] or [tokens], or None:
    pos0 + token.  stream: None is the legacy default stream, not torch's current one."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("gtq_rope needs q or k")
    shape = first.shape
    if len(shape) != 4:
        raise ValueError("gtq_rope takes [batch, heads, tokens, head_dim]")
    batch, _, tokens, _ = shape
    import torch

    dtype = torch.float16 if cfg.dtype == DTYPE_FP16 else torch.float32
    device = first.get_device()
    if device >= 0 and device != torch.cuda.current_device():
        raise ValueError("gtq_rope runs on the current device, cuda:%d" % torch.cuda.current_device())
    pos_stride = pos_ptr = 0
    if positions is not None:
        ps = positions.shape
        if positions.dtype is not torch.int64 or positions.get_device() != device:
            _need(positions, "positions", device, torch.int64)
        if not ps or ps[-1] != tokens or len(ps) > 2 or (len(ps) == 2 and ps[0] != batch):
            raise ValueError("positions must be int64 [batch, tokens] or [tokens]")
        st = positions.stride()
        if tokens > 1 and st[-1] != 1:
            raise ValueError("positions must be dense along tokens")
        if len(ps) == 2 and batch > 1:
            pos_stride = st[0]
        pos_ptr = positions.data_ptr()
    tq = None if q is None else ctypes.byref(_rope_tensor(cfg, q, q_out, batch, tokens, "q", dtype, device))
    tk = None if k is None else ctypes.byref(_rope_tensor(cfg, k, k_out, batch, tokens, "k", dtype, device))
    rc = _lib.gtq_rope(ctypes.byref(cfg), batch, tokens, pos_ptr, pos_stride, pos0, tq, tk,
                       _stream(stream))
    if rc != GTQ_OK:
        _check(rc, "gtq_rope")


def _chunk(plan, q, out, chunk_lens, causal, packed=None, workspace=None):
    import torch

    c, device = plan.cfg, plan.device
    if q.dim() != 4 or q.shape[0] != c.batch or q.shape[1] != c.n_q_heads or q.shape[3] != c.head_dim:
        raise ValueError("q must be fp16 [batch, query heads, new tokens, %d]" % c.head_dim)
    if out is not None and tuple(out.shape) != tuple(q.shape):
        raise ValueError("out must have the shape of q")
    _need(q, "q", device, torch.float16)
    _need(out, "out", device, torch.float16)
    _lens(chunk_lens, "chunk_lens", plan)
    _need(packed, "packed", device)
    _need(workspace, "workspace", device)
    ch = gtq_chunk(int(q.shape[2]), _ptr(chunk_lens) or None, int(bool(causal)), 0)
    ch.q_strides = _live_strides(q)
    ch.out_strides = _live_strides(out if out is not None else q)
    return ch


def _lens(x, what, plan):
    import torch

    _need(x, what, plan.device, torch.int32)
    if x is not None and not isinstance(x, int) and (x.numel() != plan.cfg.batch or not x.is_contiguous()):
        raise ValueError("%s must be contiguous int32 [batch]" % what)


def _live_strides(x):
    """Strides with 0 for dims of one element, whose stride says nothing."""
    return (ctypes.c_int64 * 4)(*[int(s) if n > 1 else 0 for n, s in zip(x.shape[:3], x.stride()[:3])],
                                int(x.stride(3)))


def _nbytes(x) -> int:
    return int(x.numel() * x.element_size())


def gtq_chunk_workspace(plan: Plan, T: int, n_tokens: int) -> int:
    """Bytes of the workspace gtq_chunk_attn needs for these sizes."""
    return int(_lib.gtq_chunk_workspace_bytes(plan.handle, int(T), int(n_tokens)))


def gtq_chunk_attn(plan: Plan, packed, T: int, q, out, workspace, layout=None, chunk_lens=None,
                   causal=True, stream=None) -> None:
    """Attention of the new tokens q [batch, query heads, new tokens, 128] (fp16, any strides with
    dense rows) over the cache into out (the same shape).  stream: None is the legacy default
    stream, not torch's current one."""
    ch = _chunk(plan, q, out, chunk_lens, causal, packed, workspace)
    rc = _lib.gtq_chunk_attn(plan.handle, _ptr(packed), int(T), _lay(layout), ctypes.byref(ch),
                             _ptr(q), _ptr(out), _ptr(workspace), _nbytes(workspace),
                             _stream(stream))
    _check(rc, "gtq_chunk_attn")


def gtq_weights_workspace(plan: Plan, T: int, n_tokens: int) -> int:
    """Bytes of the workspace gtq_attn_weights needs for these sizes."""
    return int(_lib.gtq_weights_workspace_bytes(plan.handle, int(T), int(n_tokens)))


def _weights2(w, plan, what):
    import torch

    if w.dim() != 3 or tuple(w.shape[:2]) != (plan.cfg.batch, plan.cfg.n_kv_heads):
        raise ValueError("%s must be fp32 [batch, kv heads, tokens]" % what)
    _need(w, what, plan.device, torch.float32)
    if w.shape[2] > 1 and w.stride(2) != 1:
        raise ValueError("%s must be dense along tokens" % what)
    return (ctypes.c_int64 * 2)(int(w.stride(0)), int(w.stride(1)))


def gtq_attn_weights(plan: Plan, packed, T: int, q, weights_out, workspace, weights_in=None,
                     layout=None, chunk_lens=None, causal=True, stream=None) -> None:
    """weights_out = weights_in (or 0) + the attention every cached token gets from q; both
    [batch, kv heads, >= T] fp32.  stream: None is the legacy default stream, not torch's current
    one."""
    ch = _chunk(plan, q, None, chunk_lens, causal, packed, workspace)
    st = _weights2(weights_out, plan, "weights_out")
    if weights_out.shape[2] < T or (weights_in is not None and (
            weights_in.shape[2] < T or tuple(_weights2(weights_in, plan, "weights_in")) != tuple(st))):
        raise ValueError("weights_in and weights_out need T tokens and the same strides")
    rc = _lib.gtq_attn_weights(plan.handle, _ptr(packed), int(T), _lay(layout), ctypes.byref(ch),
                               _ptr(q), _ptr(weights_in), _ptr(weights_out), st, _ptr(workspace),
                               _nbytes(workspace), _stream(stream))
    _check(rc, "gtq_attn_weights")


def gtq_evict_workspace(plan: Plan, T: int) -> int:
    """Bytes of the workspace gtq_evict needs for caches of up to T tokens a sequence."""
    return int(_lib.gtq_evict_workspace_bytes(plan.handle, int(T)))


def gtq_evict(plan: Plan, packed, T: int, weights, keep: int, dst, new_lens, workspace, n_first=0,
              n_recent=0, layout=None, dst_layout=None, weights_out=None, kept=None,
              stream=None) -> None:
    """Move the tokens that stay (n_first, n_recent, and the largest weights) into dst.
    weights [batch, kv heads, >= T]; weights_out [batch, kv heads, >= keep]; kept int32
    [batch, kv heads, keep]; new_lens int32 [batch].  stream: None is the legacy default stream,
    not torch's current one."""
    import torch

    c, device = plan.cfg, plan.device
    ev = gtq_eviction(int(keep), int(n_first), int(n_recent))
    ev.weights_dev, ev.w_strides = _ptr(weights), _weights2(weights, plan, "weights")
    if weights_out is not None:
        ev.weights_out_dev = _ptr(weights_out)
        ev.w_out_strides = _weights2(weights_out, plan, "weights_out")
    if weights.shape[2] < T or (weights_out is not None and weights_out.shape[2] < min(keep, T)):
        raise ValueError("weights need T tokens, weights_out min(keep, T)")
    _need(kept, "kept", device, torch.int32)
    if kept is not None and (tuple(kept.shape) != (c.batch, c.n_kv_heads, keep) or not kept.is_contiguous()):
        raise ValueError("kept must be contiguous int32 [batch, kv heads, keep]")
    _lens(new_lens, "new_lens", plan)
    for x, what in ((packed, "packed"), (dst, "dst"), (workspace, "workspace")):
        _need(x, what, device)
    ev.kept_dev = _ptr(kept) or None
    ev.new_lens_dev = _ptr(new_lens)
    rc = _lib.gtq_evict(plan.handle, _ptr(packed), int(T), _lay(layout), ctypes.byref(ev),
                        _ptr(dst), _nbytes(dst), _lay(dst_layout), _ptr(workspace),
                        _nbytes(workspace), _stream(stream))
    _check(rc, "gtq_evict")


def gtq_free(plan: Plan) -> None:
    plan.free()


def gtq_packed_bytes(plan: Plan) -> int:
    return plan.packed_bytes


def gtq_get_bits(plan: Plan, stream=None):
    import numpy as np

    c = plan.cfg
    out = np.zeros((c.batch, c.n_kv_heads, c.head_dim // 2), dtype=np.uint8)
    _check(_lib.gtq_get_bits(plan.handle, out.ctypes.data_as(ctypes.POINTER(ctypes.c_uint8)),
                             _stream(stream)), "gtq_get_bits")
    return out


def gtq_get_energy(plan: Plan, stream=None):
    import numpy as np

    c = plan.cfg
    out = np.zeros((c.batch, c.n_kv_heads, c.head_dim // 2), dtype=np.float64)
    _check(_lib.gtq_get_energy(plan.handle, out.ctypes.data_as(ctypes.POINTER(ctypes.c_double)),
                               _stream(stream)), "gtq_get_energy")
    return out


def gtq_status(plan: Plan) -> int:
    return int(_lib.gtq_status(plan.handle))


def gtq_plan_device_bytes(plan: Plan) -> int:
    return int(_lib.gtq_plan_device_bytes(plan.handle))


def gtq_raise_status(plan: Plan, code: int) -> None:
    _check(_lib.gtq_raise_status(plan.handle, int(code)), "gtq_raise_status")


def gtq_lloyd_max(bits: int):
    import numpy as np

    c = np.zeros(1 << bits)
    t = np.zeros(max(1, (1 << bits) - 1))
    d = ctypes.c_double()
    _check(_lib.gtq_lloyd_max(int(bits), c.ctypes.data_as(ctypes.POINTER(ctypes.c_double)),
                              t.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), ctypes.byref(d)),
           "gtq_lloyd_max")
    return c, t[: (1 << bits) - 1], d.value


def gtq_rotation(m: int, tag: int = TAG_KEY, seed: int = 0):
    import numpy as np

    out = np.zeros((m, m))
    _check(_lib.gtq_rotation(int(seed), int(tag), int(m),
                             out.ctypes.data_as(ctypes.POINTER(ctypes.c_double))), "gtq_rotation")
    return out


def gtq_layout_tile_bytes(k_bits: int, v_bits: int) -> int:
    return int(_lib.gtq_layout_tile_bytes(int(k_bits), int(v_bits)))
