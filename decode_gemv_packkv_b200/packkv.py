"""Python binding of the PackKV C ABI (libpackkv.so): argument marshalling only.

Every function here has the name of the C entry point it calls and forwards
torch tensors as raw device pointers on the current CUDA stream.  No step of
the encoder or of the GEMVs runs in Python or PyTorch: importing this module
raises if the CUDA library is missing, and there is no fallback.

`PackKVCache` owns the device buffers of one cache (allocated with torch) and
the `packkv_cache` struct that points into them.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("PACKKV_LIB") or os.path.join(_HERE, "libpackkv.so")

BLOCK_TOKENS = 128
HEAD_DIM = 128
FORMAT_VERSION = 1

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CAPACITY, ERR_CUDA, ERR_DEVICE = range(6)
DEV_CAPACITY, DEV_NONFINITE, DEV_BAD_RECORD, DEV_TIMEOUT = 0x1, 0x2, 0x4, 0x8
KEY_IDENTITY, KEY_K_SUM, KEY_KV_SUM = 0, 1, 2
UNITS_FOR, UNITS_WIDTH_ONLY = 0, 1      # how the encoder sizes a unit (base = min, or 0)

EXPORTED = [
    "packkv_abi_version", "packkv_cache_struct_size", "packkv_status_string", "packkv_record_bytes_max",
    "packkv_workspace_bytes", "packkv_cache_check", "packkv_cache_reset", "packkv_encode_block",
    "packkv_append_token", "packkv_qk_gemv", "packkv_pv_gemv", "packkv_get_status",
    "packkv_pv_gemv_noalloc", "packkv_attention_workspace_bytes",
    "packkv_attention_decode", "packkv_append_token_masked",
    "packkv_rope_init", "packkv_norm_rope", "packkv_append_norm_rope",
    "packkv_attention_window_workspace_bytes", "packkv_attention_window",
    "packkv_fork_sequences", "packkv_free_blocks", "packkv_compact_workspace_bytes", "packkv_compact",
]

RAGGED_MAX_BATCH = 2048

DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}  # PACKKV_DTYPE_*
ROPE_HALF, ROPE_INTERLEAVED = 0, 1                                # which channels form a pair
ROPE_SCALE_NONE, ROPE_SCALE_LINEAR, ROPE_SCALE_BASE, ROPE_SCALE_PARTS = range(4)


class PackKVError(RuntimeError):
    def __init__(self, call: str, status: int, msg: str):
        super().__init__(f"{call}: {msg} (status {status})")
        self.status = status


class Format(ctypes.Structure):
    _fields_ = [("version", ctypes.c_uint32), ("bits", ctypes.c_uint32), ("block_tokens", ctypes.c_uint32),
                ("group_tokens", ctypes.c_uint32), ("head_dim", ctypes.c_uint32), ("reorder_key", ctypes.c_uint32),
                ("unit_mode", ctypes.c_uint32)]


class CacheStruct(ctypes.Structure):
    _fields_ = [("fmt", Format), ("batch", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("n_blocks", ctypes.c_int32), ("tail_len", ctypes.c_int32),
                ("reserved0", ctypes.c_int32), ("k_arena", ctypes.c_void_p), ("v_arena", ctypes.c_void_p),
                ("arena_bytes", ctypes.c_uint64), ("k_index", ctypes.c_void_p), ("v_index", ctypes.c_void_p),
                ("k_tail", ctypes.c_void_p), ("v_tail", ctypes.c_void_p), ("ctrl", ctypes.c_void_p),
                ("perm", ctypes.c_void_p), ("seq_blocks", ctypes.POINTER(ctypes.c_int32)),
                ("seq_tail", ctypes.POINTER(ctypes.c_int32)), ("block_table", ctypes.c_void_p)]


class RopeStruct(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_uint32), ("rot_dim", ctypes.c_uint32), ("amplitude", ctypes.c_float),
                ("reserved0", ctypes.c_uint32), ("turn", ctypes.c_uint64 * 64)]


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class HeadsStruct(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("eps", ctypes.c_float), ("q", Rows), ("k", Rows), ("v", Rows), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m decode_gemv_packkv_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(CacheStruct)
    vp, i32, i64, u32, sz, f32, f64 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                       ctypes.c_size_t, ctypes.c_float, ctypes.c_double)
    sig = {
        "packkv_abi_version": (u32, []),
        "packkv_cache_struct_size": (sz, []),
        "packkv_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "packkv_record_bytes_max": (sz, [u32]),
        "packkv_workspace_bytes": (sz, [P, i32]),
        "packkv_cache_check": (ctypes.c_int, [P]),
        "packkv_cache_reset": (ctypes.c_int, [P, vp]),
        "packkv_encode_block": (ctypes.c_int, [P, vp, vp, i32, vp]),
        "packkv_append_token": (ctypes.c_int, [P, vp, vp, vp]),
        "packkv_qk_gemv": (ctypes.c_int, [P, vp, i32, f32, vp, i64, vp, sz, vp]),
        "packkv_pv_gemv": (ctypes.c_int, [P, vp, i64, i32, vp, vp, sz, vp]),
        "packkv_get_status": (ctypes.c_int, [P, vp, ctypes.POINTER(u32)]),
        "packkv_pv_gemv_noalloc": (ctypes.c_int, [P, vp, i64, i32, vp, vp]),
        "packkv_attention_workspace_bytes": (sz, [P, i32]),
        "packkv_attention_decode": (ctypes.c_int, [P, vp, i32, f32, vp, vp, sz, vp]),
        "packkv_append_token_masked": (ctypes.c_int, [P, vp, vp, ctypes.POINTER(ctypes.c_uint8), vp]),
        "packkv_rope_init": (ctypes.c_int, [vp, u32, u32, f64, i32, f64, f64, f64, f64, f32]),
        "packkv_norm_rope": (ctypes.c_int, [vp, vp, i32, i32, vp, i64, vp, vp, vp, vp]),
        "packkv_append_norm_rope": (ctypes.c_int, [P, vp, vp, vp, vp, vp]),
        "packkv_attention_window_workspace_bytes": (sz, [P, i32]),
        "packkv_attention_window": (ctypes.c_int, [P, vp, i32, i32, i32, i32, f32, vp, vp, sz, vp]),
        "packkv_fork_sequences": (ctypes.c_int, [P, vp, vp, i32, vp]),
        "packkv_free_blocks": (ctypes.c_int, [P, vp, vp, vp]),
        "packkv_compact_workspace_bytes": (sz, [P]),
        "packkv_compact": (ctypes.c_int, [P, P, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.packkv_cache_struct_size() != ctypes.sizeof(CacheStruct):
        raise ImportError("packkv_cache layout mismatch between libpackkv.so and the binding")
    return lib


_lib = _load()


def _check(call: str, status: int):
    if status != OK:
        raise PackKVError(call, status, _lib.packkv_status_string(status).decode())


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def record_bytes_max(bits: int) -> int:
    return int(_lib.packkv_record_bytes_max(bits))


class PackKVCache:
    """Device buffers + the packkv_cache struct of one layer's packed cache.

    ragged=True gives every sequence its own length (host counters seq_blocks /
    seq_tail in the struct); block_table (int32 [batch, max_blocks], on the device)
    maps each sequence's logical blocks to physical blocks of the index."""

    def __init__(self, batch: int, kv_heads: int, max_blocks: int, bits: int, reorder_key: int = KEY_K_SUM,
                 arena_bytes: int | None = None, keep_perm: bool = False, device="cuda", ragged: bool = False,
                 block_table: torch.Tensor | None = None, unit_mode: int = 0):
        dev = torch.device(device)
        if arena_bytes is None:
            arena_bytes = batch * kv_heads * max_blocks * record_bytes_max(bits)
        arena_bytes = (int(arena_bytes) + 15) // 16 * 16
        self.k_arena = torch.empty(arena_bytes, dtype=torch.uint8, device=dev)
        self.v_arena = torch.empty(arena_bytes, dtype=torch.uint8, device=dev)
        self.k_index = torch.zeros((batch, kv_heads, max_blocks, 2), dtype=torch.int32, device=dev)
        self.v_index = torch.zeros_like(self.k_index)
        self.k_tail = torch.zeros((batch, kv_heads, BLOCK_TOKENS, HEAD_DIM), dtype=torch.float16, device=dev)
        self.v_tail = torch.zeros_like(self.k_tail)
        self.ctrl = torch.zeros(4, dtype=torch.int64, device=dev)
        self.perm = (torch.zeros((batch, kv_heads, max_blocks, BLOCK_TOKENS), dtype=torch.uint8, device=dev)
                     if keep_perm else None)
        self.s = CacheStruct()
        self.s.fmt = Format(FORMAT_VERSION, bits, BLOCK_TOKENS, 32, HEAD_DIM, reorder_key, unit_mode)
        self.s.batch, self.s.kv_heads, self.s.max_blocks = batch, kv_heads, max_blocks
        self.s.n_blocks = self.s.tail_len = 0
        self.s.k_arena, self.s.v_arena = self.k_arena.data_ptr(), self.v_arena.data_ptr()
        self.s.arena_bytes = arena_bytes
        self.s.k_index, self.s.v_index = self.k_index.data_ptr(), self.v_index.data_ptr()
        self.s.k_tail, self.s.v_tail = self.k_tail.data_ptr(), self.v_tail.data_ptr()
        self.s.ctrl = self.ctrl.data_ptr()
        self.s.perm = self.perm.data_ptr() if self.perm is not None else None
        self.ragged = ragged
        if ragged:
            self._seq_blocks = (ctypes.c_int32 * batch)()
            self._seq_tail = (ctypes.c_int32 * batch)()
            self.s.seq_blocks = ctypes.cast(self._seq_blocks, ctypes.POINTER(ctypes.c_int32))
            self.s.seq_tail = ctypes.cast(self._seq_tail, ctypes.POINTER(ctypes.c_int32))
        self.block_table = None
        if block_table is not None:
            bt = block_table.to(device=dev, dtype=torch.int32).contiguous()
            if tuple(bt.shape) != (batch, max_blocks):
                raise ValueError("block_table must be int32 [batch, max_blocks]")
            self.block_table = bt
            self.s.block_table = bt.data_ptr()
        _check("packkv_cache_check", _lib.packkv_cache_check(ctypes.byref(self.s)))
        self._ws = {}

    # host counters live in the struct
    @property
    def n_blocks(self) -> int:
        return self.s.n_blocks

    @property
    def tail_len(self) -> int:
        return self.s.tail_len

    @property
    def tokens(self) -> int:
        """Tokens of the longest sequence (every sequence, for a uniform batch)."""
        if self.ragged:
            return max((self.seq_tokens(b) for b in range(self.batch)), default=0)
        return self.s.n_blocks * BLOCK_TOKENS + self.s.tail_len

    def seq_tokens(self, b: int) -> int:
        if not self.ragged:
            return self.tokens
        return self._seq_blocks[b] * BLOCK_TOKENS + self._seq_tail[b]

    @property
    def seq_blocks(self):
        return list(self._seq_blocks) if self.ragged else [self.s.n_blocks] * self.batch

    @property
    def seq_tail(self):
        return list(self._seq_tail) if self.ragged else [self.s.tail_len] * self.batch

    def set_lengths(self, blocks, tail=0):
        """Sets the host counters: packed blocks and tail tokens of the cache (ints), or of
        every sequence of a ragged one (sequences of ints).  For tokens taken back (drafts
        that were rejected, a sequence that is done) and caches filled from saved buffers;
        no device memory changes, so a longer length must already be there."""
        s = self.s
        if not self.ragged:
            old = s.n_blocks, s.tail_len
            s.n_blocks, s.tail_len = blocks, tail
        else:
            if len(blocks) != s.batch or len(tail) != s.batch:
                raise ValueError("set_lengths needs the blocks and the tail of every sequence")
            old = self._seq_blocks[:], self._seq_tail[:]
            self._seq_blocks[:], self._seq_tail[:] = blocks, tail
        status = _lib.packkv_cache_check(ctypes.byref(s))
        if status != OK:
            if self.ragged:
                self._seq_blocks[:], self._seq_tail[:] = old
            else:
                s.n_blocks, s.tail_len = old
            _check("packkv_cache_check", status)

    @property
    def bits(self) -> int:
        return self.s.fmt.bits

    @property
    def batch(self) -> int:
        return self.s.batch

    @property
    def kv_heads(self) -> int:
        return self.s.kv_heads

    def workspace(self, q_heads: int) -> torch.Tensor:
        """p·V workspace for q_heads (allocated once, reused by every call)."""
        if q_heads not in self._ws:
            n = packkv_workspace_bytes(self, q_heads)
            self._ws[q_heads] = torch.zeros(max(n, 16), dtype=torch.uint8, device=self.k_arena.device)
        return self._ws[q_heads]

    def attention_workspace(self, q_heads: int) -> torch.Tensor:
        """Fused-attention workspace for q_heads (allocated once, reused by every call)."""
        key = ("attn", q_heads)
        if key not in self._ws:
            n = int(_lib.packkv_attention_workspace_bytes(ctypes.byref(self.s), q_heads))
            self._ws[key] = torch.zeros(max(n, 16), dtype=torch.uint8, device=self.k_arena.device)
        return self._ws[key]

    def window_workspace(self, q_heads: int) -> torch.Tensor:
        """Window-attention workspace for q_heads (allocated once, reused by every call)."""
        key = ("window", q_heads)
        if key not in self._ws:
            n = int(_lib.packkv_attention_window_workspace_bytes(ctypes.byref(self.s), q_heads))
            self._ws[key] = torch.zeros(max(n, 16), dtype=torch.uint8, device=self.k_arena.device)
        return self._ws[key]

    def compact_workspace(self) -> torch.Tensor:
        """Workspace of packkv_compact from this cache (allocated once, reused by every call)."""
        if "compact" not in self._ws:
            n = packkv_compact_workspace_bytes(self)
            self._ws["compact"] = torch.empty(max(n, 16), dtype=torch.uint8, device=self.k_arena.device)
        return self._ws["compact"]

    def arena_used(self):
        """(K bytes, V bytes) in use; synchronises."""
        ends = self.ctrl[:2].cpu()
        return int(ends[0]) * 16, int(ends[1]) * 16


# --- the C entry points, same names --------------------------------------------------------
def packkv_workspace_bytes(cache: PackKVCache, q_heads: int) -> int:
    return int(_lib.packkv_workspace_bytes(ctypes.byref(cache.s), q_heads))


def packkv_cache_reset(cache: PackKVCache, stream=None):
    _check("packkv_cache_reset", _lib.packkv_cache_reset(ctypes.byref(cache.s), _stream(stream)))


def packkv_encode_block(cache: PackKVCache, k: torch.Tensor, v: torch.Tensor, n_blocks: int, stream=None):
    """k, v: fp16 [batch, kv_heads, n_blocks*128, 128]."""
    _check_kv(cache, k, v, n_blocks * BLOCK_TOKENS)
    _check("packkv_encode_block", _lib.packkv_encode_block(ctypes.byref(cache.s), _ptr(k), _ptr(v), n_blocks,
                                                           _stream(stream)))


def packkv_append_token(cache: PackKVCache, k: torch.Tensor, v: torch.Tensor, stream=None):
    """k, v: fp16 [batch, kv_heads, 128]."""
    if k.dtype != torch.float16 or v.dtype != torch.float16 or tuple(k.shape) != (cache.batch, cache.kv_heads,
                                                                                   HEAD_DIM) or k.shape != v.shape:
        raise ValueError("k, v must be fp16 [batch, kv_heads, 128]")
    _check("packkv_append_token", _lib.packkv_append_token(ctypes.byref(cache.s), _ptr(k), _ptr(v),
                                                           _stream(stream)))


def packkv_append_token_masked(cache: PackKVCache, k: torch.Tensor, v: torch.Tensor, active, stream=None):
    """Ragged caches: one token for the sequences with active[b] (k, v fp16 [batch, kv_heads, 128])."""
    if k.dtype != torch.float16 or v.dtype != torch.float16 or tuple(k.shape) != (cache.batch, cache.kv_heads,
                                                                                   HEAD_DIM) or k.shape != v.shape:
        raise ValueError("k, v must be fp16 [batch, kv_heads, 128]")
    act = (ctypes.c_uint8 * cache.batch)(*[1 if a else 0 for a in active])
    _check("packkv_append_token_masked", _lib.packkv_append_token_masked(ctypes.byref(cache.s), _ptr(k), _ptr(v),
                                                                         act, _stream(stream)))


def packkv_qk_gemv(cache: PackKVCache, q: torch.Tensor, scale: float, scores: torch.Tensor, stream=None):
    """q: fp16 [batch, q_heads, 128]; scores: fp32 [batch, q_heads, ld] with ld >= tokens, ld % 4 == 0."""
    if q.dtype != torch.float16 or q.dim() != 3 or scores.dtype != torch.float32 or scores.dim() != 3:
        raise ValueError("q must be fp16 [B, Hq, 128] and scores fp32 [B, Hq, ld]")
    _check("packkv_qk_gemv", _lib.packkv_qk_gemv(ctypes.byref(cache.s), _ptr(q), q.shape[1], float(scale),
                                                 _ptr(scores), scores.shape[2], None, 0, _stream(stream)))


def packkv_pv_gemv(cache: PackKVCache, p: torch.Tensor, out: torch.Tensor, ws: torch.Tensor | None = None,
                   stream=None):
    """p: fp32 [batch, q_heads, ld] (storage order); out: fp32 [batch, q_heads, 128]."""
    if p.dtype != torch.float32 or p.dim() != 3 or out.dtype != torch.float32:
        raise ValueError("p must be fp32 [B, Hq, ld], out fp32 [B, Hq, 128]")
    if ws is None:
        ws = cache.workspace(p.shape[1])
    _check("packkv_pv_gemv", _lib.packkv_pv_gemv(ctypes.byref(cache.s), _ptr(p), p.shape[2], p.shape[1],
                                                 _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))


def packkv_pv_gemv_noalloc(cache: PackKVCache, p: torch.Tensor, out: torch.Tensor, stream=None):
    """p·V with the library's own fixed scratch instead of a workspace, for callers that
    cannot allocate device memory.  Raises PackKVError (capacity) if the call needs more
    scratch than PV_NOALLOC_SCRATCH_BYTES; overlapping calls share the scratch."""
    if p.dtype != torch.float32 or p.dim() != 3 or out.dtype != torch.float32:
        raise ValueError("p must be fp32 [B, Hq, ld], out fp32 [B, Hq, 128]")
    _check("packkv_pv_gemv_noalloc", _lib.packkv_pv_gemv_noalloc(ctypes.byref(cache.s), _ptr(p), p.shape[2],
                                                                 p.shape[1], _ptr(out), _stream(stream)))


# size of the library's fixed p·V scratch (PACKKV_PV_NOALLOC_SCRATCH_BYTES in packkv.h)
PV_NOALLOC_SCRATCH_BYTES = 8 << 20


def packkv_attention_decode(cache: PackKVCache, q: torch.Tensor, scale: float, out: torch.Tensor,
                            ws: torch.Tensor | None = None, stream=None):
    """q: fp16 [batch, q_heads, 128]; out: fp32 [batch, q_heads, 128] = softmax(scale q·Kᵀ)·V."""
    if q.dtype != torch.float16 or q.dim() != 3 or out.dtype != torch.float32:
        raise ValueError("q must be fp16 [B, Hq, 128], out fp32 [B, Hq, 128]")
    if ws is None:
        ws = cache.attention_workspace(q.shape[1])
    _check("packkv_attention_decode", _lib.packkv_attention_decode(ctypes.byref(cache.s), _ptr(q), q.shape[1],
                                                                   float(scale), _ptr(out), _ptr(ws), ws.numel(),
                                                                   _stream(stream)))


class Rope:
    """A position rotation: the packkv_rope that packkv_rope_init lays down."""

    def __init__(self, rot_dim: int = HEAD_DIM, layout: int = ROPE_HALF, theta: float = 10000.0,
                 scaling: int = ROPE_SCALE_NONE, factor: float = 1.0, original_tokens: float = 0.0, low: float = 1.0,
                 high: float = 32.0, amplitude: float = 1.0):
        self.s = RopeStruct()
        self.ref = ctypes.addressof(self.s)
        _check("packkv_rope_init", _lib.packkv_rope_init(self.ref, rot_dim, layout, theta, scaling, factor,
                                                         original_tokens, low, high, amplitude))


def _heads(rope, q, k, v, q_weight, k_weight, eps, dims):
    """The packkv_heads of q, k, v: CUDA tensors of `dims` dimensions ([batch, tokens, heads,
    128] or [batch, heads, 128]) and any strides, channels contiguous."""
    some = q if q is not None else k
    if some is None or (k is None) != (v is None):
        raise ValueError("expected q, or k and v, or all three")
    in_ = HeadsStruct()
    if some.dtype not in DTYPES:
        raise ValueError("q, k, v must be fp16, bf16 or fp32")
    in_.dtype = DTYPES[some.dtype]
    in_.eps = -1.0 if eps is None else eps
    if eps is not None and not eps >= 0:
        raise ValueError("eps must be >= 0 (None: no norm)")
    if eps is None and (q_weight is not None or k_weight is not None):
        raise ValueError("weights need eps (a norm)")
    lead = tuple(some.shape[:dims - 2])
    for name, x in (("q", q), ("k", k), ("v", v)):
        if x is None:
            continue
        if not x.is_cuda or x.dim() != dims or x.dtype != some.dtype or x.device != some.device:
            raise ValueError(f"{name} must be a CUDA tensor of {dims} dimensions like the others")
        shape, stride = x.shape, x.stride()
        if tuple(shape[:dims - 2]) != lead or shape[-1] != HEAD_DIM or stride[-1] != 1:
            raise ValueError(f"{name} must end in heads of {HEAD_DIM} contiguous channels, batch and tokens as the others")
        rows = getattr(in_, name)
        rows.data = x.data_ptr()
        rows.batch_stride, rows.head_stride = stride[0], stride[-2]
        rows.token_stride = stride[1] if dims == 4 else 0
    if q is not None:
        in_.q_heads = q.shape[-2]
    if k is not None:
        in_.kv_heads = k.shape[-2]
        if v.shape[-2] != in_.kv_heads:
            raise ValueError("k and v must have the same heads")
    for name, w, x in (("q_weight", q_weight, q), ("k_weight", k_weight, k)):
        if w is None:
            continue
        if (x is None or w.dtype != torch.float32 or tuple(w.shape) != (HEAD_DIM,) or not w.is_contiguous()
                or w.device != some.device):
            raise ValueError(f"{name} must be a contiguous fp32 [{HEAD_DIM}] on the heads' device")
        setattr(in_, name, w.data_ptr())
    return in_, some


def _on_device(t: torch.Tensor, stream):
    """The stream a call for tensors like t goes to: `stream`, or the current one of t's
    device.  The launch itself goes to the current device, which must be t's."""
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return _stream(stream)


def _fp16_out(name, out, shape, device):
    if out is None or out.dtype != torch.float16 or tuple(out.shape) != shape or out.device != device:
        raise ValueError(f"{name} must be fp16 {shape} on the inputs' device")
    return _ptr(out)


def packkv_norm_rope(rope: Rope | None, q, k, v, q_out=None, k_out=None, v_out=None, q_weight=None, k_weight=None,
                     eps: float | None = None, positions: torch.Tensor | None = None, first: int = 0, stream=None):
    """Norm (eps given) and rotation (rope given) of q, k [batch, tokens, heads, 128], v cast,
    into q_out, k_out, v_out: fp16 [batch, heads, tokens, 128].  q, or k and v, may be None.
    Positions: int32 [batch, tokens], or first + t."""
    in_, some = _heads(rope, q, k, v, q_weight, k_weight, eps, 4)
    B, T = some.shape[0], some.shape[1]
    ptrs = [None if x is None else _fp16_out(name, out, (B, x.shape[2], T, HEAD_DIM), some.device)
            for name, x, out in (("q_out", q, q_out), ("k_out", k, k_out), ("v_out", v, v_out))]
    if positions is not None and (positions.dtype != torch.int32 or tuple(positions.shape) != (B, T)
                                  or positions.device != some.device):
        raise ValueError(f"positions must be int32 {(B, T)} on the inputs' device")
    _check("packkv_norm_rope", _lib.packkv_norm_rope(rope.ref if rope is not None else None, ctypes.byref(in_), B, T,
                                                     _ptr(positions), first, *ptrs, _on_device(some, stream)))


def packkv_append_norm_rope(cache: PackKVCache, rope: Rope | None, q, k, v, q_out=None, q_weight=None, k_weight=None,
                            eps: float | None = None, active=None, stream=None):
    """One token per sequence, q, k, v [batch, heads, 128]: norm and rotation at the position
    the cache gives it, k and v appended, q to q_out (fp16 [batch, q_heads, 128]).  active:
    as for packkv_append_token_masked (ragged caches), None for all."""
    in_, some = _heads(rope, q, k, v, q_weight, k_weight, eps, 3)
    if k is None or k.shape[0] != cache.s.batch or k.shape[1] != cache.s.kv_heads or k.device != cache.k_tail.device:
        raise ValueError("k, v must be [batch, kv_heads, 128] on the cache's device")
    qp = None if q is None else _fp16_out("q_out", q_out, tuple(q.shape), some.device)
    act = None
    if active is not None:
        if len(active) != cache.s.batch:
            raise ValueError("active needs an entry for every sequence")
        act = (ctypes.c_uint8 * cache.s.batch)(*[1 if x else 0 for x in active])
    _check("packkv_append_norm_rope", _lib.packkv_append_norm_rope(
        ctypes.byref(cache.s), rope.ref if rope is not None else None, ctypes.byref(in_), act, qp,
        _on_device(some, stream)))


def packkv_attention_window(cache: PackKVCache, q: torch.Tensor, scale: float, out: torch.Tensor, window: int,
                            sinks: int = 0, queries: int = 1, ws: torch.Tensor | None = None, stream=None):
    """Attention of the last `queries` positions over the last `window` tokens and the first
    `sinks`: q fp16 [batch, q_heads, 128] with q_heads = kv_heads * queries * G, row
    (h * queries + s) * G + g; out fp32 of the same shape.  The cache keeps its
    permutations (keep_perm=True) unless it does not reorder."""
    if (q.dtype != torch.float16 or q.dim() != 3 or q.shape[0] != cache.s.batch or q.shape[2] != HEAD_DIM
            or out.dtype != torch.float32 or out.shape != q.shape or q.device != cache.k_tail.device
            or out.device != q.device):
        raise ValueError("q must be fp16 and out fp32 [batch, q_heads, 128], on the cache's device")
    if ws is None:
        ws = cache.window_workspace(q.shape[1])
    _check("packkv_attention_window", _lib.packkv_attention_window(
        ctypes.byref(cache.s), _ptr(q), q.shape[1], queries, window, sinks, scale, _ptr(out), _ptr(ws), ws.numel(),
        _on_device(q, stream)))


def packkv_fork_sequences(cache: PackKVCache, src, dst, stream=None):
    """Sequence dst[i] becomes a copy of sequence src[i] (lists of sequence numbers)."""
    n = len(src)
    if len(dst) != n:
        raise ValueError("src and dst must have the same length")
    arr = ctypes.c_int32 * n
    _check("packkv_fork_sequences", _lib.packkv_fork_sequences(ctypes.byref(cache.s), arr(*src), arr(*dst), n,
                                                               _on_device(cache.k_tail, stream)))


def packkv_free_blocks(cache: PackKVCache, first, count, stream=None):
    """Gives up blocks first[b] .. first[b] + count[b] - 1 of every sequence (lists of ints)."""
    if len(first) != cache.s.batch or len(count) != cache.s.batch:
        raise ValueError("first and count need an entry for every sequence")
    arr = ctypes.c_int32 * cache.s.batch
    _check("packkv_free_blocks", _lib.packkv_free_blocks(ctypes.byref(cache.s), arr(*first), arr(*count),
                                                         _on_device(cache.k_tail, stream)))


def packkv_compact_workspace_bytes(cache: PackKVCache) -> int:
    return int(_lib.packkv_compact_workspace_bytes(ctypes.byref(cache.s)))


def packkv_compact(dst: PackKVCache, src: PackKVCache, ws: torch.Tensor | None = None, stream=None):
    """Copies what src holds into dst, its live records packed from the start of dst's arenas."""
    if dst.k_arena.device != src.k_arena.device:
        raise ValueError("both caches must be on one device")
    if ws is None:
        ws = src.compact_workspace()
    _check("packkv_compact", _lib.packkv_compact(ctypes.byref(dst.s), ctypes.byref(src.s), _ptr(ws), ws.numel(),
                                                 _on_device(src.k_arena, stream)))


def packkv_get_status(cache: PackKVCache, stream=None) -> int:
    """Synchronises the stream; returns the device status bits (and clears them)."""
    bits = ctypes.c_uint32(0)
    _lib.packkv_get_status(ctypes.byref(cache.s), _stream(stream), ctypes.byref(bits))
    return int(bits.value)


def _check_kv(cache, k, v, tokens):
    want = (cache.batch, cache.kv_heads, tokens, HEAD_DIM)
    if k.dtype != torch.float16 or v.dtype != torch.float16 or tuple(k.shape) != want or tuple(v.shape) != want:
        raise ValueError(f"k, v must be fp16 {want}")


def prefill(cache: PackKVCache, k: torch.Tensor, v: torch.Tensor, stream=None):
    """Encodes the full blocks of k, v [B, H, T, 128] and appends the remaining T % 128 tokens."""
    t = k.shape[2]
    nb = t // BLOCK_TOKENS
    if nb:
        packkv_encode_block(cache, k[:, :, :nb * BLOCK_TOKENS].contiguous(), v[:, :, :nb * BLOCK_TOKENS].contiguous(),
                            nb, stream)
    for i in range(nb * BLOCK_TOKENS, t):
        packkv_append_token(cache, k[:, :, i].contiguous(), v[:, :, i].contiguous(), stream)
