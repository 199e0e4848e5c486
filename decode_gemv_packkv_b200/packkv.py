"""Python binding of the PackKV C ABI (libpackkv.so): argument marshalling only.

Every function here has the name of the C entry point it calls and forwards
torch tensors as raw device pointers on the current CUDA stream.  No step of
the encoder or of the GEMVs runs in Python or PyTorch: importing this module
raises if the CUDA library is missing, and there is no fallback.

`PackKVCache` owns the device buffers of one cache (allocated with torch) and
the `packkv_cache` struct that points into them.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import os
import struct

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
_INT_MAX = (1 << 31) - 1

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
        "packkv_append_norm_rope": (ctypes.c_int, [vp, vp, vp, vp, vp, vp]),
        "packkv_attention_window_workspace_bytes": (sz, [P, i32]),
        "packkv_attention_window": (ctypes.c_int, [vp, vp, i32, i32, i32, i32, f32, vp, vp, sz, vp]),
        "packkv_fork_sequences": (ctypes.c_int, [vp, vp, vp, i32, vp]),
        "packkv_free_blocks": (ctypes.c_int, [vp, vp, vp, vp]),
        "packkv_compact_workspace_bytes": (sz, [P]),
        "packkv_compact": (ctypes.c_int, [vp, vp, vp, sz, vp]),
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
        self.addr = ctypes.addressof(self.s)
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
        return self._seq_blocks[:] if self.ragged else [self.s.n_blocks] * self.batch

    @property
    def seq_tail(self):
        return self._seq_tail[:] if self.ragged else [self.s.tail_len] * self.batch

    def set_lengths(self, blocks, tail=0):
        """Sets the host counters: packed blocks and tail tokens of the cache (ints), or of
        every sequence of a ragged one (sequences of ints).  For tokens taken back (drafts
        that were rejected, a sequence that is done) and caches filled from saved buffers;
        no device memory changes, so a longer length must already be there."""
        s = self.s
        if self.ragged and (len(blocks) != s.batch or len(tail) != s.batch):
            raise ValueError("set_lengths needs the blocks and the tail of every sequence")
        old = (self._seq_blocks[:], self._seq_tail[:]) if self.ragged else (s.n_blocks, s.tail_len)
        try:
            self._put_lengths(blocks, tail)
            _check("packkv_cache_check", _lib.packkv_cache_check(ctypes.byref(s)))
        except Exception:
            self._put_lengths(*old)
            raise

    def _put_lengths(self, blocks, tail):
        if self.ragged:
            self._seq_blocks[:], self._seq_tail[:] = blocks, tail
        else:
            self.s.n_blocks, self.s.tail_len = blocks, tail

    @property
    def bits(self) -> int:
        return self.s.fmt.bits

    @property
    def batch(self) -> int:
        return self.s.batch

    @property
    def kv_heads(self) -> int:
        return self.s.kv_heads

    def _workspace(self, key, nbytes, stream):
        """The cache's workspace `key` (a tuple) on a stream (None: the current one), allocated
        at its first use.  No call needs it initialised.  Every stream has its own, allocated
        on that stream: calls on one stream take their turns, so they share it, and no other
        stream's work (that of an earlier user of the memory among it) can still write to it."""
        dev = self.k_arena.device
        if stream is None:
            handle = torch._C._cuda_getCurrentRawStream(dev.index) if dev.type == "cuda" else 0
        else:
            handle = stream.cuda_stream
        key += (handle,)
        ws = self._ws.get(key)
        if ws is None:
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                ws = torch.empty(max(nbytes(), 16), dtype=torch.uint8, device=dev)
            self._ws[key] = ws
        return ws

    def workspace(self, q_heads: int, stream=None) -> torch.Tensor:
        """p·V workspace for q_heads: one per stream (None: the current one), allocated once and
        reused by every call there.  Graphs captured on one stream share it: replays that
        overlap in time need workspaces of their own (the calls' ws)."""
        return self._workspace(("pv", q_heads), lambda: packkv_workspace_bytes(self, q_heads), stream)

    def attention_workspace(self, q_heads: int, stream=None) -> torch.Tensor:
        """Fused-attention workspace for q_heads (one per stream, as workspace())."""
        return self._workspace(("attn", q_heads), lambda: int(
            _lib.packkv_attention_workspace_bytes(ctypes.byref(self.s), q_heads)), stream)

    def window_workspace(self, q_heads: int, stream=None) -> torch.Tensor:
        """Window-attention workspace for q_heads (one per stream, as workspace())."""
        return self._workspace(("window", q_heads), lambda: int(
            _lib.packkv_attention_window_workspace_bytes(ctypes.byref(self.s), q_heads)), stream)

    def compact_workspace(self, stream=None) -> torch.Tensor:
        """Workspace of packkv_compact from this cache (one per stream, as workspace())."""
        return self._workspace(("compact",), lambda: packkv_compact_workspace_bytes(self), stream)

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
        ws = cache.workspace(p.shape[1], stream)
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
        ws = cache.attention_workspace(q.shape[1], stream)
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


# packkv_heads: dtype, q_heads, kv_heads, eps, the rows of q, k, v, q_weight, k_weight
_HEADS = struct.Struct("=iiif QqqqQqqqQqqq QQ")


def _heads(q, k, v, q_weight, k_weight, eps, dims):
    """The packkv_heads of q, k, v ([batch, tokens, heads, 128] or [batch, heads, 128] CUDA
    tensors of any strides, channels contiguous), and the first of them."""
    like = q if q is not None else k
    if like is None or (k is None) != (v is None):
        raise ValueError("expected q, or k and v, or all three")
    kind, at, shape = like.dtype, like.get_device(), like.shape
    dtype, lead = DTYPES.get(kind), shape[:-2]
    if dtype is None or at < 0:
        raise ValueError("q, k, v must be fp16, bf16 or fp32 CUDA tensors")
    heads, rows = [0, 0, 0], []
    for i, x in enumerate((q, k, v)):
        if x is None:
            rows += (0, 0, 0, 0)
            continue
        stride = x.stride()
        if x is not like:
            shape = x.shape
            if shape[:-2] != lead or x.dtype != kind or x.get_device() != at:
                raise ValueError("q, k, v must have the same batch, tokens, dtype and device")
        if len(shape) != dims or shape[-1] != HEAD_DIM or stride[-1] != 1:
            raise ValueError(f"q, k, v must have {dims} dimensions, the last one {HEAD_DIM} contiguous channels")
        heads[i] = shape[-2]
        rows += (x.data_ptr(), stride[0], stride[1] if dims == 4 else 0, stride[-2])
    if heads[1] != heads[2]:
        raise ValueError("k and v must have the same heads")
    if eps is None:
        if q_weight is not None or k_weight is not None:
            raise ValueError("weights need eps (a norm)")
        return _HEADS.pack(dtype, heads[0], heads[1], -1.0, *rows, 0, 0), like
    if not eps >= 0:
        raise ValueError("eps must be >= 0 (None: no norm)")
    weights = []
    for w, x in ((q_weight, q), (k_weight, k)):
        if w is None:
            weights.append(0)
            continue
        if x is None or w.dtype != torch.float32 or w.shape != (HEAD_DIM,) or w.stride(0) != 1 or w.get_device() != at:
            raise ValueError(f"a weight must be a contiguous fp32 [{HEAD_DIM}] on the device of heads that are given")
        weights.append(w.data_ptr())
    return _HEADS.pack(dtype, heads[0], heads[1], eps, *rows, *weights), like


def _stream_of(t: torch.Tensor, stream):
    """The stream a call for tensors like t goes to: `stream`, or the current one.  The
    launch goes to the current device, which must be t's."""
    at = t.get_device()
    if at != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    # the raw handle; torch.cuda.current_stream() would wrap it in an object first
    return torch._C._cuda_getCurrentRawStream(at) if stream is None else stream.cuda_stream


def _out_ptr(name, out, dtype, shape, at):
    """A contiguous output's address."""
    if out is None or out.dtype != dtype or out.shape != shape or out.get_device() != at or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {tuple(shape)} on the inputs' device")
    return out.data_ptr()


def _int32s(values):
    """A host int32 array and its address (keep the array until the call has returned)."""
    a = array.array("i", values)
    return a, a.buffer_info()[0]


def packkv_norm_rope(rope: Rope | None, q, k, v, q_out=None, k_out=None, v_out=None, q_weight=None, k_weight=None,
                     eps: float | None = None, positions: torch.Tensor | None = None, first: int = 0, stream=None):
    """Norm (eps given) and rotation (rope given) of q, k [batch, tokens, heads, 128], v cast,
    into q_out, k_out, v_out: fp16 [batch, heads, tokens, 128].  q, or k and v, may be None.
    Positions: int32 [batch, tokens], or first + t."""
    heads, like = _heads(q, k, v, q_weight, k_weight, eps, 4)
    B, T = like.shape[0], like.shape[1]
    at = like.get_device()
    ptrs = [None if x is None else _out_ptr(name, out, torch.float16, (B, x.shape[2], T, HEAD_DIM), at)
            for name, x, out in (("q_out", q, q_out), ("k_out", k, k_out), ("v_out", v, v_out))]
    pos = None
    if positions is not None:
        if (positions.dtype != torch.int32 or positions.shape != (B, T) or positions.get_device() != at
                or not positions.is_contiguous()):
            raise ValueError(f"positions must be a contiguous int32 {(B, T)} on the inputs' device")
        pos = positions.data_ptr()
    if B == 0 or T == 0:  # nothing to do (and such tensors have no address)
        return
    status = _lib.packkv_norm_rope(None if rope is None else rope.ref, heads, B, T, pos, first, *ptrs,
                                   _stream_of(like, stream))
    if status:
        _check("packkv_norm_rope", status)


def packkv_append_norm_rope(cache: PackKVCache, rope: Rope | None, q, k, v, q_out=None, q_weight=None, k_weight=None,
                            eps: float | None = None, active=None, stream=None):
    """One token per sequence, q, k, v [batch, heads, 128]: norm and rotation at the position
    the cache gives it, k and v appended, q to q_out (fp16 [batch, q_heads, 128]).  active:
    as for packkv_append_token_masked (ragged caches), None for all."""
    heads, like = _heads(q, k, v, q_weight, k_weight, eps, 3)
    at, batch = like.get_device(), cache.s.batch
    if k is None or k.shape[0] != batch or k.shape[1] != cache.s.kv_heads or at != cache.k_tail.get_device():
        raise ValueError("k, v must be [batch, kv_heads, 128] on the cache's device")
    qp = None if q is None else _out_ptr("q_out", q_out, torch.float16, q.shape, at)
    if active is not None:
        active = bytes(map(bool, active))
        if len(active) != batch:
            raise ValueError("active needs an entry for every sequence")
    status = _lib.packkv_append_norm_rope(cache.addr, None if rope is None else rope.ref, heads, active, qp,
                                          _stream_of(like, stream))
    if status:
        _check("packkv_append_norm_rope", status)


def packkv_attention_window(cache: PackKVCache, q: torch.Tensor, scale: float, out: torch.Tensor, window: int,
                            sinks: int = 0, queries: int = 1, ws: torch.Tensor | None = None, stream=None):
    """Attention of the last `queries` positions over the last `window` tokens and the first
    `sinks`: q fp16 [batch, q_heads, 128] with q_heads = kv_heads * queries * G, row
    (h * queries + s) * G + g; out fp32 of the same shape.  The cache keeps its
    permutations (keep_perm=True) unless it does not reorder."""
    shape, at = q.shape, cache.k_tail.get_device()
    if len(shape) != 3 or shape[0] != cache.s.batch or shape[2] != HEAD_DIM:
        raise ValueError("q must be fp16 [batch, q_heads, 128] on the cache's device")
    handle = _stream_of(q, stream)
    if ws is None:
        ws = cache._ws.get(("window", shape[1], handle))
        if ws is None:
            ws = cache.window_workspace(shape[1], stream)
    # no sequence has more than 2^31 tokens: larger limits mean the same
    window, sinks = min(window, _INT_MAX), min(sinks, _INT_MAX)
    status = _lib.packkv_attention_window(cache.addr, _out_ptr("q", q, torch.float16, shape, at), shape[1], queries,
                                          window, sinks, float(scale), _out_ptr("out", out, torch.float32, shape, at),
                                          _ws_ptr(ws, at), ws.nbytes, handle)
    if status:
        _check("packkv_attention_window", status)


def _ws_ptr(ws, at):
    if ws.get_device() != at or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous tensor on the cache's device")
    return ws.data_ptr()


def packkv_fork_sequences(cache: PackKVCache, src, dst, stream=None):
    """Sequence dst[i] becomes a copy of sequence src[i] (lists of sequence numbers)."""
    a, ap = _int32s(src)
    b, bp = _int32s(dst)
    if len(a) != len(b):
        raise ValueError("src and dst must have the same length")
    status = _lib.packkv_fork_sequences(cache.addr, ap, bp, len(a), _stream_of(cache.k_tail, stream))
    if status:
        _check("packkv_fork_sequences", status)


def packkv_free_blocks(cache: PackKVCache, first, count, stream=None):
    """Gives up blocks first[b] .. first[b] + count[b] - 1 of every sequence (lists of ints)."""
    a, ap = _int32s(first)
    b, bp = _int32s(count)
    if len(a) != cache.s.batch or len(b) != cache.s.batch:
        raise ValueError("first and count need an entry for every sequence")
    status = _lib.packkv_free_blocks(cache.addr, ap, bp, _stream_of(cache.k_tail, stream))
    if status:
        _check("packkv_free_blocks", status)


def packkv_compact_workspace_bytes(cache: PackKVCache) -> int:
    return int(_lib.packkv_compact_workspace_bytes(ctypes.byref(cache.s)))


def packkv_compact(dst: PackKVCache, src: PackKVCache, ws: torch.Tensor | None = None, stream=None):
    """Copies what src holds into dst, its live records packed from the start of dst's arenas."""
    at = src.k_arena.get_device()
    if dst.k_arena.get_device() != at:
        raise ValueError("both caches must be on one device")
    handle = _stream_of(src.k_arena, stream)
    if ws is None:
        ws = src._ws.get(("compact", handle))
        if ws is None:
            ws = src.compact_workspace(stream)
    status = _lib.packkv_compact(dst.addr, src.addr, _ws_ptr(ws, at), ws.nbytes, handle)
    if status:
        _check("packkv_compact", status)


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
