"""Refusals of the head, window and block calls, on the host before any launch (no GPU)."""
import ctypes
import math

import pytest

from test_abi_cpu import _fake_cache


@pytest.fixture(scope="module")
def pk():
    from decode_gemv_packkv_b200 import build
    build.build()
    from decode_gemv_packkv_b200 import packkv
    return packkv


X = ctypes.c_void_p(0x20000000)
ODD = ctypes.c_void_p(0x20000004)


def test_rope_init(pk):
    r = pk.Rope(128, pk.ROPE_HALF, 10000.0)
    assert abs(r.s.turn[0] / 2.0 ** 64 - 1 / (2 * math.pi)) < 2.0 ** -52
    assert abs(r.s.turn[32] / 2.0 ** 64 - 0.01 / (2 * math.pi)) < 2.0 ** -52
    for bad in (dict(rot_dim=3), dict(rot_dim=130), dict(layout=2), dict(theta=1.0), dict(theta=float("nan")),
                dict(scaling=4), dict(scaling=1, factor=0.0), dict(scaling=1, factor=float("inf")),
                dict(scaling=3, factor=2.0, original_tokens=0.0), dict(amplitude=float("nan")),
                dict(scaling=3, factor=2.0, original_tokens=10.0, low=4.0, high=4.0),
                dict(scaling=1, factor=0.1)):          # frequencies above half a turn per position
        with pytest.raises(pk.PackKVError) as e:
            pk.Rope(**bad)
        assert e.value.status == pk.ERR_INVALID_ARG, bad


def _heads(pk, **over):
    """A packkv_heads of fp16 rows (q 4 heads, k and v 2), fields replaced by name."""
    f = dict(dtype=0, q_heads=4, kv_heads=2, eps=-1.0, q=0x30000000, k=0x30000000, v=0x30000000, q_weight=0, k_weight=0)
    f.update(over)
    rows = [x for name in "qkv" for x in (f[name], 1024, 1024, 128)]
    return pk._HEADS.pack(f["dtype"], f["q_heads"], f["kv_heads"], f["eps"], *rows, f["q_weight"], f["k_weight"])


def test_norm_rope_refusals(pk):
    call = pk._lib.packkv_norm_rope

    def run(h, batch=1, tokens=1, positions=None, q=X, k=X, v=X, rope=None):
        return call(rope, h, batch, tokens, positions, 0, q, k, v, None)

    bad = pk.ERR_INVALID_ARG
    assert run(_heads(pk), batch=0) == pk.OK and run(_heads(pk), tokens=0) == pk.OK
    assert run(_heads(pk, dtype=3)) == bad
    assert run(_heads(pk, q_heads=0)) == bad                      # q without heads
    assert run(_heads(pk, q=0)) == bad                            # heads without q
    assert run(_heads(pk, k=0)) == bad                            # v without k
    assert run(_heads(pk, q=0, k=0, v=0, q_heads=0)) == bad       # nothing
    assert run(_heads(pk, q=0x30000001)) == bad
    assert run(_heads(pk, dtype=2, q=0x30000002)) == bad
    assert run(_heads(pk, eps=float("nan"))) == bad
    assert run(_heads(pk, q_weight=0x30000000)) == bad            # weight without a norm
    assert run(_heads(pk, kv_heads=0)) == bad
    assert run(_heads(pk), q=ODD) == bad and run(_heads(pk), k=None) == bad
    assert run(_heads(pk), positions=ctypes.c_void_p(0x30000002)) == bad
    assert run(_heads(pk), batch=-1) == bad and run(_heads(pk), batch=1 << 16, tokens=1 << 16) == bad
    r = pk.RopeStruct()
    r.rot_dim = 5
    assert run(_heads(pk), rope=ctypes.addressof(r), batch=0) == bad
    assert call(None, None, 1, 1, None, 0, X, X, X, None) == bad


def test_append_norm_rope_refusals(pk):
    call = pk._lib.packkv_append_norm_rope
    s = _fake_cache(pk)
    act = (ctypes.c_uint8 * 2)(1, 1)
    assert call(ctypes.addressof(s), None, (_heads(pk, kv_heads=3)), None, X, None) == pk.ERR_INVALID_ARG
    assert call(ctypes.addressof(s), None, (_heads(pk, k=0, v=0)), None, X, None) == pk.ERR_INVALID_ARG
    assert call(ctypes.addressof(s), None, (_heads(pk)), None, ODD, None) == pk.ERR_INVALID_ARG
    assert call(ctypes.addressof(s), None, (_heads(pk)), act, X, None) == pk.ERR_UNSUPPORTED
    s = _fake_cache(pk, n_blocks=4, tail_len=127)
    assert call(ctypes.addressof(s), None, (_heads(pk)), None, X, None) == pk.ERR_CAPACITY
    assert s.n_blocks == 4 and s.tail_len == 127
    P = ctypes.POINTER(ctypes.c_int32)
    blocks, tail = (ctypes.c_int32 * 2)(4, 1), (ctypes.c_int32 * 2)(127, 5)
    s = _fake_cache(pk)
    s.seq_blocks, s.seq_tail = ctypes.cast(blocks, P), ctypes.cast(tail, P)
    assert call(ctypes.addressof(s), None, (_heads(pk)), None, X, None) == pk.ERR_CAPACITY
    none = (ctypes.c_uint8 * 2)(0, 0)
    assert call(ctypes.addressof(s), None, (_heads(pk)), none, X, None) == pk.OK   # no token: nothing runs
    assert list(blocks) == [4, 1] and list(tail) == [127, 5]


def test_window_refusals(pk):
    call = pk._lib.packkv_attention_window

    def run(s, q=X, q_heads=4, queries=1, window=8, sinks=0, out=X):
        return call(ctypes.addressof(s), q, q_heads, queries, window, sinks, 1.0, out, X, 1 << 40, None)

    def cache(**over):
        s = _fake_cache(pk, n_blocks=2, **over)
        s.perm = 0x11000000
        return s

    bad = pk.ERR_INVALID_ARG
    assert run(cache(), q_heads=3) == bad
    assert run(cache(), q_heads=6) == pk.ERR_UNSUPPORTED
    assert run(cache(), q_heads=256) == pk.ERR_UNSUPPORTED
    assert run(cache(), queries=0) == bad and run(cache(), q_heads=8, queries=3) == bad
    assert run(cache(), queries=4) == bad                          # more positions than rows
    assert run(cache(), window=0) == bad and run(cache(), sinks=-1) == bad
    assert run(cache(), q=ODD) == bad and run(cache(), out=None) == bad
    s = cache()
    s.perm = 0x11000004
    assert run(s) == bad
    s.perm = None
    assert run(s) == bad                                           # reordered, no permutations
    big = _fake_cache(pk, batch=1 << 14, kv_heads=1 << 10, max_blocks=2000, n_blocks=2000)
    big.perm = 0x11000000
    assert run(big, q_heads=64 << 10, window=1 << 30) == pk.ERR_UNSUPPORTED  # 2^41 items


def test_block_call_refusals(pk):
    lib, bad = pk._lib, pk.ERR_INVALID_ARG
    A = ctypes.c_int32 * 2

    def fork(src, dst, s=None):
        s = s or _fake_cache(pk, n_blocks=2)
        n = len(src)
        return lib.packkv_fork_sequences(ctypes.addressof(s), (ctypes.c_int32 * n)(*src), (ctypes.c_int32 * n)(*dst), n, None)

    assert fork([], []) == pk.OK
    assert fork([0], [0]) == bad and fork([0, 1], [1, 0]) == bad and fork([0, 0], [1, 1]) == bad
    assert fork([2], [0]) == bad and fork([-1], [0]) == bad and fork([0], [2]) == bad
    assert fork([0, 0, 0], [1, 1, 1]) == bad                       # more pairs than sequences
    s = _fake_cache(pk, batch=pk.RAGGED_MAX_BATCH + 1)
    assert fork([0], [1], s) == pk.ERR_UNSUPPORTED
    s = _fake_cache(pk, n_blocks=2)
    assert lib.packkv_fork_sequences(ctypes.addressof(s), None, None, 1, None) == bad

    def free(first, count):
        return lib.packkv_free_blocks(ctypes.addressof(s), A(*first), A(*count), None)

    assert free([0, 0], [0, 0]) == pk.OK
    assert free([0, 0], [3, 0]) == bad and free([2, 0], [1, 0]) == bad and free([-1, 0], [1, 0]) == bad
    assert free([0, 0], [0, -1]) == bad and free([1 << 30, 0], [(1 << 31) - 1, 0]) == bad
    assert lib.packkv_free_blocks(ctypes.addressof(s), None, A(0, 0), None) == bad

    def other(**over):
        d = _fake_cache(pk, **over)
        for i, f in enumerate(["k_arena", "v_arena", "k_index", "v_index", "k_tail", "v_tail", "ctrl"]):
            setattr(d, f, 0x50000000 + i * 0x100000)
        return d

    need = lib.packkv_compact_workspace_bytes(ctypes.byref(s))
    assert need > 0

    def compact(d, ws=X, size=None, src=s):
        return lib.packkv_compact(ctypes.addressof(d), ctypes.addressof(src), ws, need if size is None else size, None)

    assert compact(other(bits=3)) == bad and compact(other(batch=1)) == bad and compact(other(kv_heads=1)) == bad
    assert compact(other(max_blocks=1)) == pk.ERR_CAPACITY
    assert compact(other(), ws=ODD) == bad and compact(other(), size=need - 16) == bad and compact(other(), ws=None) == bad
    assert compact(s) == bad                                       # itself
    d = other()
    d.v_tail = s.k_arena + 4096
    assert compact(d) == bad                                       # an overlap
    d = other()
    d.perm = 0x60000000
    assert compact(d) == bad                                       # permutations that src does not keep
    P = ctypes.POINTER(ctypes.c_int32)
    d = other()
    blocks, tail = A(0, 0), A(0, 0)
    d.seq_blocks, d.seq_tail = ctypes.cast(blocks, P), ctypes.cast(tail, P)
    assert compact(d) == bad                                       # ragged into uniform
