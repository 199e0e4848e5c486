"""Forking, freeing and compacting the cache's blocks, bit for bit, and the operators run
together as a serving loop runs them."""
import numpy as np
import pytest
import torch

import oracle as O
from decode_gemv_packkv_b200 import synth
from parity_util import gpu_records, to_dev

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(128.0)
FREED = 0xFFFFFFFF


@pytest.fixture(scope="module")
def pk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_gemv_packkv_b200 import packkv
    return packkv


def _filled(pk, B, H, mb, bits, tokens, seed, structured=True, **kw):
    T = max(tokens)
    k, v, _ = synth.small_case(seed, B, H, 1, T, structured=structured)
    cache = pk.PackKVCache(B, H, mb, bits, ragged=True, keep_perm=True, **kw)
    nb = [t // 128 for t in tokens]
    if max(nb):
        pk.packkv_encode_block(cache, to_dev(k[:, :, :max(nb) * 128]), to_dev(v[:, :, :max(nb) * 128]), max(nb))
    for b, t in enumerate(tokens):
        cache.k_tail[b, :, :t % 128] = to_dev(k[b, :, nb[b] * 128:t])
        cache.v_tail[b, :, :t % 128] = to_dev(v[b, :, nb[b] * 128:t])
    cache.set_lengths(nb, [t % 128 for t in tokens])
    return cache


def _snapshot(cache):
    return {n: getattr(cache, n).clone() for n in ("k_index", "v_index", "perm", "k_tail", "v_tail", "ctrl")}


def _check_compacted(pk, dst, src, physical=lambda b, j: (b, j), dst_physical=lambda b, j: (b, j)):
    for which in ("k", "v"):
        arena, index = gpu_records(src, which)
        entries, want = O.compacted(index, arena.tobytes(), src.seq_blocks, physical)
        got_arena, got_index = gpu_records(dst, which)
        for (b, h, j), entry in entries.items():
            rb, jb = dst_physical(b, j)
            assert tuple(int(x) for x in got_index[rb, h, jb]) == entry, (which, b, h, j)
        assert int(dst.ctrl[0 if which == "k" else 1]) * 16 == len(want)
        assert got_arena[:len(want)].tobytes() == want
    assert dst.seq_blocks == src.seq_blocks and dst.seq_tail == src.seq_tail
    for b in range(src.batch):
        t = src.seq_tail[b]
        assert torch.equal(dst.k_tail[b, :, :t], src.k_tail[b, :, :t])
        assert torch.equal(dst.v_tail[b, :, :t], src.v_tail[b, :, :t])
        for j in range(src.seq_blocks[b]):
            (rb, jb), (sb, sj) = dst_physical(b, j), physical(b, j)
            assert torch.equal(dst.perm[rb, :, jb], src.perm[sb, :, sj])
    assert pk.packkv_get_status(dst) == 0


@pytest.mark.parametrize("heads", [1, 3])
def test_fork(pk, heads):
    cache = _filled(pk, 5, heads, 6, 4, [700, 130, 0, 256, 90], 3)
    before = _snapshot(cache)
    pk.packkv_fork_sequences(cache, [0, 3, 0], [1, 2, 4])
    assert cache.seq_blocks == [5, 5, 2, 2, 5] and cache.seq_tail == [60, 60, 0, 0, 60]
    for src, dst in ((0, 1), (3, 2), (0, 4)):
        n, t = cache.seq_blocks[src], cache.seq_tail[src]
        for name in ("k_index", "v_index", "perm"):
            x = getattr(cache, name)
            assert torch.equal(x[dst, :, :n], before[name][src, :, :n])
            assert torch.equal(x[dst, :, n:], before[name][dst, :, n:])      # behind: left as it was
        for name in ("k_tail", "v_tail"):
            x = getattr(cache, name)
            assert torch.equal(x[dst, :, :t], before[name][src, :, :t])
            assert torch.equal(x[dst, :, t:], before[name][dst, :, t:])
    for b in (0, 3):
        for name in ("k_index", "v_index", "perm", "k_tail", "v_tail"):
            assert torch.equal(getattr(cache, name)[b], before[name][b])
    assert torch.equal(cache.ctrl, before["ctrl"])


def test_fork_uniform_and_through_a_table(pk):
    k, v, _ = synth.small_case(5, 3, 2, 1, 300)
    cache = pk.PackKVCache(3, 2, 3, 3, keep_perm=True)
    pk.prefill(cache, to_dev(k), to_dev(v))
    pk.packkv_fork_sequences(cache, [2], [0])
    assert torch.equal(cache.k_index[0, :, :2], cache.k_index[2, :, :2])
    assert torch.equal(cache.v_tail[0, :, :44], cache.v_tail[2, :, :44])
    table = torch.tensor([[0, 1, 2], [5, 4, 3], [8, 6, 7]], dtype=torch.int32)
    cache = pk.PackKVCache(3, 2, 3, 3, keep_perm=True, block_table=table)
    pk.packkv_encode_block(cache, to_dev(k[:, :, :256]), to_dev(v[:, :, :256]), 2)
    pk.packkv_fork_sequences(cache, [1], [2])
    for j in range(2):  # logical block j of sequence 1 is (1, 2 - j), of sequence 2 (2, (2, 0)[j])
        assert torch.equal(cache.k_index[2, :, (2, 0)[j]], cache.k_index[1, :, 2 - j])
        assert torch.equal(cache.perm[2, :, (2, 0)[j]], cache.perm[1, :, 2 - j])


def test_free(pk):
    cache = _filled(pk, 3, 2, 5, 2, [640, 300, 50], 4)
    before = _snapshot(cache)
    pk.packkv_free_blocks(cache, [1, 0, 0], [3, 2, 0])
    for name in ("k_index", "v_index"):
        want = before[name].clone()
        want[0, :, 1:4] = torch.tensor([-1, 0], dtype=torch.int32)
        want[1, :, 0:2] = torch.tensor([-1, 0], dtype=torch.int32)
        assert torch.equal(getattr(cache, name), want)
    assert cache.seq_blocks == [5, 2, 0]
    for name in ("perm", "k_tail", "v_tail", "ctrl"):
        assert torch.equal(getattr(cache, name), before[name])


@pytest.mark.parametrize("bits,structured", [(2, True), (3, False), (4, True)])
def test_compact(pk, bits, structured):
    src = _filled(pk, 4, 3, 9, bits, [1000, 40, 513, 1152], 20 + bits, structured)
    pk.packkv_free_blocks(src, [2, 0, 1, 0], [3, 0, 2, 9])
    dst = pk.PackKVCache(4, 3, 12, bits, ragged=True, keep_perm=True)
    pk.packkv_compact(dst, src)
    _check_compacted(pk, dst, src)
    assert dst.arena_used()[0] < src.arena_used()[0]


def test_compact_shared_records(pk):
    """Forked sequences keep sharing their records, freed ones on one side included."""
    src = _filled(pk, 4, 2, 8, 4, [900, 10, 10, 400], 7)
    pk.packkv_fork_sequences(src, [0, 0], [1, 2])
    pk.packkv_free_blocks(src, [0, 3, 0, 0], [4, 1, 0, 0])
    dst = pk.PackKVCache(4, 2, 8, 4, ragged=True, keep_perm=True)
    pk.packkv_compact(dst, src)
    _check_compacted(pk, dst, src)
    assert torch.equal(dst.k_index[0, :, 4:7], dst.k_index[2, :, 4:7])
    again = pk.PackKVCache(4, 2, 8, 4, ragged=True, keep_perm=True)  # a compacted cache stays as it is
    pk.packkv_compact(again, dst)
    n = dst.arena_used()
    assert again.arena_used() == n and torch.equal(again.k_arena[:n[0]], dst.k_arena[:n[0]])


def test_compact_empty_uniform_and_tables(pk):
    src = pk.PackKVCache(2, 2, 3, 4, ragged=True, keep_perm=True)
    dst = pk.PackKVCache(2, 2, 3, 4, ragged=True, keep_perm=True)
    dst.ctrl[0] = 5
    pk.packkv_compact(dst, src)
    assert dst.arena_used() == (0, 0) and dst.seq_blocks == [0, 0]
    k, v, _ = synth.small_case(5, 2, 2, 1, 300)
    src = pk.PackKVCache(2, 2, 3, 3)
    pk.prefill(src, to_dev(k), to_dev(v))
    dst = pk.PackKVCache(2, 2, 2, 3)
    pk.packkv_compact(dst, src)
    assert (dst.n_blocks, dst.tail_len) == (2, 44)
    assert torch.equal(dst.k_index, src.k_index[:, :, :2])
    n = src.arena_used()[0]
    assert torch.equal(dst.k_arena[:n], src.k_arena[:n])
    table = np.array([[2, 1, 0], [5, 3, 4]], np.int32)
    a = _filled(pk, 2, 2, 3, 3, [384, 256], 9, block_table=torch.from_numpy(table))
    b = pk.PackKVCache(2, 2, 3, 3, ragged=True, keep_perm=True)
    pk.packkv_compact(b, a)
    _check_compacted(pk, b, a, lambda s, j: divmod(int(table[s, j]), 3))
    c = pk.PackKVCache(2, 2, 3, 3, ragged=True, keep_perm=True, block_table=torch.from_numpy(table))
    pk.packkv_compact(c, b)
    _check_compacted(pk, c, b, dst_physical=lambda s, j: divmod(int(table[s, j]), 3))


def test_compact_capacity_and_bad_entries(pk):
    src = _filled(pk, 2, 2, 4, 4, [512, 512], 2, structured=False)
    raw = pk.record_bytes_max(4)
    small = pk.PackKVCache(2, 2, 4, 4, ragged=True, keep_perm=True, arena_bytes=15 * raw)
    pk.packkv_compact(small, src)
    assert pk.packkv_get_status(small) & pk.DEV_CAPACITY
    assert small.arena_used() == (0, 0) and torch.all(small.k_index[..., 0] == -1)
    src.k_index[0, 1, 2, 1] = 7            # a length no record has
    src.v_index[1, 0, 0, 0] = 1 << 30      # past the arena
    src.k_index[1, 1, 3, 0] += 1           # overlaps its neighbours' slot with another start
    dst = pk.PackKVCache(2, 2, 4, 4, ragged=True, keep_perm=True)
    pk.packkv_compact(dst, src)
    assert pk.packkv_get_status(dst) == pk.DEV_BAD_RECORD
    assert dst.k_index[0, 1, 2].tolist() == [-1, 0] and dst.v_index[1, 0, 0].tolist() == [-1, 0]


def test_many_tiles(pk):
    """More entries than one look-back tile, most of them short sequences."""
    B = 70                                   # past the small plans of 64 sequences
    src = _filled(pk, B, 2, 20, 2, [128 * (1 + b % 20) for b in range(B)], 6)
    pk.packkv_free_blocks(src, [0] * B, [b % 3 if b % 20 >= 2 else 0 for b in range(B)])
    dst = pk.PackKVCache(B, 2, 20, 2, ragged=True, keep_perm=True)
    pk.packkv_compact(dst, src)
    _check_compacted(pk, dst, src)
    before = dst.k_index.clone()
    pk.packkv_fork_sequences(dst, [19] * 66, [b for b in range(B) if b not in (0, 19, 68, 69)])
    assert torch.equal(dst.k_index[67], before[19]) and torch.equal(dst.k_index[68], before[68])
    assert dst.seq_blocks[5] == 20 and dst.seq_blocks[0] == 1


def test_serving_loop(pk):
    """The operators together: a prompt prepared and encoded, forked into two samples, both
    decoded with a sliding window (norm, rotation, append, attention), blocks behind the
    window freed, the cache compacted halfway; every step against 64-bit arithmetic."""
    B, hq, hkv, P, steps, W, N0, bits = 3, 4, 2, 500, 24, 200, 4, 4
    g = torch.Generator().manual_seed(1)
    spec = dict(scaling=3, factor=4.0, original_tokens=256.0, low=1.0, high=32.0)
    rope = pk.Rope(128, pk.ROPE_HALF, 10000.0, **spec)
    freq = O.rope_frequencies(128, 10000.0, **spec)
    wq, wk = 1 + 0.1 * torch.randn(128, generator=g), 1 + 0.1 * torch.randn(128, generator=g)
    prompt = torch.randn(B, P, hq + 2 * hkv, 128, generator=g).bfloat16()
    cache = pk.PackKVCache(B, hkv, 6, bits, ragged=True, keep_perm=True)
    oc = O.RaggedOracleCache(B, hkv, 6, bits)
    outs = [torch.empty((B, h, P, 128), dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv)]
    d = prompt.cuda()
    pk.packkv_norm_rope(rope, d[:, :, :hq], d[:, :, hq:hq + hkv], d[:, :, hq + hkv:], *outs, q_weight=wq.cuda(),
                        k_weight=wk.cuda(), eps=1e-6)
    ref = O.norm_rope(prompt.double().numpy()[:, :, hq:hq + hkv].transpose(0, 2, 1, 3),
                      np.broadcast_to(np.arange(P), (B, hkv, P)), freq, O.ROPE_HALF, 1.0, 1e-6, wk.numpy())
    assert np.abs(outs[1].double().cpu().numpy() - ref).max() <= np.abs(ref).max() * 2.0 ** -11 + 2.0 ** -18
    full = P // 128
    pk.packkv_encode_block(cache, outs[1][:, :, :full * 128].contiguous(), outs[2][:, :, :full * 128].contiguous(), full)
    kh, vh = outs[1].cpu().numpy(), outs[2].cpu().numpy()
    oc.encode_blocks_ragged(kh[:, :, :full * 128], vh[:, :, :full * 128], full)
    for t in range(full * 128, P):
        pk.packkv_append_token(cache, outs[1][:, :, t].contiguous(), outs[2][:, :, t].contiguous())
        oc.append_token_ragged(kh[:, :, t], vh[:, :, t])
    # sequence 2 becomes a second sample of sequence 0
    pk.packkv_fork_sequences(cache, [0], [2])
    n = oc.seq_blocks[0]
    for name in ("k_index", "v_index", "perm"):
        getattr(oc, name)[2, :, :n] = getattr(oc, name)[0, :, :n]
    oc.k_tail[2], oc.v_tail[2] = oc.k_tail[0], oc.v_tail[0]
    oc._decoded.clear()
    for step in range(steps):
        x = torch.randn(B, hq + 2 * hkv, 128, generator=g).bfloat16()
        dx = x.cuda()
        q_out = torch.empty((B, hq, 128), dtype=torch.float16, device="cuda")
        on = [True, step % 3 != 0, True]
        q_out.zero_()
        pk.packkv_append_norm_rope(cache, rope, dx[:, :hq], dx[:, hq:hq + hkv], dx[:, hq + hkv:], q_out,
                                   q_weight=wq.cuda(), k_weight=wk.cuda(), eps=1e-6, active=on)
        pos = np.array([oc.seq_tokens(b) for b in range(B)])
        kref = O.norm_rope(x.double().numpy()[:, hq:hq + hkv], np.broadcast_to(pos[:, None], (B, hkv)), freq,
                           O.ROPE_HALF, 1.0, 1e-6, wk.numpy())
        # the tail's own bits go on into the oracle (they are within half a step of kref)
        slot = [t % 128 for t in pos]
        for b in range(B):
            if not on[b]:
                continue
            if slot[b] < 127:
                got = cache.k_tail[b, :, slot[b]].double().cpu().numpy()
                assert np.abs(got - kref[b]).max() <= np.abs(kref[b]).max() * 2.0 ** -11 + 2.0 ** -18
        kt = np.stack([cache.k_tail[b, :, slot[b]].cpu().numpy() for b in range(B)])
        vt = np.stack([cache.v_tail[b, :, slot[b]].cpu().numpy() for b in range(B)])
        oc.append_token_ragged(kt, vt, [b for b in range(B) if on[b]])
        assert cache.seq_blocks == oc.seq_blocks and cache.seq_tail == oc.seq_tail
        out = torch.empty((B, hq, 128), device="cuda")
        pk.packkv_attention_window(cache, q_out, SCALE, out, W, sinks=N0)
        want, terms = O.window_attention(oc, q_out.cpu().numpy(), SCALE, W, N0, 1)
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= 1e-3 * terms)
        if step == steps // 2:
            # block 0 holds the sinks; whole blocks behind the window go
            behind = [max(0, (oc.seq_tokens(b) - W) // 128 - 1) for b in range(B)]
            pk.packkv_free_blocks(cache, [1] * B, behind)
            assert max(behind) > 0
            spare = pk.PackKVCache(B, hkv, 6, bits, ragged=True, keep_perm=True)
            used = cache.arena_used()
            pk.packkv_compact(spare, cache)
            cache = spare
            assert cache.arena_used()[0] < used[0]
    assert pk.packkv_get_status(cache) == 0
    assert max(oc.seq_blocks) >= full + 1     # a tail was encoded on the way


def test_reset_sequence_and_reuse(pk):
    """A sequence that is done: its blocks freed, its counters zeroed, its room taken back by
    a compaction, and a new request encoded after it."""
    cache = _filled(pk, 2, 1, 4, 4, [400, 300], 11, arena_bytes=8 * 8720)
    pk.packkv_free_blocks(cache, [0, 0], [3, 0])
    cache.set_lengths([0, cache.seq_blocks[1]], [0, cache.seq_tail[1]])
    dst = pk.PackKVCache(2, 1, 4, 4, ragged=True, keep_perm=True, arena_bytes=8 * 8720)
    pk.packkv_compact(dst, cache)
    _check_compacted(pk, dst, cache)
    k = torch.randn(2, 1, 128, device="cuda").half()
    for _ in range(128):
        pk.packkv_append_token_masked(dst, k, k, [True, False])
    assert dst.seq_blocks == [1, 2] and pk.packkv_get_status(dst) == 0


def test_captured_and_replayed(pk):
    """Fork, free and compact in one graph, replayed after the source has changed."""
    src = _filled(pk, 3, 2, 4, 4, [400, 256, 30], 21)
    dst = pk.PackKVCache(3, 2, 4, 4, ragged=True, keep_perm=True)
    lengths = src.seq_blocks, src.seq_tail
    keep = src.k_index.clone(), src.v_index.clone()

    def calls():
        pk.packkv_fork_sequences(src, [0], [2])
        pk.packkv_free_blocks(src, [0, 1, 0], [1, 1, 0])
        pk.packkv_compact(dst, src)

    calls()
    torch.cuda.synchronize()
    want = _snapshot(dst), dst.k_arena.clone()
    src.set_lengths(*lengths)
    src.k_index.copy_(keep[0])
    src.v_index.copy_(keep[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for x in (dst.k_index, dst.v_index, dst.k_arena, dst.ctrl, dst.perm):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    n = dst.arena_used()[0]
    for name, x in want[0].items():
        assert torch.equal(getattr(dst, name), x), name
    assert torch.equal(dst.k_arena[:n], want[1][:n])
    _check_compacted(pk, dst, src)


def test_lengths_are_checked(pk):
    cache = pk.PackKVCache(2, 1, 3, 4, ragged=True)
    cache.set_lengths([1, 3], [127, 0])
    for bad in (([4, 0], [0, 0]), ([0, 0], [128, 0]), ([-1, 0], [0, 0])):
        with pytest.raises(pk.PackKVError):
            cache.set_lengths(*bad)
    for bad in (([1], [0]), ([1, 1], [0])):
        with pytest.raises(ValueError):
            cache.set_lengths(*bad)
    with pytest.raises(TypeError):
        cache.set_lengths([0, 0], ["a", 0])
    assert cache.seq_blocks == [1, 3] and cache.seq_tail == [127, 0]
    flat = pk.PackKVCache(1, 1, 3, 4)
    flat.set_lengths(2, 5)
    with pytest.raises(pk.PackKVError):
        flat.set_lengths(4)
    assert (flat.n_blocks, flat.tail_len) == (2, 5)
