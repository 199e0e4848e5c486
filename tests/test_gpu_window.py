"""packkv_attention_window against the oracle: sliding windows with first tokens that stay
visible, one and several query positions, ragged batches, block tables, freed blocks.

Tolerance: the repository's own, 1e-3 * sum|terms| per element, and on the whole output a
relative 2-norm of 1e-5: the scores' integer products carry q' to 2^-22 of its largest
value or better (three digits), which leaves scores of these inputs (|q'| up to about 16,
128 channels, codes up to 15 with a spread of about 3, scale 0.09) off by
0.09 * sqrt(128) * 3 * 16 * 2^-22 / sqrt(3) = 7e-6 on average, and an output by about as much.
"""
import numpy as np
import pytest
import torch

import oracle as O
from decode_gemv_packkv_b200 import synth
from parity_util import assert_within_terms, to_dev

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(128.0)


@pytest.fixture(scope="module")
def pk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_gemv_packkv_b200 import packkv
    return packkv


def _caches(pk, B, H, bits, tokens, seed, structured=False, key=O.KEY_K_SUM, mb=None):
    """A ragged GPU cache and its oracle with tokens[b] tokens in sequence b."""
    T = max(max(tokens), 1)
    k, v, _ = synth.small_case(seed, B, H, 1, T, structured=structured)
    nb = [t // 128 for t in tokens]
    mb = mb or max(max(nb), 1)
    cache = pk.PackKVCache(B, H, mb, bits, reorder_key=key, ragged=True, keep_perm=True)
    oc = O.RaggedOracleCache(B, H, mb, bits, key)
    most = max(nb)
    if most:
        pk.packkv_encode_block(cache, to_dev(k[:, :, :most * 128]), to_dev(v[:, :, :most * 128]), most)
        oc.encode_blocks_ragged(k[:, :, :most * 128], v[:, :, :most * 128], most)
    cache.set_lengths(nb, [0] * B)
    oc.seq_blocks, oc.seq_tail = list(nb), [t % 128 for t in tokens]
    for b, t in enumerate(tokens):
        oc.k_tail[b, :, :t % 128] = k[b, :, nb[b] * 128:t]
        oc.v_tail[b, :, :t % 128] = v[b, :, nb[b] * 128:t]
    cache.k_tail.copy_(to_dev(oc.k_tail))
    cache.v_tail.copy_(to_dev(oc.v_tail))
    cache.set_lengths(nb, oc.seq_tail)
    return cache, oc


def _queries(B, rows, seed):
    return np.random.default_rng(seed).standard_normal((B, rows, 128)).astype(np.float16)


def _check(pk, cache, oc, rows, queries, window, sinks, seed, what=""):
    q = _queries(oc.batch, oc.kv_heads * rows, seed)
    out = torch.full(q.shape, 7.0, device="cuda")
    pk.packkv_attention_window(cache, to_dev(q), SCALE, out, window, sinks=sinks, queries=queries)
    ref, terms = O.window_attention(oc, q, SCALE, window, sinks, queries)
    got = out.double().cpu().numpy()
    assert_within_terms(got, ref, terms, f"{what} window {window} sinks {sinks}")
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(got - ref) <= 1e-5 * norm
    assert pk.packkv_get_status(cache) == 0
    return out


# bits, rows per kv head, queries, structured
SHAPES = [(4, 1, 1, False), (4, 4, 1, True), (3, 2, 2, False), (2, 8, 4, True), (3, 8, 1, True), (4, 16, 4, False),
          (2, 1, 1, True), (2, 64, 8, False), (3, 4, 4, True), (4, 2, 1, True)]


@pytest.mark.parametrize("bits,rows,queries,structured", SHAPES)
def test_windows_over_ragged_lengths(pk, bits, rows, queries, structured):
    """Lengths of nothing, one token, less than the queries, whole blocks, and tails; windows
    that end inside blocks, hold one token, and hold everything."""
    cache, oc = _caches(pk, 6, 2, bits, [700, 0, 1, 3, 256, 399], 40 + bits + rows, structured)
    for window, sinks in [(300, 4), (1, 0), (128, 0), (100000, 0), (129, 130), (37, 1)]:
        _check(pk, cache, oc, rows, queries, window, sinks, window, f"{bits} bits, {rows} rows")


@pytest.mark.parametrize("tokens", [127, 128, 129, 159, 160, 161, 255, 383])
def test_borders_of_tail_and_window(pk, tokens):
    cache, oc = _caches(pk, 1, 1, 4, [tokens], tokens)
    for window in (1, 31, 32, 33, 127, 128, 129, tokens - 1, tokens, tokens + 1):
        _check(pk, cache, oc, 2, 2, window, 0, window)
        _check(pk, cache, oc, 1, 1, window, 5, window)


def test_large_limits(pk):
    cache, oc = _caches(pk, 2, 1, 2, [300, 70], 3)
    big = (1 << 31) - 1
    for window, sinks in [(big, 0), (1, big), (big, big), (1 << 40, 1 << 33)]:
        _check(pk, cache, oc, 1, 1, window, sinks, 1)
        _check(pk, cache, oc, 8, 8, window, sinks, 2)


def test_uniform_batch_and_identity_order(pk):
    """A uniform batch (no ragged counters), and an unreordered cache without permutations;
    with everything in the window the result is packkv_attention_decode's to rounding."""
    B, H, T = 2, 3, 500
    k, v, _ = synth.small_case(77, B, H, 1, T)
    cache = pk.PackKVCache(B, H, 4, 4, reorder_key=pk.KEY_IDENTITY)
    pk.prefill(cache, to_dev(k), to_dev(v))
    oc = O.RaggedOracleCache(B, H, 4, 4, O.KEY_IDENTITY)
    oc.encode_blocks_ragged(k[:, :, :384], v[:, :, :384], 3)
    for t in range(384, T):
        oc.append_token_ragged(k[:, :, t], v[:, :, t])
    _check(pk, cache, oc, 4, 2, 200, 3, 1)
    out = _check(pk, cache, oc, 4, 1, T, 0, 9)
    full = torch.empty_like(out)
    pk.packkv_attention_decode(cache, to_dev(_queries(B, H * 4, 9)), SCALE, full)
    assert torch.linalg.norm(out - full) <= 2e-5 * torch.linalg.norm(full)


def test_reordered_cache_needs_its_permutations(pk):
    cache = pk.PackKVCache(1, 1, 1, 4)
    q = torch.zeros((1, 1, 128), dtype=torch.float16, device="cuda")
    with pytest.raises(pk.PackKVError) as e:
        pk.packkv_attention_window(cache, q, 1.0, torch.empty((1, 1, 128), device="cuda"), 8)
    assert e.value.status == pk.ERR_INVALID_ARG


def test_block_table(pk):
    """Shared and permuted physical blocks."""
    cache, oc = _caches(pk, 3, 2, 3, [600, 300, 290], 12, True, mb=5)
    table = np.arange(15, dtype=np.int32).reshape(3, 5)
    table[2, :2] = table[0, :2]
    table[0, :4] = [3, 1, 0, 2]
    oc.table = table.astype(np.int64)
    oc._decoded.clear()
    cache.block_table = torch.from_numpy(table).cuda()
    cache.s.block_table = cache.block_table.data_ptr()
    for window, sinks in [(200, 4), (1000, 0), (10, 140)]:
        _check(pk, cache, oc, 4, 2, window, sinks, window)


def test_freed_blocks_behind_the_window(pk):
    """Blocks that no query sees may be freed; a freed block that one sees is reported and
    its tokens are left out."""
    cache, oc = _caches(pk, 2, 2, 4, [1100, 900], 31)
    pk.packkv_free_blocks(cache, [1, 1], [5, 3])   # sequence 0: blocks 1..5, 1: 1..3
    out = _check(pk, cache, oc, 2, 1, 300, 4, 5)
    q = to_dev(_queries(2, 4, 5))
    pk.packkv_attention_window(cache, q, SCALE, out, 400, sinks=4)   # sequence 0's block 5 is seen
    assert pk.packkv_get_status(cache) & pk.DEV_BAD_RECORD
    keep = torch.isfinite(out)
    assert torch.all(keep)


def test_masked_infinities_do_not_spread(pk):
    """Infinite and NaN tail values behind a query's position leave its output alone."""
    cache, oc = _caches(pk, 1, 2, 4, [200], 8)
    q = to_dev(_queries(1, 2 * 4, 3))
    clean = torch.empty((1, 8, 128), device="cuda")
    pk.packkv_attention_window(cache, q, SCALE, clean, 64, queries=4)
    cache.v_tail[0, 0, 71, 5] = float("inf")    # the last token: only the last query sees it
    cache.v_tail[0, 1, 70, 9] = float("nan")
    cache.k_tail[0, 1, 71, 7] = float("nan")
    out = torch.empty_like(clean)
    pk.packkv_attention_window(cache, q, SCALE, out, 64, queries=4)
    same = torch.isclose(out, clean, rtol=1e-5, atol=1e-6)
    assert torch.all(same[0, :3])                # kv head 0, positions 0..2
    assert torch.isinf(out[0, 3, 5]) and torch.all(torch.isfinite(out[0, 3, 6:]))
    assert torch.all(same[0, 4:6])               # kv head 1, positions 0..1
    assert torch.isnan(out[0, 6, 9]) and torch.all(torch.isfinite(out[0, 6, 10:]))
    assert torch.all(torch.isnan(out[0, 7]))     # a NaN key that it sees


def test_masked_infinities_in_the_even_split(pk):
    """The same with enough sequences that every warp takes several items: the last tail token
    is infinite in half of them and seen by the last of two queries alone."""
    B, H = 96, 16
    k, v, _ = synth.small_case(3, 1, H, 1, 300)
    cache = pk.PackKVCache(B, H, 2, 4, ragged=True, keep_perm=True)
    kd, vd = to_dev(k).expand(B, -1, -1, -1), to_dev(v).expand(B, -1, -1, -1)
    pk.packkv_encode_block(cache, kd[:, :, :256].contiguous(), vd[:, :, :256].contiguous(), 2)
    cache.k_tail[:, :, :44] = kd[:, :, 256:]
    cache.v_tail[:, :, :44] = vd[:, :, 256:]
    cache.set_lengths([2] * B, [44] * B)
    q = to_dev(_queries(B, H * 2, 5))
    clean, out = torch.empty((B, H * 2, 128), device="cuda"), torch.empty((B, H * 2, 128), device="cuda")
    pk.packkv_attention_window(cache, q, SCALE, clean, 1000, queries=2)
    cache.v_tail[::2, :, 43, 17] = float("-inf")
    pk.packkv_attention_window(cache, q, SCALE, out, 1000, queries=2)
    assert torch.all(torch.isclose(out[:, 0::2], clean[:, 0::2], rtol=1e-5, atol=1e-6))
    assert torch.equal(out[1::2], clean[1::2])
    assert torch.all(torch.isinf(out[::2, 1::2, 17])) and torch.all(torch.isfinite(out[::2, 1::2, 18:]))


def test_nan_and_infinite_queries(pk):
    cache, _ = _caches(pk, 1, 1, 3, [300], 4)
    q = torch.randn(1, 2, 128, device="cuda").half()
    clean = torch.empty((1, 2, 128), device="cuda")
    pk.packkv_attention_window(cache, q, SCALE, clean, 200)
    q[0, 1, 3] = float("nan")
    out = torch.empty_like(clean)
    pk.packkv_attention_window(cache, q, SCALE, out, 200)
    assert torch.equal(out[0, 0], clean[0, 0]) and torch.all(torch.isnan(out[0, 1]))


def test_repeatable_and_in_a_graph(pk):
    """The same bits every time, eager and replayed, on a stream of its own."""
    cache, oc = _caches(pk, 3, 4, 4, [3000, 1300, 90], 6)
    q = to_dev(_queries(3, 16, 1))
    out = torch.empty((3, 16, 128), device="cuda")
    pk.packkv_attention_window(cache, q, SCALE, out, 1500, sinks=4)
    want = out.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        out.zero_()
        stream.wait_stream(torch.cuda.current_stream())
        pk.packkv_attention_window(cache, q, SCALE, out, 1500, sinks=4, stream=stream)
        torch.cuda.current_stream().wait_stream(stream)
        assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.packkv_attention_window(cache, q, SCALE, out, 1500, sinks=4)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("rows,queries", [(1, 1), (2, 2), (4, 1), (8, 4)])
def test_many_sequences(pk, rows, queries):
    """More items than half the device's warps (the even split): 72 sequences forked from two,
    every one with queries of its own."""
    B, H = 72, 8
    k, v, _ = synth.small_case(15, 2, H, 1, 400)
    cache = pk.PackKVCache(B, H, 3, 4, ragged=True, keep_perm=True)
    oc = O.RaggedOracleCache(2, H, 3, 4)
    oc.encode_blocks_ragged(k[:, :, :384], v[:, :, :384], 3)
    for t in range(384, 400):
        oc.append_token_ragged(k[:, :, t], v[:, :, t], [0] if t >= 390 else None)
    wide = np.zeros((B, H, 384, 128), np.float16)
    wide[:2] = k[:, :, :384]
    kd = to_dev(wide)
    wide[:2] = v[:, :, :384]
    pk.packkv_encode_block(cache, kd, to_dev(wide), 3)
    cache.k_tail[:2] = to_dev(oc.k_tail)
    cache.v_tail[:2] = to_dev(oc.v_tail)
    cache.set_lengths([3] * B, [16, 6] + [0] * (B - 2))
    pk.packkv_fork_sequences(cache, [b % 2 for b in range(2, B)], list(range(2, B)))
    q = _queries(B, H * rows, rows)
    out = torch.empty(q.shape, device="cuda")
    for window, sinks in [(1000, 0), (140, 2)]:
        pk.packkv_attention_window(cache, to_dev(q), SCALE, out, window, sinks=sinks, queries=queries)
        got = out.double().cpu().numpy()
        for b in range(0, B, 2):
            ref, terms = O.window_attention(oc, q[b:b + 2], SCALE, window, sinks, queries)
            assert_within_terms(got[b:b + 2], ref, terms, f"sequences {b}, {b + 1}")
            assert np.linalg.norm(got[b:b + 2] - ref) <= 1e-5 * np.linalg.norm(ref)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    qd = to_dev(q)
    with torch.cuda.graph(graph):
        pk.packkv_attention_window(cache, qd, SCALE, out, window, sinks=sinks, queries=queries)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert pk.packkv_get_status(cache) == 0


def test_long_row_and_empty_caches(pk):
    cache, oc = _caches(pk, 1, 1, 3, [128 * 30 + 77], 16)
    _check(pk, cache, oc, 2, 1, 3500, 4, 2)
    for ragged in (False, True):
        cache = pk.PackKVCache(2, 2, 1, 4, ragged=ragged, keep_perm=True)
        out = torch.full((2, 4, 128), 7.0, device="cuda")
        pk.packkv_attention_window(cache, torch.ones((2, 4, 128), device="cuda").half(), SCALE, out, 5, queries=2)
        assert torch.all(out == 0)


def test_refusals_of_the_binding(pk):
    cache = pk.PackKVCache(1, 1, 1, 4, keep_perm=True)
    q = torch.zeros((1, 2, 128), dtype=torch.float16, device="cuda")
    out = torch.empty((1, 2, 128), device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[:, :, :64]), dict(out=out[:, :1]), dict(out=out.half()), dict(q=q.cpu()),
                dict(q=q[0]), dict(ws=torch.empty(16, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            pk.packkv_attention_window(cache, bad.get("q", q), 1.0, bad.get("out", out), 8, ws=bad.get("ws"))
    with pytest.raises(pk.PackKVError) as e:
        pk.packkv_attention_window(cache, q, 1.0, out, 8, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == pk.ERR_INVALID_ARG


def test_uniform_batch_beyond_the_ragged_limit(pk):
    """More sequences than a ragged cache may have; everything in the window."""
    B, T = 2100, 150
    k, v = (torch.randn(B, 1, T, 128, generator=torch.Generator().manual_seed(s)).half().cuda() for s in (1, 2))
    cache = pk.PackKVCache(B, 1, 2, 3, keep_perm=True)
    pk.prefill(cache, k, v)
    q = to_dev(_queries(B, 4, 11))
    out, full = torch.empty(q.shape, device="cuda"), torch.empty(q.shape, device="cuda")
    pk.packkv_attention_window(cache, q, SCALE, out, T)
    pk.packkv_attention_decode(cache, q, SCALE, full)
    assert torch.linalg.norm(out - full) <= 2e-5 * torch.linalg.norm(full)
    assert pk.packkv_get_status(cache) == 0


def test_two_calls_at_once(pk):
    """Two streams, a workspace each, over one cache: the bits of calls made one by one."""
    cache, _ = _caches(pk, 4, 8, 4, [2000, 1000, 500, 90], 9)
    qs = [to_dev(_queries(4, 32, s)) for s in (1, 2)]
    outs = [torch.empty((4, 32, 128), device="cuda") for _ in qs]
    want = []
    for q, out in zip(qs, outs):
        pk.packkv_attention_window(cache, q, SCALE, out, 1500)
        want.append(out.clone())
    need = cache.window_workspace(32).nbytes
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, out, w, stream in zip(qs, outs, ws, streams):
            pk.packkv_attention_window(cache, q, SCALE, out, 1500, ws=w, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@pytest.mark.parametrize("bits", [2, 4])
def test_records_past_four_gib(pk, bits):
    """Records whose offsets in bytes pass 32 bits: the window reads them where they are, and
    compaction brings them to the start of a small cache."""
    tokens, at = 700, 5 << 30
    k, v, _ = synth.small_case(19, 2, 2, 1, tokens)
    caches = [pk.PackKVCache(2, 2, 5, bits, keep_perm=True),
              pk.PackKVCache(2, 2, 5, bits, keep_perm=True, arena_bytes=at + (1 << 20)),
              pk.PackKVCache(2, 2, 5, bits, keep_perm=True)]
    low, high, back = caches
    high.ctrl[:2] = at // 16
    q = to_dev(_queries(2, 8, 4))
    for cache in (low, high):
        pk.prefill(cache, to_dev(k), to_dev(v))
    pk.packkv_compact(back, high)
    outs = [torch.empty((2, 8, 128), device="cuda") for _ in caches]
    for cache, out in zip(caches, outs):
        pk.packkv_attention_window(cache, q, SCALE, out, 600, sinks=4)
        assert pk.packkv_get_status(cache) == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert int(high.k_index[..., 0].long().bitwise_and(0xFFFFFFFF).min()) >= at // 16
