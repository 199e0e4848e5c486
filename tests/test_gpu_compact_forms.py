"""Compaction over index entries made for the purpose (it reads lengths and copies bytes, so a
record may hold anything): entries that overlap, caches of several batches per warp, and
offsets summed over more tiles than one look-back step reads.  Bit for bit against the oracle.
"""
import numpy as np
import pytest
import torch

import oracle as O
from parity_util import gpu_records

pytestmark = pytest.mark.gpu

FREED = 0xFFFFFFFF
MIN = 65  # 16-byte units of the smallest record


@pytest.fixture(scope="module")
def pk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_gemv_packkv_b200 import packkv
    return packkv


def _made(pk, B, H, mb, bits, blocks, seed, fresh=0.5, shared=0.3):
    """A ragged cache whose sequences hold blocks[b] blocks: an entry names a record of its
    own (with probability `fresh`), one that an earlier entry names, or none (freed).
    Records lie in a shuffled order, with gaps."""
    rng = np.random.default_rng(seed)
    most = pk.record_bytes_max(bits) // 16
    index, end = {}, 0
    for which in "kv":
        n = B * H * mb
        kind = rng.random(n)
        own = np.flatnonzero(kind < fresh)
        length = rng.integers(MIN, most + 1, own.size)
        order = rng.permutation(own.size)
        gap = rng.integers(0, 4, own.size)
        at = np.empty(own.size, np.int64)
        at[order] = np.cumsum(length[order] + gap[order]) - length[order]
        end = max(end, int((length + gap).sum()))
        x = np.full((n, 2), (FREED, 0), np.int64)
        x[own, 0], x[own, 1] = at, length
        again = np.flatnonzero((kind >= fresh) & (kind < fresh + shared))
        x[again] = x[rng.choice(own, again.size)]
        index[which] = x.reshape(B, H, mb, 2)
    cache = pk.PackKVCache(B, H, mb, bits, ragged=True, keep_perm=True, arena_bytes=16 * (end + 8))
    cache.k_index.copy_(torch.from_numpy(index["k"].astype(np.uint32).view(np.int32)))
    cache.v_index.copy_(torch.from_numpy(index["v"].astype(np.uint32).view(np.int32)))
    for x in (cache.k_arena, cache.v_arena, cache.perm):
        x.copy_(torch.randint(0, 256, x.shape, dtype=torch.uint8, generator=torch.Generator().manual_seed(seed)))
    for x in (cache.k_tail, cache.v_tail):
        x.normal_()
    cache.ctrl[:2] = end + 8
    cache.set_lengths(blocks, [(37 * b) % 128 for b in range(B)])
    return cache


def _target(pk, src):
    dst = pk.PackKVCache(src.batch, src.kv_heads, src.s.max_blocks, src.bits, ragged=True, keep_perm=True,
                         arena_bytes=src.k_arena.numel())
    for x in (dst.k_arena, dst.v_arena, dst.perm):
        x.fill_(0xEE)
    for x in (dst.k_index, dst.v_index):
        x.fill_(7)
    return dst


def _check(pk, dst, src, bad=()):
    """bad: (tensor, b, h, j) of entries that come out as freed, with the status bit."""
    for t, which in enumerate("kv"):
        arena, index = gpu_records(src, which)
        for name, b, h, j in bad:
            if name == which:
                index[b, h, j] = (FREED, 0)
        entries, want = O.compacted(index, arena.tobytes(), src.seq_blocks, lambda b, j: (b, j))
        got_arena, got = gpu_records(dst, which)
        expect = np.full(got.shape, 7, np.int64)  # behind the lengths: left as it was
        for (b, h, j), entry in entries.items():
            expect[b, h, j] = entry
        assert np.array_equal(got, expect)
        assert int(dst.ctrl[t]) * 16 == len(want)
        assert got_arena[:len(want)].tobytes() == want and np.all(got_arena[len(want):] == 0xEE)
    held = torch.tensor(src.seq_blocks, device="cuda")[:, None] > torch.arange(src.s.max_blocks, device="cuda")
    held = held[:, None, :, None].expand_as(src.perm)
    assert torch.equal(dst.perm, torch.where(held, src.perm, torch.full_like(src.perm, 0xEE)))
    held = torch.tensor(src.seq_tail, device="cuda")[:, None] > torch.arange(128, device="cuda")
    held = held[:, None, :, None].expand_as(src.k_tail)
    for name in ("k_tail", "v_tail"):
        x, y = getattr(dst, name), getattr(src, name)
        assert torch.equal(x, torch.where(held, y, torch.zeros_like(y)))
    assert pk.packkv_get_status(dst) == (pk.DEV_BAD_RECORD if bad else 0)


# entries: one tile; up to 4736 (a batch of four per warp); more; more than 32 tiles of 1024
@pytest.mark.parametrize("B,H,mb", [(5, 3, 9), (6, 7, 40), (66, 4, 40), (60, 32, 20), (130, 16, 19)])
def test_sizes(pk, B, H, mb):
    src = _made(pk, B, H, mb, 2, [(7 * b + 3) % (mb + 1) if b else mb for b in range(B)], B)
    dst = _target(pk, src)
    pk.packkv_compact(dst, src)
    _check(pk, dst, src)
    before = [x.clone() for x in (dst.k_index, dst.v_index, dst.k_arena, dst.v_arena)]
    pk.packkv_compact(dst, src)  # the same workspace again: the same bits
    for x, y in zip((dst.k_index, dst.v_index, dst.k_arena, dst.v_arena), before):
        assert torch.equal(x, y)


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("B,H,mb", [(2, 2, 8), (20, 4, 16)])   # one tile, and two
def test_overlapping_entries(pk, B, H, mb, bits):
    """Two entries whose records begin within 65 units of each other cannot both be records:
    the first in order keeps its own, the other comes out as freed, and the status says so.
    The same of an entry that gives a record another length."""
    src = pk.PackKVCache(B, H, mb, bits, ragged=True, keep_perm=True, arena_bytes=16 * 1000)
    for x in (src.k_arena, src.v_arena):
        x.random_(0, 256)
    for x in (src.k_index, src.v_index):
        x.copy_(torch.tensor([-1, 0], dtype=torch.int32).expand_as(x))
    src.set_lengths([mb] * B, [0] * B)
    a, b = (0, 0, 1), (B - 1, H - 1, mb - 2)
    for index, base in ((src.k_index, 195), (src.v_index, 390)):
        index[0, 0, 0] = torch.tensor([0, 80], dtype=torch.int32)
        index[a] = torch.tensor([base, 70], dtype=torch.int32)
        index[b] = torch.tensor([base + 1, 70], dtype=torch.int32)
    src.v_index[b] = torch.tensor([390, 71], dtype=torch.int32)
    dst = _target(pk, src)
    pk.packkv_compact(dst, src)
    assert dst.k_index[b].tolist() == [-1, 0] and dst.v_index[b].tolist() == [-1, 0]
    assert dst.k_index[a].tolist() == [80, 70] and dst.v_index[a].tolist() == [80, 70]
    _check(pk, dst, src, bad=[("k", *b), ("v", *b)])
