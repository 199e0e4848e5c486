"""Plain 64-bit definitions of the operators around the packed cache: norm and rotation
of the heads, windowed attention, and what forking, freeing and compacting do.

The pages do not describe these steps (they start at the cached K and V and end at the
attention output); the definitions are the textbook ones, written out.
"""
from __future__ import annotations

import numpy as np

from .packkv_oracle import BLOCK_TOKENS, HEAD_DIM, RaggedOracleCache, softmax

ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_SCALE_NONE, ROPE_SCALE_LINEAR, ROPE_SCALE_BASE, ROPE_SCALE_PARTS = range(4)


def rope_frequencies(rot_dim, theta, scaling=ROPE_SCALE_NONE, factor=1.0, original_tokens=0.0, low=1.0, high=32.0):
    """Angle per position of pair i = theta^(-2i/rot_dim), scaled for long contexts."""
    out = []
    for i in range(rot_dim // 2):
        base = theta
        if scaling == ROPE_SCALE_BASE and rot_dim > 2:
            base = theta * factor ** (rot_dim / (rot_dim - 2))
        f = base ** (-2.0 * i / rot_dim)
        if scaling == ROPE_SCALE_LINEAR:
            f = f / factor
        if scaling == ROPE_SCALE_PARTS:
            turns = original_tokens * f / (2 * np.pi)
            keep = min(max((turns - low) / (high - low), 0.0), 1.0)
            f = keep * f + (1 - keep) * f / factor
        out.append(f)
    return np.array(out, np.float64)


def norm_rope(x, positions, freq, layout, amplitude=1.0, eps=None, weight=None):
    """Heads x [..., 128] at positions [...] (broadcast over x's leading dimensions), fp64."""
    y = np.asarray(x, np.float64).copy()
    if eps is not None:
        y = y / np.sqrt((y * y).sum(-1, keepdims=True) / HEAD_DIM + eps)
        if weight is not None:
            y = y * np.asarray(weight, np.float64)
    n = len(freq)
    out = y.copy()
    for i in range(n):
        a, b = (i, i + n) if layout == ROPE_HALF else (2 * i, 2 * i + 1)
        angle = np.asarray(positions, np.float64) * freq[i]
        c, s = np.cos(angle) * amplitude, np.sin(angle) * amplitude
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def window_mask(tokens, queries, window, sinks):
    """[queries, tokens]: query s sits at tokens - queries + s and sees i <= p with
    i > p - window or i < sinks."""
    p = np.arange(tokens - queries, tokens)[:, None]
    i = np.arange(tokens)[None, :]
    return (i <= p) & ((i > p - window) | (i < sinks))


def arrival_order(cache: RaggedOracleCache, which, b, h):
    """Sequence b, head h decoded to fp64 [T_b, 128] in arrival order (the permutations of
    the blocks undone); freed blocks give NaN."""
    stored = cache.decoded(which, b, h)
    out = stored.copy()
    for j in range(cache.seq_blocks[b]):
        rb, jb = cache.physical(b, j)
        at = j * BLOCK_TOKENS
        out[at + cache.perm[rb, h, jb].astype(np.int64)] = stored[at:at + BLOCK_TOKENS]
    return out


def window_attention(cache: RaggedOracleCache, q, scale, window, sinks, queries):
    """q [B, Hkv * queries * G, 128], row (h * queries + s) * G + g.  Returns the outputs
    (zero rows where nothing is seen) and sum_i |p_i v_ic|."""
    B, rows, _ = q.shape
    n = rows // cache.kv_heads
    g = n // queries
    out, terms = np.zeros((B, rows, HEAD_DIM)), np.zeros((B, rows, HEAD_DIM))
    for b in range(B):
        t = cache.seq_tokens(b)
        if t == 0:
            continue
        mask = window_mask(t, queries, window, sinks)
        for h in range(cache.kv_heads):
            k, v = arrival_order(cache, "k", b, h), arrival_order(cache, "v", b, h)
            for s in range(queries):
                see = mask[s]
                if not see.any():
                    continue
                r = slice((h * queries + s) * g, (h * queries + s) * g + g)
                score = scale * np.asarray(q[b, r], np.float64) @ k[see].T
                p = softmax(score)
                out[b, r] = p @ v[see]
                terms[b, r] = p @ np.abs(v[see])
    return out, terms


def compacted(index, arena, blocks, physical):
    """Index entries int64 [B, H, max_blocks, 2] and the arena (bytes) of a compaction:
    live records in (sequence, head, logical block) order of their first entry, once
    each; freed entries (offset 0xFFFFFFFF) stay freed.  physical(b, j): the index place of
    logical block j.  Returns {(b, h, j): (offset, length)} and the new arena."""
    where, entries, out = {}, {}, bytearray()
    B, H = index.shape[:2]
    for b in range(B):
        for h in range(H):
            for j in range(blocks[b]):
                rb, jb = physical(b, j)
                off, length = (int(x) for x in index[rb, h, jb])
                if off == 0xFFFFFFFF:
                    entries[b, h, j] = (0xFFFFFFFF, 0)
                    continue
                if off not in where:
                    where[off] = len(out) // 16
                    out += arena[off * 16:(off + length) * 16]
                entries[b, h, j] = (where[off], length)
    return entries, bytes(out)
