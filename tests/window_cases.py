"""Caches of many sequences and the 64-bit reference for the tests of windowed attention.

`many` makes a batch of 72 sequences x 8 heads over the blocks of two: with three blocks
and a tail it has over 2300 items of one query row, more than half of the warps a B200
holds, so the calls take the even split (`test_gpu_window`'s small batches take clusters).
"""
from __future__ import annotations

import numpy as np
import torch

import oracle as O
from decode_gemv_packkv_b200 import synth
from parity_util import to_dev

SCALE = 1.0 / np.sqrt(128.0)


def queries(B, rows, seed, size=1.0):
    return (size * np.random.default_rng(seed).standard_normal((B, rows, 128))).astype(np.float16)


def many(pk, bits, structured, seed, B=72, H=8, tokens=(400, 390), table=False):
    """The cache, and the oracle of its first two sequences: sequence b is a copy of
    sequence b % 2, forked (index entries of its own) or through a block table."""
    k, v, _ = synth.small_case(seed, 2, H, 1, max(tokens), structured=structured)
    nb = tokens[0] // 128
    assert nb == tokens[1] // 128
    cache = pk.PackKVCache(B, H, nb, bits, ragged=True, keep_perm=True)
    oc = O.RaggedOracleCache(2, H, nb, bits)
    oc.encode_blocks_ragged(k[:, :, :nb * 128], v[:, :, :nb * 128], nb)
    tail = [t % 128 for t in tokens]
    oc.seq_tail = list(tail)
    for b in range(2):
        oc.k_tail[b, :, :tail[b]] = k[b, :, nb * 128:tokens[b]]
        oc.v_tail[b, :, :tail[b]] = v[b, :, nb * 128:tokens[b]]
    wide = [torch.zeros((B, H, nb * 128, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    for w, x in zip(wide, (k, v)):
        w[:2] = to_dev(x[:, :, :nb * 128])
    pk.packkv_encode_block(cache, *wide, nb)
    cache.k_tail[:2] = to_dev(oc.k_tail)
    cache.v_tail[:2] = to_dev(oc.v_tail)
    if not table:
        cache.set_lengths([nb] * B, tail + [0] * (B - 2))
        pk.packkv_fork_sequences(cache, [b % 2 for b in range(2, B)], list(range(2, B)))
    else:
        for x in (cache.k_tail, cache.v_tail):
            x[2:] = x[:2].repeat(B // 2 - 1, 1, 1, 1)
        cache.set_lengths([nb] * B, tail * (B // 2))
        cache.block_table = (torch.arange(2).repeat(B // 2)[:, None] * nb + torch.arange(nb)).int().cuda()
        cache.s.block_table = cache.block_table.data_ptr()
    return cache, oc


def reference(oc, of, q, window, sinks, n_queries, scale=SCALE, without=()):
    """Outputs and sum_i p_i |v_i| of the queries q [B, heads * rows, 128], sequence b
    attending to the oracle's sequence of[b]; without: (b, head, logical block) whose tokens
    do not count."""
    B, rows = q.shape[0], q.shape[1] // oc.kv_heads
    out, terms = np.zeros(q.shape), np.zeros(q.shape)
    masks = {}
    for s in set(of):
        masks[s] = O.window_mask(oc.seq_tokens(s), n_queries, window, sinks)
    keys = {(s, h): [O.arrival_order(oc, which, s, h) for which in "kv"] for s in set(of) for h in range(oc.kv_heads)}
    for b in range(B):
        for h in range(oc.kv_heads):
            see = masks[of[b]].copy()
            for j in range(oc.seq_blocks[of[b]]):
                if (b, h, j) in without:
                    see[:, 128 * j:128 * j + 128] = False
            see = np.repeat(see, rows // n_queries, axis=0)
            if see.shape[1] == 0:
                continue
            k, v = keys[of[b], h]
            r = slice(h * rows, (h + 1) * rows)
            score = np.where(see, scale * np.asarray(q[b, r], np.float64) @ k.T, -np.inf)
            top = score.max(axis=1, keepdims=True)
            p = np.exp(score - np.where(np.isfinite(top), top, 0.0))
            total = p.sum(axis=1, keepdims=True)
            p = p / np.where(total > 0, total, 1.0)
            out[b, r] = p @ v
            terms[b, r] = p @ np.abs(v)
    return out, terms


def whole_softmax_with_digits(oc, q, digits, scale=SCALE):
    """The oracle's outputs over sequence 0, head 0 (whole blocks, everything seen) with q'
    rounded as the kernels' integer digits round it: per block q' = q times the channels'
    steps, scaled to 127 (three digits, 2^-14 the last) or to a power of two below 64 (four,
    2^-21).  digits None: exact."""
    k, v = (O.arrival_order(oc, which, 0, 0) for which in "kv")
    q = np.asarray(q, np.float64)
    score = scale * q @ k.T
    for j in range(oc.seq_blocks[0]) if digits else ():
        block = k[128 * j:128 * j + 128]
        low = block.min(axis=0)
        step = (block.max(axis=0) - low) / (2 ** oc.bits - 1)
        code = (block - low) / np.where(step > 0, step, 1.0)
        top = np.abs(q * step).max(axis=1, keepdims=True)
        f = 127 / top if digits == 3 else 2.0 ** (5 - np.floor(np.log2(top)))
        last = 2.0 ** (14 if digits == 3 else 21)
        y = np.rint(q * step * f * last) / last
        score[:, 128 * j:128 * j + 128] = scale * ((y / f) @ code.T + (q @ low)[:, None])
    return O.softmax(score) @ v
