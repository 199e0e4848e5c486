"""Windowed attention in the even split over every kind of record, with block tables, freed
blocks and tails, and the precision of the scores.

Tolerance on the relative 2-norm of unstructured inputs (normal k, v and q, 16 to 20 tokens'
worth of weight per row), from the kernel's arithmetic:
  scores: digits of q' 2^-27 of the largest value, below 1e-7 of an output; the joined sum
    sum q' code is around 80, so each of about five fp32 roundings is at most 2^-18 there,
    0.088 * 2^-18 * sqrt(5 / 3) = 4e-7 in a score, and about 2e-7 in an output (an output
    moves by about half of its scores' error, over rows that differ);
  values: sum p' code and the min term are each about 2.5 against an output of 0.25, with
    about five roundings of at most 2^-23: 2^-23 * sqrt(5 / 3) / 0.25 = 6e-7.
Together 7e-7; the tests allow 2e-6, which three digits would pass (test_window_digits_cpu).
Structured inputs and their compressed records: the repository's 1e-5 of test_gpu_window.
"""
import numpy as np
import pytest
import torch

import oracle as O
from decode_gemv_packkv_b200 import synth
from parity_util import assert_within_terms, to_dev
from window_cases import SCALE, many, queries, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_gemv_packkv_b200 import packkv
    return packkv


def _check(pk, cache, oc, of, rows, n_queries, window, sinks, norm):
    q = queries(len(of), oc.kv_heads * rows, window + rows)
    qd = to_dev(q)
    out = torch.full(q.shape, 7.0, device="cuda")
    pk.packkv_attention_window(cache, qd, SCALE, out, window, sinks=sinks, queries=n_queries)
    got = out.double().cpu().numpy()
    ref, terms = reference(oc, of, q, window, sinks, n_queries)
    assert_within_terms(got, ref, terms, f"window {window} sinks {sinks}")
    off = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert off <= norm, off
    want = out.clone()
    for _ in range(2):  # the same bits every time
        out.zero_()
        pk.packkv_attention_window(cache, qd, SCALE, out, window, sinks=sinks, queries=n_queries)
        assert torch.equal(out, want)
    assert pk.packkv_get_status(cache) == 0


EVEN = [(2, False, 1, 1, False), (2, True, 2, 1, True), (3, False, 1, 1, False), (3, False, 2, 2, True),
        (3, True, 4, 2, False), (4, True, 1, 1, True), (4, True, 8, 4, False), (2, False, 4, 1, True),
        (4, False, 16, 4, True), (3, True, 2, 1, True), (2, True, 1, 1, False)]


@pytest.mark.parametrize("bits,structured,rows,n_queries,table", EVEN)
def test_even_split(pk, bits, structured, rows, n_queries, table):
    cache, oc = many(pk, bits, structured, 100 + bits, table=table)
    of = [b % 2 for b in range(cache.batch)]
    norm = 1e-5 if structured else 2e-6
    for window, sinks in ((1000, 0), (140, 2)):
        _check(pk, cache, oc, of, rows, n_queries, window, sinks, norm)
    # the block between the first tokens and the window is given up: with four queries the
    # window of 130 reaches back to token 390 - 4 - 130 + 1 = 257, the start of block 2 is 256
    first = [1] * cache.batch
    pk.packkv_free_blocks(cache, first, [1] * cache.batch)
    _check(pk, cache, oc, of, rows, n_queries, 130, 2, norm)


@pytest.mark.parametrize("bits", [2, 3, 4])
def test_scores_carry_four_digits(pk, bits):
    """The inputs of test_window_digits_cpu in the cluster form."""
    k, v, _ = synth.small_case(90, 1, 1, 1, 384)
    oc = O.RaggedOracleCache(1, 1, 3, bits)
    oc.encode_blocks_ragged(k, v, 3)
    cache = pk.PackKVCache(1, 1, 3, bits, ragged=True, keep_perm=True)
    pk.packkv_encode_block(cache, to_dev(k), to_dev(v), 3)
    q = queries(1, 16, 1)
    out = torch.empty(q.shape, device="cuda")
    pk.packkv_attention_window(cache, to_dev(q), SCALE, out, 1000)
    ref, _ = reference(oc, [0], q, 1000, 0, 1)
    off = np.linalg.norm(out.double().cpu().numpy() - ref) / np.linalg.norm(ref)
    assert off <= 2e-6, off
