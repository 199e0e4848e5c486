"""Windowed attention over index entries that name no record: the tokens of such a block
are left out, whichever of its two entries is the bad one, in both forms of the kernel.

Tolerance as in test_gpu_window: 1e-3 * sum|terms| per element and a relative 2-norm of 1e-5.
A block that is left out by its values alone would scale a row down by the block's weight,
about a third here.
"""
import numpy as np
import pytest
import torch

from parity_util import assert_within_terms, to_dev
from test_gpu_window import _caches
from window_cases import SCALE, many, queries, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_gemv_packkv_b200 import packkv
    return packkv


def _invalidate(cache, tensors, places, entry=(-1, 0)):
    for name in tensors:
        index = getattr(cache, f"{name}_index")
        for b, h, j in places:
            index[b, h, j] = torch.tensor(entry, dtype=torch.int32)


def _check(pk, cache, oc, of, rows, n_queries, window, sinks, without):
    q = queries(len(of), oc.kv_heads * rows, window)
    out = torch.full(q.shape, 7.0, device="cuda")
    pk.packkv_attention_window(cache, to_dev(q), SCALE, out, window, sinks=sinks, queries=n_queries)
    got = out.double().cpu().numpy()
    ref, terms = reference(oc, of, q, window, sinks, n_queries, without=without)
    assert_within_terms(got, ref, terms, f"window {window} sinks {sinks}")
    assert np.linalg.norm(got - ref) <= 1e-5 * np.linalg.norm(ref)


@pytest.mark.parametrize("structured", [False, True])
@pytest.mark.parametrize("tensors", ["k", "v", "kv"])
@pytest.mark.parametrize("form", ["clusters", "even"])
def test_blocks_with_a_bad_entry_are_left_out(pk, form, tensors, structured):
    if form == "clusters":
        cache, oc = _caches(pk, 2, 2, 4, [500, 300], 50, structured)
        of, places = [0, 1], {(0, 1, 1), (0, 0, 2), (1, 0, 0), (1, 0, 1)}
    else:
        cache, oc = many(pk, 4, structured, 51)
        of = [b % 2 for b in range(cache.batch)]
        places = {(b, h, (b + h) % 3) for b in range(0, cache.batch, 3) for h in range(0, 8, 2)}
    for entry in ((-1, 0), (7, 3)):  # freed, and a length that no record has
        _invalidate(cache, tensors, places, entry)
        for rows, n_queries, window, sinks in ((1, 1, 100000, 0), (4, 2, 100000, 0), (2, 1, 270, 4)):
            _check(pk, cache, oc, of, rows, n_queries, window, sinks, places)
            assert pk.packkv_get_status(cache) == pk.DEV_BAD_RECORD


def test_a_row_that_sees_only_bad_blocks_is_zero(pk):
    cache, oc = _caches(pk, 1, 2, 3, [256], 52)
    _invalidate(cache, "v", [(0, 0, 0), (0, 0, 1)])
    q = to_dev(queries(1, 4, 1))
    out = torch.full((1, 4, 128), 7.0, device="cuda")
    pk.packkv_attention_window(cache, q, SCALE, out, 300)
    assert torch.all(out[0, :2] == 0) and torch.all(out[0, 2:] != 0)
    assert pk.packkv_get_status(cache) == pk.DEV_BAD_RECORD
