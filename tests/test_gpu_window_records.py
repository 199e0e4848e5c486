"""Windowed attention over index entries that name no record (the tokens of such a block are
left out, whichever of its two entries is the bad one) and with queries that are not finite,
in both forms of the kernel.

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


def _wild(pk, cache, oc, of, rows, n_queries, window, places, value):
    """Rows whose q holds `value` are NaN where they see a token and zero where not; the
    others keep their bits."""
    q = queries(len(of), oc.kv_heads * rows, 7)
    clean, out = (torch.empty(q.shape, device="cuda") for _ in range(2))
    pk.packkv_attention_window(cache, to_dev(q), SCALE, clean, window, queries=n_queries)
    hit = np.zeros(q.shape[:2], bool)
    for b, r, c in places:
        q[b, r, c] = value
        hit[b, r] = True
    pk.packkv_attention_window(cache, to_dev(q), SCALE, out, window, queries=n_queries)
    hit = torch.from_numpy(hit).cuda()
    g = rows // n_queries
    position = torch.arange(q.shape[1], device="cuda") // g % n_queries - n_queries
    tokens = torch.tensor([oc.seq_tokens(s) for s in of], device="cuda")
    sees = tokens[:, None] + position[None] >= 0
    assert torch.equal(out[~hit], clean[~hit])
    assert torch.all(torch.isnan(out[hit & sees])) and torch.all(out[hit & ~sees] == 0)
    assert pk.packkv_get_status(cache) == 0


@pytest.mark.parametrize("structured", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_infinite_queries(pk, value, structured):
    """An infinity in a query shows as NaN, whatever its sign and the keys', over records
    and over tail tokens; rows of the same chunk keep their bits."""
    cache, oc = _caches(pk, 4, 2, 4, [300, 256, 1, 3], 60, structured)
    for rows, n_queries, window in ((1, 1, 1), (4, 4, 2), (8, 2, 400), (2, 1, 130)):
        places = {(b, r, (37 * (b + r)) % 128) for b in range(4) for r in range(b % 2, 2 * rows, 3)}
        _wild(pk, cache, oc, range(4), rows, n_queries, window, places, value)


@pytest.mark.parametrize("structured", [False, True])
def test_infinite_queries_in_the_even_split(pk, structured):
    cache, oc = many(pk, 2, structured, 61)
    of = [b % 2 for b in range(cache.batch)]
    for rows, n_queries, value in ((1, 1, float("-inf")), (4, 2, float("inf")), (2, 2, float("nan"))):
        places = {(b, r, (b + 3 * r) % 128) for b in range(0, cache.batch, 2) for r in range(0, 8 * rows, 3)}
        _wild(pk, cache, oc, of, rows, n_queries, 300, places, value)
