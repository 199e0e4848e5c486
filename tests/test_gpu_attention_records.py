"""Fused attention over index entries that name no record: the tokens of such a block are left
out, whichever of its two entries is the bad one.  Tolerance as in test_gpu_attention.
"""
import pytest
import torch

from parity_util import assert_within_terms, to_dev
from test_gpu_window import _caches
from window_cases import SCALE, queries, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_gemv_packkv_b200 import packkv
    return packkv


@pytest.mark.parametrize("structured", [False, True])
@pytest.mark.parametrize("tensors", ["k", "v", "kv"])
@pytest.mark.parametrize("bits,group", [(4, 1), (3, 4), (2, 16)])
def test_blocks_with_a_bad_entry_are_left_out(pk, bits, group, tensors, structured):
    cache, oc = _caches(pk, 2, 2, bits, [500, 300], 70, structured)
    places = {(0, 1, 1), (0, 0, 2), (1, 0, 0), (1, 0, 1)}
    q = queries(2, 2 * group, 3)
    ref, terms = reference(oc, [0, 1], q, 1 << 30, 0, 1, without=places)
    for entry in ((-1, 0), (7, 3)):  # freed, and a length that no record has
        for name in tensors:
            for b, h, j in places:
                getattr(cache, f"{name}_index")[b, h, j] = torch.tensor(entry, dtype=torch.int32)
        out = torch.full(q.shape, 7.0, device="cuda")
        pk.packkv_attention_decode(cache, to_dev(q), SCALE, out)
        assert_within_terms(out.double().cpu().numpy(), ref, terms, f"{tensors} {entry}")
        assert pk.packkv_get_status(cache) == pk.DEV_BAD_RECORD
