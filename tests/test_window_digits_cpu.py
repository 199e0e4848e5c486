"""What the tests of windowed attention can tell apart (host only): with three digits of q' the
output is off by more than the 2e-6 that the GPU tests allow, with four by a tenth of it."""
import numpy as np
import pytest

import oracle as O
from decode_gemv_packkv_b200 import synth
from window_cases import queries, whole_softmax_with_digits


@pytest.mark.parametrize("bits", [2, 3, 4])
def test_three_digits_would_show(bits):
    k, v, _ = synth.small_case(90, 1, 1, 1, 384)
    oc = O.RaggedOracleCache(1, 1, 3, bits)
    oc.encode_blocks_ragged(k, v, 3)
    q = queries(1, 16, 1)[0]
    exact = whole_softmax_with_digits(oc, q, None)
    off = {d: np.linalg.norm(whole_softmax_with_digits(oc, q, d) - exact) / np.linalg.norm(exact) for d in (3, 4)}
    assert off[3] > 2 * 2e-6 and off[4] < 2e-7, off
