"""The oracle's definitions of the operators around the cache, pinned on small cases that
can be checked by hand or by another route (complex numbers, explicit loops)."""
import numpy as np
import pytest

import oracle as O


@pytest.mark.parametrize("layout", [O.ROPE_HALF, O.ROPE_INTERLEAVED])
@pytest.mark.parametrize("rot", [0, 2, 66, 96, 128])
def test_rotation_is_a_complex_product(layout, rot):
    rng = np.random.default_rng(rot + layout)
    x = rng.standard_normal((3, 128))
    pos = np.array([0, 5, 1_000_003])
    freq = O.rope_frequencies(rot, 10000.0)
    y = O.norm_rope(x, pos, freq, layout, amplitude=1.5)
    n = rot // 2
    a = np.arange(n) if layout == O.ROPE_HALF else 2 * np.arange(n)
    b = a + n if layout == O.ROPE_HALF else a + 1
    z = (x[:, a] + 1j * x[:, b]) * np.exp(1j * pos[:, None] * freq) * 1.5
    assert np.allclose(y[:, a], z.real, atol=1e-12) and np.allclose(y[:, b], z.imag, atol=1e-12)
    rest = np.setdiff1d(np.arange(128), np.concatenate([a, b]))
    assert np.array_equal(y[:, rest], x[:, rest])


def test_frequencies_and_their_scalings():
    f = O.rope_frequencies(128, 10000.0)
    assert f[0] == 1.0 and np.isclose(f[32], 0.01) and len(f) == 64
    assert np.allclose(O.rope_frequencies(128, 10000.0, O.ROPE_SCALE_LINEAR, 4.0), f / 4)
    base = O.rope_frequencies(128, 10000.0, O.ROPE_SCALE_BASE, 4.0)
    assert base[0] == 1.0 and np.isclose(base[-1], f[-1] / 4)      # the slowest pair is interpolated whole
    parts = O.rope_frequencies(128, 10000.0, O.ROPE_SCALE_PARTS, 4.0, 8192, 1.0, 32.0)
    turns = 8192 * f / (2 * np.pi)
    assert np.allclose(parts[turns >= 32], f[turns >= 32]) and np.allclose(parts[turns <= 1], f[turns <= 1] / 4)
    assert np.all(np.diff(parts) < 0)


def test_norm():
    x = np.arange(128.0)[None]
    w = np.linspace(0.5, 1.5, 128)
    y = O.norm_rope(x, np.zeros(1), O.rope_frequencies(0, 10000.0), O.ROPE_HALF, eps=1e-6, weight=w)
    assert np.allclose(y, x / np.sqrt(np.mean(x ** 2) + 1e-6) * w)
    assert np.array_equal(O.norm_rope(np.zeros((1, 128)), np.zeros(1), [], 0, eps=1e-6), np.zeros((1, 128)))


def test_window_mask_by_loops():
    for t, s, w, n0 in [(1, 1, 1, 0), (5, 2, 2, 1), (9, 3, 4, 2), (3, 5, 2, 1), (7, 1, 100, 3)]:
        m = O.window_mask(t, s, w, n0)
        for a in range(s):
            p = t - s + a
            for i in range(t):
                assert m[a, i] == (i <= p and (i > p - w or i < n0))
        if s > t:
            assert not m[:s - t].any()


def test_window_attention_over_everything_is_plain_attention():
    """A window that holds every token, one query: the cache's full attention."""
    rng = np.random.default_rng(0)
    B, H, G = 2, 2, 2
    oc = O.RaggedOracleCache(B, H, 3, 4)
    k = rng.standard_normal((B, H, 256, 128)).astype(np.float16)
    v = rng.standard_normal((B, H, 256, 128)).astype(np.float16)
    oc.encode_blocks_ragged(k, v, 2)
    for _ in range(5):
        oc.append_token_ragged(k[:, :, 3], v[:, :, 3], [0])
    q = rng.standard_normal((B, H * G, 128)).astype(np.float16)
    want, _ = O.ragged_attention(oc, q, 0.1)
    got, _ = O.window_attention(oc, q, 0.1, 1000, 0, 1)
    assert np.allclose(got, want, atol=1e-12)


def test_compaction_keeps_shared_records_once():
    index = np.zeros((2, 1, 3, 2), np.int64)
    index[0, 0] = [(10, 65), (75, 70), (0xFFFFFFFF, 0)]
    index[1, 0] = [(75, 70), (200, 66), (0, 0)]
    arena = bytes(np.arange(300 * 16, dtype=np.uint32).astype(np.uint8))
    entries, out = O.compacted(index, arena, [3, 2], lambda b, j: (b, j))
    assert entries == {(0, 0, 0): (0, 65), (0, 0, 1): (65, 70), (0, 0, 2): (0xFFFFFFFF, 0),
                       (1, 0, 0): (65, 70), (1, 0, 1): (135, 66)}
    assert out == arena[160:160 + 135 * 16] + arena[3200:3200 + 66 * 16]
