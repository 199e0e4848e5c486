"""packkv_norm_rope and packkv_append_norm_rope against the oracle's 64-bit definition.

Tolerance.  The kernels compute in fp32 and round once to fp16, so an output y is off by
at most half an fp16 step, |y| * 2^-11 (or 2^-25, half the smallest step, near zero), plus
the fp32 error of y.  With N = |a| + |b| of the pair (times the amplitude): the angle is
off by at most 2^-24 half turns = 2^-24 pi, i.e. N * 2^-22; the sine, cosine, products and
sum by a few 2^-24 N; the norm's factor by about 8 * 2^-24 (a sum of 128 squares in fp32,
partly as a tree, rsqrt within 2 ulp, two products).  Together below N * 2^-20.
"""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SCALED = {"none": dict(), "linear": dict(scaling=1, factor=4.0), "base": dict(scaling=2, factor=8.0),
          "parts": dict(scaling=3, factor=8.0, original_tokens=8192.0, low=1.0, high=32.0)}


@pytest.fixture(scope="module")
def pk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_gemv_packkv_b200 import packkv
    return packkv


def _check(got, x, pos, freq, layout, amplitude, eps, w, what):
    ref = O.norm_rope(x, pos, freq, layout, amplitude, eps, w)
    # N of the pair of every channel, of the normed head
    y = np.abs(O.norm_rope(x, np.zeros_like(pos), [], layout, 1.0, eps, w))
    n = len(freq)
    a = np.arange(n) if layout == O.ROPE_HALF else 2 * np.arange(n)
    b = a + n if layout == O.ROPE_HALF else a + 1
    N = y.copy()
    N[..., a] = N[..., b] = (y[..., a] + y[..., b]) * abs(amplitude)
    tol = np.maximum(np.abs(ref) * 2.0 ** -11, 2.0 ** -25) * (1 + 2.0 ** -10) + N * 2.0 ** -20
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= tol), (what, float((err / tol).max()))


def _inputs(B, T, hq, hkv, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = (1.5 * torch.randn(B, T, hq + 2 * hkv, 128, generator=g)).to(DT[dt])
    return x, 1 + 0.2 * torch.randn(128, generator=g), 1 + 0.2 * torch.randn(128, generator=g)


CASES = [  # B, T, hq, hkv, dtype, norm, layout, rot, scaling, far
    (1, 1, 1, 1, "fp16", False, 0, 128, "none", False),
    (2, 5, 3, 2, "bf16", True, 0, 128, "parts", True),
    (1, 9, 4, 1, "fp32", True, 1, 128, "linear", False),
    (3, 4, 2, 2, "fp16", True, 1, 96, "base", True),
    (1, 7, 17, 1, "bf16", False, 0, 64, "none", True),
    (2, 3, 1, 3, "fp32", True, 0, 66, "linear", True),     # pairs that no vector access fits
    (1, 6, 2, 1, "fp16", True, 0, 2, "base", False),
    (1, 6, 2, 1, "bf16", True, 1, 126, "none", False),
    (1, 2, 5, 5, "fp32", True, 0, 0, "none", False),       # norm alone
]


@pytest.mark.parametrize("case", CASES)
def test_norm_rope(pk, case):
    B, T, hq, hkv, dt, norm, layout, rot, scaling, far = case
    x, wq, wk = _inputs(B, T, hq, hkv, dt, 11)
    d = x.cuda()
    rope = pk.Rope(rot, layout, 10000.0, amplitude=1.25, **SCALED[scaling])
    pos = np.tile(100 + np.arange(T), (B, 1))
    positions = None
    if far:
        positions = torch.randint(-1000, 1 << 30, (B, T), generator=torch.Generator().manual_seed(3)).int()
        positions[0, 0] = (1 << 31) - 1
        pos = positions.numpy()
        positions = positions.cuda()
    outs = [torch.full((B, h, T, 128), 7.0, dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv)]
    eps = 1e-5 if norm else None
    pk.packkv_norm_rope(rope, d[:, :, :hq], d[:, :, hq:hq + hkv], d[:, :, hq + hkv:], *outs,
                        q_weight=wq.cuda() if norm else None, k_weight=wk.cuda() if norm else None, eps=eps,
                        positions=positions, first=100)
    freq = O.rope_frequencies(rot, 10000.0, **SCALED[scaling])
    xd = x.double().numpy()
    p = pos[:, None, :]
    heads = np.transpose(xd, (0, 2, 1, 3))
    _check(outs[0], heads[:, :hq], np.broadcast_to(p, heads[:, :hq].shape[:3]), freq, layout, 1.25, eps,
           wq.numpy() if norm else None, "q")
    _check(outs[1], heads[:, hq:hq + hkv], np.broadcast_to(p, heads[:, :hkv].shape[:3]), freq, layout, 1.25, eps,
           wk.numpy() if norm else None, "k")
    assert torch.equal(outs[2].cpu(), x[:, :, hq + hkv:].permute(0, 2, 1, 3).half())


@pytest.mark.parametrize("first", [0, 1, (1 << 40) + 12345, -17])
def test_positions_from_first(pk, first):
    """A far first position turns as the wrapped angle says (fp64 holds first * f to 2^-12
    of a turn at 2^40, so the reference takes the angle in exact steps of the table)."""
    x, _, _ = _inputs(1, 3, 1, 1, "fp32", 2)
    rope = pk.Rope(128, pk.ROPE_HALF)
    out = torch.empty((1, 1, 3, 128), dtype=torch.float16, device="cuda")
    pk.packkv_norm_rope(rope, x[:, :, :1].cuda(), None, None, q_out=out, first=first)
    xs = x[0, :, 0].double().numpy()
    for t in range(3):
        turn = np.array([((first + t) * int(rope.s.turn[i])) % (1 << 64) / 2.0 ** 64 for i in range(64)])
        c, s = np.cos(2 * np.pi * turn), np.sin(2 * np.pi * turn)
        a, b = xs[t, :64], xs[t, 64:]
        ref = np.concatenate([a * c - b * s, b * c + a * s])
        N = np.abs(np.concatenate([a, a])) + np.abs(np.concatenate([b, b]))
        err = np.abs(out[0, 0, t].double().cpu().numpy() - ref)
        assert np.all(err <= np.maximum(np.abs(ref) * 2.0 ** -11, 2.0 ** -25) * (1 + 2.0 ** -10) + N * 2.0 ** -20)


def test_keys_alone_and_several_launch_shapes(pk):
    """k and v without q; prompts short and long enough for every number of tokens per CTA
    give the same bits per token."""
    rope = pk.Rope(128, pk.ROPE_HALF)
    B, T, h = 2, 1800, 3
    x = torch.randn(B, T, 2 * h, 128, device="cuda").half()
    full = [torch.empty((B, h, T, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    pk.packkv_norm_rope(rope, None, x[:, :, :h], x[:, :, h:], None, *full, eps=1e-6, first=7)
    assert torch.equal(full[1], x[:, :, h:].transpose(1, 2))
    for t0, t1 in ((0, 1), (5, 105), (900, 1250)):
        part = [torch.empty((B, h, t1 - t0, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
        pk.packkv_norm_rope(rope, None, x[:, t0:t1, :h], x[:, t0:t1, h:], None, *part, eps=1e-6, first=7 + t0)
        assert torch.equal(part[0], full[0][:, :, t0:t1]) and torch.equal(part[1], full[1][:, :, t0:t1])


def test_strides_and_unaligned_rows(pk):
    """Head-major rows, a batch stride of its own, and data that starts one element off a
    vector: the same bits as from the fused projection."""
    B, T, hq, hkv = 2, 6, 4, 2
    x, wq, wk = _inputs(B, T, hq, hkv, "bf16", 5)
    d = x.cuda()
    rope = pk.Rope(128, pk.ROPE_INTERLEAVED)

    def call(q, k, v):
        outs = [torch.empty((B, h, T, 128), dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv)]
        pk.packkv_norm_rope(rope, q, k, v, *outs, q_weight=wq.cuda(), k_weight=wk.cuda(), eps=1e-6)
        return outs

    want = call(d[:, :, :hq], d[:, :, hq:hq + hkv], d[:, :, hq + hkv:])
    hm = d.transpose(1, 2).contiguous().transpose(1, 2)
    got = call(hm[:, :, :hq], hm[:, :, hq:hq + hkv], hm[:, :, hq + hkv:])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    buf = torch.zeros(d.numel() + 1, dtype=torch.bfloat16, device="cuda")
    off = buf[1:].view(d.shape)
    off.copy_(d)
    got = call(off[:, :, :hq], off[:, :, hq:hq + hkv], off[:, :, hq + hkv:])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    rev = d.flip(1).contiguous().flip(1)  # (torch flips copy: same values, plain strides)
    got = call(rev[:, :, :hq], rev[:, :, hq:hq + hkv], rev[:, :, hq + hkv:])
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_infinities_stay_in_their_pair_and_unrotated_channels(pk):
    """An infinity spoils its own pair only; channels past rot_dim pass as they are."""
    x = torch.ones(1, 1, 1, 128)
    x[0, 0, 0, 100] = float("inf")
    x[0, 0, 0, 3] = float("nan")
    for layout, pair in ((pk.ROPE_HALF, (3, 35)), (pk.ROPE_INTERLEAVED, (2, 3))):
        out = torch.empty((1, 1, 1, 128), dtype=torch.float16, device="cuda")
        pk.packkv_norm_rope(pk.Rope(64, layout), x.cuda(), None, None, q_out=out, first=1)
        bad = torch.nonzero(~torch.isfinite(out[0, 0, 0].float())).flatten().tolist()
        assert bad == sorted(list(pair) + [100]), layout
        assert torch.all(out[0, 0, 0, 64:100] == 1) and torch.all(out[0, 0, 0, 101:] == 1)
    big = torch.full((1, 1, 1, 128), 1e6)
    out = torch.empty((1, 1, 1, 128), dtype=torch.float16, device="cuda")
    pk.packkv_norm_rope(None, big.cuda(), None, None, q_out=out)
    assert torch.all(torch.isinf(out))


@pytest.mark.parametrize("ragged", [False, True])
def test_append_norm_rope_grows_the_cache(pk, ragged):
    """Appended step by step through a block boundary, the cache's records, tails and the
    q rows are those of packkv_norm_rope followed by packkv_append_token(_masked)."""
    B, hq, hkv, steps = 3, 4, 2, 131
    rope = pk.Rope(96, pk.ROPE_HALF, 10000.0, scaling=pk.ROPE_SCALE_LINEAR, factor=2.0)
    x, wq, wk = _inputs(B, steps, hq, hkv, "bf16", 9)
    x = x.cuda()
    wq, wk = wq.cuda(), wk.cuda()
    a = pk.PackKVCache(B, hkv, 2, 4, ragged=ragged, keep_perm=True)
    b = pk.PackKVCache(B, hkv, 2, 4, ragged=ragged, keep_perm=True)
    held = [0] * B
    for t in range(steps):
        on = [True] * B if not ragged else [True, t % 2 == 0, t < 40]
        q, k, v = x[:, t, :hq], x[:, t, hq:hq + hkv], x[:, t, hq + hkv:]
        q_out = torch.full((B, hq, 128), 7.0, dtype=torch.float16, device="cuda")
        pk.packkv_append_norm_rope(a, rope, q, k, v, q_out, q_weight=wq, k_weight=wk, eps=1e-6,
                                   active=on if ragged else None)
        outs = [torch.empty((B, h, 1, 128), dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv)]
        pk.packkv_norm_rope(rope, q[:, None], k[:, None], v[:, None], *outs, q_weight=wq, k_weight=wk, eps=1e-6,
                            positions=torch.tensor(held, dtype=torch.int32, device="cuda")[:, None])
        for s in range(B):
            assert torch.equal(q_out[s], outs[0][s, :, 0]) if on[s] else torch.all(q_out[s] == 7.0)
        kk, vv = outs[1][:, :, 0].contiguous(), outs[2][:, :, 0].contiguous()
        if ragged:
            pk.packkv_append_token_masked(b, kk, vv, on)
        else:
            pk.packkv_append_token(b, kk, vv)
        held = [h + o for h, o in zip(held, on)]
    assert a.seq_blocks == b.seq_blocks and a.seq_tail == b.seq_tail and max(a.seq_blocks) == 1
    for name in ("k_index", "v_index", "k_tail", "v_tail", "perm", "ctrl"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    used = a.arena_used()
    assert torch.equal(a.k_arena[:used[0]], b.k_arena[:used[0]])
    assert torch.equal(a.v_arena[:used[1]], b.v_arena[:used[1]])
    assert pk.packkv_get_status(a) == 0


def test_append_to_many_ragged_sequences(pk):
    B = 70                                   # past the small plans of 64 sequences
    x, _, _ = _inputs(B, 1, 1, 1, "fp32", 4)
    d = x[:, 0].cuda()
    cache = pk.PackKVCache(B, 1, 3, 4, ragged=True)
    held = [(17 * b) % 300 for b in range(B)]
    cache.set_lengths([t // 128 for t in held], [t % 128 for t in held])
    on = [b % 5 != 3 for b in range(B)]
    q_out = torch.zeros((B, 1, 128), dtype=torch.float16, device="cuda")
    rope = pk.Rope()
    pk.packkv_append_norm_rope(cache, rope, d[:, :1], d[:, 1:2], d[:, 2:], q_out, active=on)
    want = [torch.empty((B, 1, 1, 128), dtype=torch.float16, device="cuda") for _ in range(3)]
    pos = torch.tensor(held, dtype=torch.int32, device="cuda")[:, None]
    pk.packkv_norm_rope(rope, d[:, None, :1], d[:, None, 1:2], d[:, None, 2:], *want, positions=pos)
    for b in range(B):
        if on[b]:
            assert torch.equal(q_out[b], want[0][b, :, 0])
            assert torch.equal(cache.k_tail[b, :, held[b] % 128], want[1][b, :, 0])
        else:
            assert torch.all(q_out[b] == 0) and torch.all(cache.k_tail[b] == 0)
    grown = [128 * n + t for n, t in zip(cache.seq_blocks, cache.seq_tail)]
    assert grown == [h + o for h, o in zip(held, on)]


def test_append_in_a_graph(pk):
    """Captured and replayed with other inputs: the position is the captured one, the tail
    slot takes the new token."""
    B, hq, hkv = 2, 2, 1
    cache = pk.PackKVCache(B, hkv, 1, 4)
    cache.set_lengths(0, 17)
    rope = pk.Rope()
    x = torch.randn(B, hq + 2 * hkv, 128, device="cuda", dtype=torch.float16)
    q_out = torch.empty((B, hq, 128), dtype=torch.float16, device="cuda")
    args = (x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], q_out)
    pk.packkv_append_norm_rope(cache, rope, *args)
    cache.set_lengths(0, 17)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.packkv_append_norm_rope(cache, rope, *args)
    x.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    want = [torch.empty((B, h, 1, 128), dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv)]
    pk.packkv_norm_rope(rope, x[:, None, :hq], x[:, None, hq:hq + hkv], x[:, None, hq + hkv:], *want, first=17)
    assert torch.equal(q_out, want[0][:, :, 0])
    assert torch.equal(cache.k_tail[:, :, 17], want[1][:, :, 0])
    assert torch.equal(cache.v_tail[:, :, 17], want[2][:, :, 0])


def test_refusals(pk):
    x = torch.zeros(1, 1, 2, 128, device="cuda")
    out = torch.empty((1, 2, 1, 128), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        pk.packkv_norm_rope(None, x.double(), None, None, q_out=out)
    with pytest.raises(ValueError):
        pk.packkv_norm_rope(None, x, x, None, q_out=out, k_out=out)
    with pytest.raises(ValueError):
        pk.packkv_norm_rope(None, x[..., :64], None, None, q_out=out)
    with pytest.raises(ValueError):
        pk.packkv_norm_rope(None, x, None, None, q_out=out.float())
    with pytest.raises(ValueError):
        pk.packkv_norm_rope(None, x, None, None, q_out=out, q_weight=torch.ones(128, device="cuda"))
    with pytest.raises(ValueError):
        pk.packkv_norm_rope(None, x, None, None, q_out=out, positions=torch.zeros(1, 1, device="cuda"))
    cache = pk.PackKVCache(1, 1, 1, 4)
    with pytest.raises(pk.PackKVError) as e:
        pk.packkv_append_norm_rope(cache, None, None, x[:, 0, :1], x[:, 0, :1], active=[True])
    assert e.value.status == pk.ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        pk.packkv_append_norm_rope(cache, None, None, x[:, 0], x[:, 0])


@pytest.mark.parametrize("shape", [(2, 0), (0, 3)])
def test_no_tokens(pk, shape):
    """Tensors without elements have no address; a call on them does nothing."""
    B, T = shape
    x = torch.empty((B, T, 3, 128), dtype=torch.float16, device="cuda")
    out = torch.empty((B, 3, T, 128), dtype=torch.float16, device="cuda")
    pk.packkv_norm_rope(pk.Rope(), x, x, x, out, out, out, eps=1e-6)
    with pytest.raises(ValueError):
        pk.packkv_norm_rope(None, x, None, None, q_out=out.float())
