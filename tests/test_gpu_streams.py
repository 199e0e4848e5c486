"""Calls that bring no workspace, on streams of their own: the first call on a new cache behind
a busy current stream, and calls on two streams at once, give the bits of calls one by one."""
import pytest
import torch

from parity_util import to_dev
from window_cases import SCALE, many, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_gemv_packkv_b200 import packkv
    return packkv


def _busy():
    """Some milliseconds of work on the current stream."""
    x = torch.ones((8192, 8192), dtype=torch.float16, device="cuda")
    for _ in range(10):
        x = x @ x * 1e-4
    return x


def _calls(pk, cache, q, p):
    """The calls that need a workspace, by name: f(out, stream)."""
    def compact(out, stream):
        pk.packkv_compact(out, cache, stream=stream)
    def pv(out, stream):
        pk.packkv_pv_gemv(cache, p, out, stream=stream)
    def attention(out, stream):
        pk.packkv_attention_decode(cache, q, SCALE, out, stream=stream)
    def window(out, stream):
        pk.packkv_attention_window(cache, q, SCALE, out, 300, stream=stream)
    return {"pv": pv, "attention": attention, "window": window, "compact": compact}


def _target(pk, cache, name, q):
    if name != "compact":
        return torch.zeros(q.shape, device="cuda")
    dst = pk.PackKVCache(cache.batch, cache.kv_heads, 3, 4, ragged=True, keep_perm=True)
    dst.k_arena.zero_()
    dst.v_arena.zero_()
    return dst


def _bits(out):
    if isinstance(out, torch.Tensor):
        return [out.clone()]
    return [x.clone() for x in (out.k_index, out.v_index, out.k_arena, out.v_arena, out.perm, out.ctrl)]


@pytest.mark.parametrize("name", ["pv", "attention", "window", "compact"])
def test_default_workspaces(pk, name):
    cache, _ = many(pk, 4, False, 80)
    qs = [to_dev(queries(cache.batch, 8, s)) for s in (1, 2)]
    p = torch.rand((cache.batch, 8, 400), device="cuda")
    calls = [_calls(pk, cache, q, p * (i + 1))[name] for i, q in enumerate(qs)]
    want = []
    for call, q in zip(calls, qs):
        out = _target(pk, cache, name, q)
        call(out, None)
        want.append(_bits(out))
    cache._ws.clear()
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [_target(pk, cache, name, q) for q in qs]
    torch.cuda.synchronize()
    keep = _busy()
    calls[0](outs[0], streams[0])           # the first call with a workspace, behind a busy stream
    streams[0].synchronize()
    assert all(torch.equal(a, b) for a, b in zip(_bits(outs[0]), want[0]))
    torch.cuda.synchronize()
    for _ in range(20):
        for call, out, stream in zip(calls, outs, streams):
            call(out, stream)
    torch.cuda.synchronize()
    for out, bits in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(_bits(out), bits))
    assert len(cache._ws) == 2 and keep is not None
