"""The cache's own workspaces on the host: one per stream, allocated on that stream, never
written by the binding (a fill on one stream could land behind a kernel's sums on another)."""
import contextlib

import pytest
import torch


@pytest.fixture(scope="module")
def pk():
    from decode_gemv_packkv_b200 import build
    build.build()
    from decode_gemv_packkv_b200 import packkv
    return packkv


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("name,args", [("workspace", (2,)), ("attention_workspace", (2,)), ("window_workspace", (2,)),
                                       ("compact_workspace", ())])
def test_a_workspace_belongs_to_its_stream(pk, monkeypatch, name, args):
    cache = pk.PackKVCache(1, 1, 2, 4, device="cpu")
    current, made = [], []
    real = torch.empty

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(*a, **kw):
        made.append(current[-1] if current else None)
        return real(*a, **kw)

    def written(*a, **kw):
        raise AssertionError("a workspace is not initialised")

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)
    for fill in ("zeros", "full", "ones", "zeros_like"):
        monkeypatch.setattr(torch, fill, written)
    a, b = Stream(17), Stream(18)
    get = getattr(cache, name)
    first, second, third = get(*args, stream=a), get(*args, stream=b), get(*args)
    assert made == [a, b, None]
    assert len({t.data_ptr() for t in (first, second, third)}) == 3
    assert get(*args, stream=Stream(17)) is first and get(*args) is third and len(made) == 3
