"""packkv_norm_rope through the C call with strides of either sign (torch tensors have none
below zero): the rows of a flipped tensor, bit for bit."""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_gemv_packkv_b200 import packkv
    return packkv


@pytest.mark.parametrize("dtype,tag,pad", [(torch.bfloat16, 1, 0), (torch.float32, 2, 0), (torch.float16, 0, 1)])
@pytest.mark.parametrize("flip", [f for n in range(1, 4) for f in itertools.combinations(range(3), n)])
def test_negative_strides(pk, dtype, tag, pad, flip):
    """flip: of batch, tokens, heads; pad 1: rows that no vector access fits."""
    B, T, H = 3, 5, 4
    g = torch.Generator().manual_seed(7)
    row = 128 + pad
    x = torch.randn(3, B, T, H, row, generator=g).to(dtype).cuda()   # q, k, v
    rope = pk.Rope(96, pk.ROPE_HALF)
    strides, size = [T * H * row, H * row, row], [B, T, H]
    start = sum(strides[d] * (size[d] - 1) for d in flip)
    signed = [-s if d in flip else s for d, s in enumerate(strides)]
    for d in range(3):  # every element stays inside its tensor
        assert 0 <= start + sum(min(0, signed[e] * (size[e] - 1)) for e in range(3))
    rows = []
    for t in x:
        rows += [t.data_ptr() + start * t.element_size(), *signed]
    outs = [torch.full((B, H, T, 128), 7.0, dtype=torch.float16, device="cuda") for _ in range(3)]
    want = [torch.empty_like(o) for o in outs]
    heads = pk._HEADS.pack(tag, H, H, 1e-5, *rows, 0, 0)
    status = pk._lib.packkv_norm_rope(rope.ref, heads, B, T, None, 3, *[o.data_ptr() for o in outs],
                                      torch.cuda.current_stream().cuda_stream)
    assert status == pk.OK
    flipped = [t.flip(flip)[..., :128] for t in x]
    pk.packkv_norm_rope(rope, *flipped, *want, eps=1e-5, first=3)
    for got, ref in zip(outs, want):
        assert torch.equal(got, ref)
