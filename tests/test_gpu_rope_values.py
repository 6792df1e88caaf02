"""lora_rope: what passes through keeps its bits; the way back.

The way back in fp32, u = 2^-24, S = |a| + |b| of a pair, f the factor: the forward turn is off by 8 u f S
(tests/test_gpu_rope.py) and a rounding, at most 9 u f S; its two outputs together are at most 2 f S.  Turned back with
1 / f, both errors enter with at most 1 / f (18 u S), the turn's own is 8 u (2 f S) / f, 1 / f itself and the output are
rounded: 36 u S together, and f^2 times that with f both ways."""

import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

from .gpu_util import log

pytestmark = pytest.mark.gpu

T = {L.LORA_BF16: torch.bfloat16, L.LORA_F32: torch.float32}
LAYOUTS = [L.LORA_ROPE_HALF, L.LORA_ROPE_INTERLEAVED]


# M, q heads, k heads, head_dim, rot_dim: pairs in whole 16-byte pieces, and not
@pytest.mark.parametrize("shape", [(5, 3, 1, 24, 6), (3, 2, 2, 104, 52), (2, 4, 1, 64, 2), (9, 2, 0, 96, 64), (700, 1, 1, 40, 30)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("layout", LAYOUTS, ids=["half", "inter"])
@pytest.mark.parametrize("dtype", [L.LORA_BF16, L.LORA_F32], ids=["bf16", "f32"])
def test_what_passes_through_keeps_its_bits(shape, layout, dtype):
    """Any bits behind rot_dim: NaN of either kind, with any payload, infinities, subnormals."""
    M, hq, hk, D, rot = shape
    log(f"rope bits {shape} {layout} {dtype}")
    bits = torch.int16 if dtype == L.LORA_BF16 else torch.int32
    mant, size = (7, 16) if dtype == L.LORA_BF16 else (23, 32)
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    x = torch.randint(-2 ** (size - 1), 2 ** (size - 1), (M, hq + hk, D), device="cuda", generator=g).to(bits)
    x[:, :, -1] = (2 ** (size - 1) - 2 ** mant) + 1 + torch.randint(0, 8, (M, hq + hk), device="cuda", generator=g).to(bits)  # signalling
    x[:, :, :rot] = torch.empty(M, hq + hk, rot, device="cuda").normal_(generator=g).to(T[dtype]).view(bits)
    q, k = (t.reshape(M, -1).contiguous().view(T[dtype]) for t in (x[:, :hq], x[:, hq:]))
    freqs, factor = L.lora_rope_freqs(rot)
    pos = torch.arange(M, device="cuda", dtype=torch.int32)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    L.lora_rope(q, k if hk else None, pos, freqs, M, hq, hk, D, rot, hq * D, hk * D, layout, factor, 0, qo, hq * D,
                ko if hk else None, hk * D, dtype)
    torch.cuda.synchronize()
    for heads, was, got in ((hq, q, qo), (hk, k, ko)):
        was, got = (t.view(bits).view(M, heads, D) for t in (was, got))
        assert torch.equal(got[:, :, rot:], was[:, :, rot:])


@pytest.mark.parametrize("layout", LAYOUTS, ids=["half", "inter"])
def test_one_over_the_factor_turns_back(layout):
    M, h, D, rot = 130, 3, 72, 64
    freqs, f = L.lora_rope_freqs(rot, 10000.0, L.LORA_ROPE_YARN, 8.0, 4096.0)
    assert f > 1.2
    x = torch.empty(M, h * D, device="cuda").normal_()
    pos = torch.randint(-1000, 30000, (M,), device="cuda", dtype=torch.int32)

    def turn(v, factor, inverse):
        y = torch.empty_like(v)
        L.lora_rope(v, None, pos, freqs, M, h, 0, D, rot, h * D, h * D, layout, factor, inverse, y, h * D, None, 0,
                    L.LORA_F32)
        return y

    y = turn(x, f, 0)
    back, again = turn(y, 1.0 / f, 1), turn(y, f, 1)
    torch.cuda.synchronize()
    v = x.view(M, h, D)[:, :, :rot].abs().double()
    if layout == L.LORA_ROPE_HALF:
        size = (v[:, :, :rot // 2] + v[:, :, rot // 2:]).repeat(1, 1, 2)
    else:
        size = (v[:, :, 0::2] + v[:, :, 1::2]).repeat_interleave(2, 2)
    bound = torch.zeros(M, h, D, dtype=torch.float64, device="cuda")
    bound[:, :, :rot] = 36 * 2.0 ** -24 * size
    bound = bound.view(M, h * D)
    assert bool(((back.double() - x.double()).abs() <= bound).all())
    # with the factor both ways: the gradient's direction, the factor's square of what passed the pairs
    square = torch.ones(D, dtype=torch.float64, device="cuda")
    square[:rot] = f * f
    square = square.repeat(h)
    assert bool(((again.double() - x.double() * square).abs() <= bound * f * f).all())
