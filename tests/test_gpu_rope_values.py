"""lora_rope: what passes through keeps its bits."""

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
