"""The activations of lora_linear_act and lora_linear_fp8 alone, relative to their own size: x is
zero, so that z is the bias (bf16, exact) and y, in fp32, is act(z).

Bounds, in units of 2^-24 of the value (the hardware's exp2 and reciprocal are off by a step, two
units; a product or sum by one unit):
  silu       z rcp(1 + exp2(c z)): exp2's argument 1.5 roundings of |z| log2(e), times ln 2: 1.5 |z|;
             exp2 2, sum 1, rcp 2, product 1, and log2(e) itself 1
  gelu_tanh  the same on 2 v = 2 sqrt(2 / pi) (z + 0.044715 z^3): two constants, z^2, the fma and the
             product, up to 5 units of it: 5 |2 v|
  gelu       t = 1 / (1 + p a): 3 units, times up to 2.9 in t P(t); P in fp32 4, its fit 1; products 3,
             exp2 2; its argument z^2 / 2 with 2.5 roundings: 1.25 z^2; 24 + 1.5 z^2 in all
Below 2^-126 nothing is asked of the value's own size (hence the absolute 1e-36: |z| times a flushed
exponential).
"""

import math

import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

from .epilogue_util import ACTS, act64
from .gpu_util import log

pytestmark = pytest.mark.gpu

DEC, PRE = L.LORA_MODE_DECODE, L.LORA_MODE_PREFILL
# one call per launch sequence: (layer, M, d_in, mode)
CALLS = [("act", 3, 128, DEC), ("act", 200, 128, DEC), ("act", 300, 2048, DEC), ("act", 300, 16384, DEC),
         ("act", 130, 64, PRE), ("fp8", 3, 128, 0), ("fp8", 150, 128, 0), ("fp8", 300, 64, 0)]


def activated(call, act, z, f32=True):
    """y[M, len(z)] of a call whose z is the given bf16 vector in every row."""
    op, M, K, mode = call
    N = z.numel()
    bf = torch.bfloat16

    def zeros(*s, dtype=bf):
        return torch.zeros(s, dtype=dtype, device="cuda")

    y = torch.full((M, N), 7.0, dtype=torch.float32 if f32 else bf, device="cuda")
    lora = (zeros(2, K, 8), zeros(2, 8, N), torch.ones(2, device="cuda"), None,
            torch.arange(M, dtype=torch.int32, device="cuda") % 3 - 1, M, K, N, 8, 2, None)
    tail = (L.lora_epilogue(ACTS.index(act), z), y, L.LORA_F32 if f32 else L.LORA_BF16, mode)
    if op == "act":
        ws, nbytes = L.workspace(M, K, N, 8, 2)
        L.lora_linear_act(zeros(M, K), zeros(K, N), *lora, *tail, ws, nbytes)
    else:
        ws, nbytes = L.fp8_workspace(M, K, N, 8, 2)
        L.lora_linear_fp8(zeros(M, K, dtype=torch.uint8), torch.ones(M, device="cuda"),
                          zeros(N, K, dtype=torch.uint8), torch.ones(N, device="cuda"), *lora, *tail, ws, nbytes)
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("call", CALLS, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("act", ACTS)
def test_relative_to_their_own_size(call, act):
    log(f"activation {act} {call}")
    z = torch.cat([-torch.logspace(-3, math.log10(12.0), 2048, dtype=torch.float64),
                   torch.logspace(-3, 3, 512, dtype=torch.float64)]).bfloat16().cuda()
    z64 = z.double()
    if act == "gelu_tanh":
        z = z[z64 > -6.5]  # beyond, 1 + tanh loses the 64-bit form its digits
        z = z[:z.numel() // 8 * 8].contiguous()
        z64 = z.double()
        v2 = 2 * math.sqrt(2 / math.pi) * (z64 + 0.044715 * z64 ** 3)
        want, units = z64 * torch.sigmoid(v2), 8 + 5 * v2.abs()
    elif act == "silu":
        want, units = act64(z64, act), 8 + 1.5 * z64.abs()
    elif act == "gelu":
        want, units = act64(z64, act), 24 + 1.5 * z64 ** 2
    else:
        want, units = act64(z64, act), 0 * z64
    units = torch.where(z64 > 0, units.clamp_max(64.0), units)  # e^-|z| next to 1
    got = activated(call, act, z)
    off = (got.double() - want).abs()
    bad = off > units * 2.0 ** -24 * want.abs() + 1e-36
    i = int((off / (want.abs() + 1e-30)).amax(0).argmax())
    assert not bad.any(), f"worst at z={float(z[i])}: {float(got[0, i])} for {float(want[i])}"


@pytest.mark.parametrize("call", CALLS, ids=lambda c: "x".join(map(str, c)))
def test_infinities_and_nan(call):
    inf = float("inf")
    z = torch.tensor([inf, -inf, float("nan"), 0.0, -0.0, 3e38, -3e38, 1.0], device="cuda").bfloat16()
    for act in ACTS:
        for f32 in (True, False):
            y = activated(call, act, z, f32).float()
            assert (y[:, 0] == inf).all() and torch.isnan(y[:, 2]).all() and (y[:, 3:5] == 0).all(), act
            assert (y[:, 5] == z[5].float()).all(), act
            if act == "none":
                assert (y[:, 1] == -inf).all() and (y[:, 6] == z[6].float()).all()
            elif act == "relu":
                assert (y[:, 1] == 0).all() and (y[:, 6] == 0).all()
            else:  # -infinity times zero; any finite z has its limit
                assert torch.isnan(y[:, 1]).all() and (y[:, 6] == 0).all(), act
