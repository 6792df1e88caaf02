"""lora_linear_act and lora_linear_fp8 where their other tests do not go: operands past 4 GiB (64-bit
addresses in every kernel that has both kinds), and decode batches whose d_in is an odd multiple of
8 on pools narrower than an adapter slot.

Large cases: x in +-1, +-1.5 (and their neighbours in bf16), W, A and B in +-1, +-1.5 or powers of
two, scale 1: products are multiples of 2^-4, and sums of up to 2^20 of them stay far below 2^24 of these,
so every fp32 sum is exact in any order and y in fp32 has to be equal.  bf16 y adds its rounding,
2^-8, and that of scale t to two bf16 values, 2^-16 of each of the r_max products."""

import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

from .epilogue_util import assert_within
from .gpu_util import log
from .test_gpu_act import Call

pytestmark = pytest.mark.gpu

GIB4 = 1 << 32


def signs(*shape, g):
    """+-1 or +-1.5, as E4M3 codes"""
    b = torch.empty(shape, dtype=torch.uint8, device="cuda").random_(0, 256, generator=g)
    return b.bitwise_and_(0x84).bitwise_or_(0x38)


# (op, M, d_in, d_out, mode): fused tiles of 256 x 256 and 128 x 128, and K slices, x past 4 GiB
LARGE = [("fp8", 300000, 14400, 264, 0), ("fp8", 16400, 262160, 264, 0), ("fp8", 8200, 524304, 264, 0),
         ("act", 150000, 14400, 264, L.LORA_MODE_PREFILL), ("act", 8200, 262152, 264, L.LORA_MODE_PREFILL)]


@pytest.mark.parametrize("case", LARGE, ids=lambda c: "x".join(map(str, c)))
def test_operands_past_4_gib(case):
    op, M, K, N, mode = case
    size = M * K * (1 if op == "fp8" else 2)
    assert size > GIB4
    if torch.cuda.mem_get_info()[0] < 4 * size + (16 << 30):
        pytest.skip("not enough memory")
    log(f"past 4 GiB {case}")
    g = torch.Generator(device="cuda").manual_seed(M + K)
    n, r = 3, 8

    def pm(*s):
        return 1.0 - 2.0 * torch.randint(0, 2, s, device="cuda", generator=g)

    A, B = pm(n, K, r).bfloat16(), (pm(n, r, N) * 0.5).bfloat16()
    ids = torch.randint(-1, n, (M,), device="cuda", generator=g, dtype=torch.int32)
    bias = pm(N).bfloat16()
    if op == "fp8":
        x, W = signs(M, K, g=g), signs(N, K, g=g)
        ones = torch.ones(max(M, N), device="cuda")
    else:
        x = torch.empty(M, K, dtype=torch.int16, device="cuda").random_(-32768, 32767, generator=g)
        x = x.bitwise_and_(-32656).bitwise_or_(0x3F80).view(torch.bfloat16)  # +-1 .. 1.875 in steps of 2^-3
        W = pm(K, N).bfloat16()
    edge = (GIB4 // (size // M))  # the row that 4 GiB end in
    rows = torch.tensor([0, 1, 127, 128, M // 2, edge - 1, edge, edge + 1, M - 129, M - 2, M - 1], device="cuda")
    xr = x[rows].view(torch.float8_e4m3fn).double() if op == "fp8" else x[rows].double()
    Wd = W.view(torch.float8_e4m3fn).double().t().contiguous() if op == "fp8" else W.double()
    z = xr @ Wd
    d = torch.zeros_like(z)  # the sum of |t B|
    for k, i in enumerate(ids[rows].tolist()):
        if i >= 0:
            t = xr[k] @ A[i].double()
            z[k] += t @ B[i].double()
            d[k] = t.abs() @ B[i].double().abs()
    want = z + bias.double()
    del Wd, xr
    for f32 in (True, False):
        y = torch.full((M, N), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        lora = (A, B, torch.ones(n, device="cuda"), None, ids, M, K, N, r, n, None, L.lora_epilogue(bias=bias), y,
                L.LORA_F32 if f32 else L.LORA_BF16, mode)
        if op == "fp8":
            ws, nb = L.fp8_workspace(M, K, N, r, n)
            L.lora_linear_fp8(x, ones, W, ones, *lora, ws, nb)
        else:
            ws, nb = L.workspace(M, K, N, r, n)
            L.lora_linear_act(x, W, *lora, ws, nb)
        torch.cuda.synchronize()
        off = (y[rows].double() - want).abs()
        if f32:
            assert (off == 0).all(), float(off.max())
        else:
            assert (off <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * d).all(), float(off.max())
        del y, ws, lora
    del x, W
    torch.cuda.empty_cache()


# (M, d_in, d_out, adapters, r_max): slots by id (adapters <= rows) and by row, one and two row
# tiles, d_in 8 past a step of 16, strides of 8 to 56 in slots of 16 to 64
TAILS = [(5, 1032, 264, 3, 8), (3, 136, 264, 40, 8), (33, 1160, 520, 90, 24), (100, 136, 264, 200, 40),
         (100, 1048, 264, 7, 40), (128, 136, 1032, 128, 48), (64, 4104, 264, 9, 56), (1, 136, 8, 1, 24),
         (77, 264, 264, 300, 56), (128, 2072, 264, 2, 8)]


@pytest.mark.parametrize("shape", TAILS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("ranks", ["mixed", "full"])
def test_decode_with_a_tail_and_narrow_adapters(shape, ranks):
    log(f"decode tail {shape} ranks {ranks}")
    for f32 in (True, False):
        c = Call(sum(shape), *shape, act="silu", bias=True, residual=True, f32=f32, mode=L.LORA_MODE_DECODE,
                 ranks=ranks)
        c.check(c.run(), f"{shape} {ranks} f32={f32}")
    # adapters that no row has are not read into any other's columns
    c = Call(sum(shape), *shape, mode=L.LORA_MODE_DECODE, ranks=ranks, ids=[0] * shape[0])
    want = c.want()
    c.A[1:] = float("nan")
    c.B[1:] = float("inf")
    assert_within(c.run(), *want, f"{shape} one adapter")
