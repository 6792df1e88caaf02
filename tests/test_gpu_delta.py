"""The adapter's delta of the fused tiles (lora_linear_act and lora_linear_fp8 on many rows) alone: W is
zero, t = x A_i is exact in fp32 whatever the order of its sums, and each adapter has one rank row
that its B holds values in, so that y = scale_i t[j] B_i[j] of a single product."""

import numpy as np
import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

from .gpu_util import log

pytestmark = pytest.mark.gpu

# (M, d_in, d_out, adapters, r_max): 128 x 128 and 256 x 256 tiles, each rank bucket, few and many runs
SHAPES = [(300, 128, 264, 1, 1), (777, 144, 264, 40, 5), (900, 144, 520, 33, 16), (300, 128, 264, 9, 24),
          (800, 256, 520, 300, 64), (4100, 128, 3080, 50, 8), (4100, 128, 3080, 12, 64), (4100, 160, 3080, 700, 33)]


class Case:
    """t[m, j] = x0 A0 + x1 A1 + x2 A2 with x = (1, 2^-8, 2^-8) and A of 8 bits each, A2 scaled by
    2^-8: 24 bits from 2^0 to 2^-23 (the partial sums of any order fit them too)."""

    def __init__(self, op, M, K, N, n, r, f32=True, seed=0, t_scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.op, self.f32, self.dims = op, f32, (M, K, N, r, n)

        def mantissa(*s):  # 8 bits in [1, 2)
            return 1.0 + torch.randint(0, 120, s, device="cuda", generator=g) / 128.0

        at = (0, 40, K - 1)  # in different octets of k
        A = torch.zeros(n, K, r, device="cuda")
        for i, k in enumerate(at):
            A[:, k] = mantissa(n, r) * (2.0 ** -8 if i == 2 else 1.0) * t_scale
        x = torch.zeros(M, K, device="cuda")
        sign = 1.0 - 2.0 * torch.randint(0, 2, (M,), device="cuda", generator=g)
        x[:, at[0]] = sign
        x[:, at[1]] = x[:, at[2]] = sign * 2.0 ** -8
        self.j = torch.arange(n, device="cuda") * 7 % r  # the adapter's rank row
        B = torch.zeros(n, r, N, device="cuda")
        B[torch.arange(n, device="cuda"), self.j] = mantissa(n, N)
        self.A, self.B = A.bfloat16(), B.bfloat16()
        self.scale = torch.where(torch.arange(n, device="cuda") % 2 == 0, 2.0, 0.5)
        self.ids = torch.as_tensor(np.arange(M) * 5 % (n + 1) - 1, dtype=torch.int32, device="cuda")
        if op == "fp8":
            self.x = x.to(torch.float8_e4m3fn)
            self.W = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
            self.ones = torch.ones(max(M, N), device="cuda")
        else:
            self.x = x.bfloat16()
            self.W = torch.zeros(K, N, dtype=torch.bfloat16, device="cuda")
        assert torch.equal(self.x.float(), x) and torch.equal(self.A.float(), A)

    def t64(self):
        """scale_i t[m, j_i] in 64 bits, 0 without an adapter."""
        i = self.ids.long().clamp_min(0)
        a = self.A[i, :, self.j[i]].double()
        return torch.where(self.ids >= 0, (self.x.double() * a).sum(1) * self.scale[i].double(), 0.0)

    def run(self):
        M, K, N, r, n = self.dims
        y = torch.full((M, N), 7.0, dtype=torch.float32 if self.f32 else torch.bfloat16, device="cuda")
        epi = L.lora_epilogue(bias=torch.zeros(N, dtype=torch.bfloat16, device="cuda"))
        lora = (self.A, self.B, self.scale, None, self.ids, M, K, N, r, n, None, epi, y,
                L.LORA_F32 if self.f32 else L.LORA_BF16)
        if self.op == "fp8":
            ws, nb = L.fp8_workspace(M, K, N, r, n)
            L.lora_linear_fp8(self.x, self.ones, self.W, self.ones, *lora, L.LORA_MODE_AUTO, ws, nb)
        else:
            ws, nb = L.workspace(M, K, N, r, n)
            L.lora_linear_act(self.x, self.W, *lora, L.LORA_MODE_PREFILL, ws, nb)
        torch.cuda.synchronize()
        return y


@pytest.mark.parametrize("op", ["act", "fp8"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_fp32_delta_keeps_24_bits(op, shape):
    """The product t B has three parts of up to 16 bits; each of its six additions (three matrix steps
    of two octets) is off by at most one fp32 step of the sum so far, 2^-23: 6 2^-23 < 2^-20 in
    all.  (t carried as two bf16 values would be off by up to 2^-17.)"""
    log(f"delta in fp32 {op} {shape}")
    c = Case(op, *shape, seed=sum(shape))
    i = c.ids.long().clamp_min(0)
    want = c.t64()[:, None] * c.B[i, c.j[i]].double()
    off = (c.run().double() - want).abs()
    assert (off <= 6 * 2.0 ** -23 * want.abs()).all(), float((off / (want.abs() + 1e-30)).max() * 2 ** 23)


@pytest.mark.parametrize("op", ["act", "fp8"])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_infinite_b(op, f32, shape):
    """An infinity in B gives its adapter's rows t times it: an infinity of the product's sign, NaN
    for t = 0.  Other rows and columns keep their bits."""
    log(f"infinite B {op} {shape} f32={f32}")
    c = Case(op, *shape, f32=f32, seed=sum(shape))
    M, K, N, r, n = c.dims
    c.x.view(torch.uint8).view(M, -1)[M - 2] = 0  # t = 0
    base = c.run()
    i = c.ids.long().clamp_min(0)
    c.B[0, c.j[0], 3] = float("inf")
    c.B[n - 1, c.j[n - 1], N - 1] = float("-inf")
    c.B[n // 2, c.j[n // 2], 8] = float("inf")
    want = c.t64()[:, None] * c.B[i, c.j[i]].double()
    want[c.ids < 0] = 0
    got = c.run()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf].sign(), want[inf].sign().to(got.dtype))
    fine = torch.isfinite(want)
    assert inf.sum() > 0 and torch.equal(got[fine], base[fine])


@pytest.mark.parametrize("op", ["act", "fp8"])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("shape", [(300, 128, 264, 9, 1), (4100, 128, 3080, 50, 1)], ids=lambda s: "x".join(map(str, s)))
def test_ends_of_the_range(op, f32, shape):
    """scale t between the largest bf16 and the largest fp32 value stays finite; an infinite one
    gives an infinity of the product's sign, also times an infinite B, and NaN times 0."""
    log(f"ends of the range {op} {shape} f32={f32}")
    c = Case(op, *shape, f32=f32, seed=3)
    M, K, N, r, n = c.dims
    c.A.zero_()
    c.A[:, 0] = float.fromhex("0x1.fep127")  # the largest bf16
    c.A[:, 40] = float.fromhex("0x1.8p127")  # times 2^-8
    c.A[1, 0] = c.A[1, 40] = float.fromhex("-0x1.8p127")
    c.scale.fill_(1.0)
    c.scale[1] = 2.0  # t beyond fp32
    c.B[:] = (c.B.float() * 2.0 ** -20).bfloat16()
    c.B[1, 0, 1] = float("inf")
    c.B[1, 0, 2] = 0.0
    got = c.run().double()
    t = c.t64()
    one = c.ids == 1
    i = c.ids.long().clamp_min(0)
    want = t[:, None] * c.B[i, 0].double()
    rest = want[~one]
    step = 6 * 2.0 ** -23 if f32 else 2.0 ** -8 + 2.0 ** -15
    assert t.abs().max() > float.fromhex("0x1.ffp127")
    assert ((got[~one] - rest).abs() <= step * rest.abs()).all()
    assert torch.isnan(got[one][:, 2]).all()
    keep = torch.arange(N, device="cuda") != 2
    assert torch.isinf(got[one][:, keep]).all()
    assert torch.equal(got[one][:, keep].sign(), want[one][:, keep].sign())
