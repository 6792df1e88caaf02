"""A decoder block's step as a serving program runs it on 8-bit integers: norm and rows in 8 bits, the q, k and v
projection, rotary positions in place, (attention, here a plain product,) rows in 8 bits, the output projection
with the residual added in place, norm, and the expert layer on the same residual stream.

Stage by stage, each one's 64-bit result is formed from the stage's own inputs (with the bounds of its own
tests); then the whole step captured in a graph gives the eager bits at every replay."""

import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

from .epilogue_util import assert_within
from .gpu_util import log
from .test_gpu_int8_act import Call
from .test_gpu_int8_rows import check_norm, check_plain
from .test_gpu_moe_layer import Layer
from .test_gpu_rope import check as check_rope

pytestmark = pytest.mark.gpu

EPS = 1e-5


class Block:
    def __init__(self, M, d=512, hq=6, hk=2, D=64, ff=400, n=5, r=16):
        g = torch.Generator(device="cuda").manual_seed(M)

        def normal(*s):
            return torch.empty(s, device="cuda").normal_(0, 1, generator=g).bfloat16()

        self.M, self.d, self.hq, self.hk, self.D, self.n, self.r = M, d, hq, hk, D, n, r
        self.row = (hq + 2 * hk) * D
        self.x, self.res = normal(M, d), normal(M, d)
        self.w1, self.w2 = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
        self.pos = torch.arange(M, device="cuda", dtype=torch.int32) + 3000
        self.freqs, self.factor = L.lora_rope_freqs(D, 10000.0, L.LORA_ROPE_YARN, 4.0, 2048.0)
        self.qkv_p = Call(1, M, d, self.row, n, r)
        self.out_p = Call(2, M, hq * D, d, n, r, residual=True)
        self.moe = Layer(3, M, 3, 8, d, ff, n, r, residual=True)
        for c in (self.out_p, self.moe):
            c.ids, c.ranks, c.scale = self.qkv_p.ids, self.qkv_p.ranks, self.qkv_p.scale
        self.moe.rank_of = self.qkv_p.ranks.cpu().numpy()
        kept = torch.arange(r, device="cuda") < self.qkv_p.ranks[:, None]
        self.out_p.A *= kept[:, None, :]
        self.out_p.B *= kept[:, :, None]
        for p in "gud":
            self.moe.A[p] *= kept[:, None, None, :]
            self.moe.B[p] *= kept[:, None, :, None]
        self.stream = torch.empty_like(self.x)
        self.x8, self.xs = torch.empty(M, d, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        self.qkv = torch.empty(M, self.row, dtype=torch.bfloat16, device="cuda")
        self.a = torch.empty(M, hq * D, dtype=torch.bfloat16, device="cuda")
        self.a8, self.as_ = torch.empty(M, hq * D, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        self.y2 = torch.empty_like(self.x)

    def norm(self):
        L.lora_rmsnorm_int8(self.x, self.res, self.w1, EPS, self.M, self.d, self.stream, None, self.x8, self.xs)

    def project(self):
        c = self.qkv_p
        c.x8, c.x_scale = self.x8, self.xs
        c.enqueue(epi=None, y=self.qkv)

    def rope(self):
        q, k = self.qkv[:, :self.hq * self.D], self.qkv[:, self.hq * self.D:(self.hq + self.hk) * self.D]
        L.lora_rope(q, k, self.pos, self.freqs, self.M, self.hq, self.hk, self.D, self.D, self.row, self.row,
                    L.LORA_ROPE_HALF, self.factor, 0, q, self.row, k, self.row, L.LORA_BF16)

    def attention(self):  # stands in for the attention between them
        v = self.qkv.view(self.M, -1, self.D)
        rep = self.hq // self.hk
        mixed = v[:, :self.hq] * v[:, self.hq:self.hq + self.hk].repeat_interleave(rep, 1) \
            + v[:, self.hq + self.hk:].repeat_interleave(rep, 1)
        self.a.copy_(mixed.reshape(self.M, -1))

    def rows(self):
        L.lora_quant_int8(self.a, self.M, self.hq * self.D, self.a8, self.as_)

    def output(self):
        c = self.out_p
        c.x8, c.x_scale, c.residual = self.a8, self.as_, self.stream
        c.enqueue(y=self.stream)

    def norm2(self):
        L.lora_rmsnorm(self.stream, None, self.w2, EPS, self.M, self.d, None, self.y2, None, None)

    def experts(self):
        self.moe.x, self.moe.residual = self.y2, self.stream
        self.moe.enqueue(y=self.stream)

    def step(self):
        for stage in (self.norm, self.project, self.rope, self.attention, self.rows, self.output, self.norm2,
                      self.experts):
            stage()


@pytest.mark.parametrize("M", [1, 5, 37, 150, 600])
def test_decoder_block(M):
    log(f"decoder block M={M}")
    b = Block(M)
    b.norm()
    torch.cuda.synchronize()
    check_norm((b.stream, None, b.x8, b.xs), b.x, b.res, b.w1)
    b.project()
    torch.cuda.synchronize()
    b.qkv_p.check(b.qkv, "qkv")
    before = b.qkv.clone().view(M, -1, b.D)
    b.rope()
    torch.cuda.synchronize()
    after = b.qkv.view(M, -1, b.D)
    heads = b.hq + b.hk
    check_rope(after[:, :heads], before[:, :heads], b.pos, b.freqs, b.D, L.LORA_ROPE_HALF, b.factor, 0)
    assert torch.equal(after[:, heads:], before[:, heads:])
    b.attention()
    b.rows()
    torch.cuda.synchronize()
    check_plain((None, None, b.a8, b.as_), b.a)
    res = b.stream.clone()
    b.output()
    torch.cuda.synchronize()
    b.out_p.residual = res
    b.out_p.check(b.stream, "output")
    b.norm2()
    torch.cuda.synchronize()
    h = b.stream.double()
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * b.w2.double()
    assert ((b.y2.double() - n).abs() <= n.abs() * (2.0 ** -8 * 1.01 + 2.0 ** -17) + 2.0 ** -134).all()
    res = b.stream.clone()
    b.experts()
    torch.cuda.synchronize()
    b.moe.residual = res
    assert_within(b.stream, *b.moe.want(), "experts")

    # the same step in a graph
    b.step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (b.x8, b.xs, b.qkv, b.a8, b.as_, b.y2, b.stream)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for rep in range(3):
        for t in (b.x8, b.xs, b.qkv, b.a8, b.as_, b.y2, b.stream):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((b.x8, b.xs, b.qkv, b.a8, b.as_, b.y2, b.stream), want):
            assert torch.equal(got, w), rep
        b.step()
        torch.cuda.synchronize()
        assert torch.equal(b.stream, want[-1])
