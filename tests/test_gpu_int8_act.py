"""lora_linear_int8 against the layer on its integers and the epilogue in 64 bits.

Tolerance of z, with S = |x| |W| w_scale and D = |scale| (|x| |A|) |B| element by element:
  * the integer sum is exact; its at most 16 slices are each rounded to fp32, scaled and added:
    (16 + 3) 2^-24 S;
  * the delta: MFMA chains over k = max(d_in, 64) products, at least eight of them per rounding,
    the split sums and the expand's r_max products: (k / 8 + 64) 2^-24 D;
  * with y in bf16 the fused tiles carry scale t as two bf16 values: 2^-16 D;
  * the column scale and the row scale are one product each.
What follows z is epilogue_util's."""

import numpy as np
import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

from .epilogue_util import ACTS, assert_within, epilogue64
from .gpu_util import log
from .test_gpu_fp8_act import BATCHES, SHAPES
from .test_gpu_fp8_act import Call as Fp8Call

pytestmark = pytest.mark.gpu


class Call(Fp8Call):
    """One layer's inputs and its lora_linear_int8 call."""

    def __init__(self, seed, M, K, N, n, r, codes="normal", **opt):
        super().__init__(seed, M, K, N, n, r, **opt)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        if codes == "normal":
            def ints(rows):
                v = torch.empty(rows, K, device="cuda").normal_(0, 1, generator=g)
                return torch.round(v / v.abs().amax(1, keepdim=True) * 127).to(torch.int8)
            self.x8, self.W8 = ints(M), ints(N)
            self.x_scale = (torch.rand(M, device="cuda", generator=g) + 0.5) / 30
            self.w_scale = (torch.rand(N, device="cuda", generator=g) + 0.5) / 30 * K ** -0.5
        else:  # every integer, -128 among them
            self.x8, self.W8 = (torch.randint(-128, 128, s, device="cuda", generator=g).to(torch.int8)
                                for s in ((M, K), (N, K)))
            self.x_scale = (torch.rand(M, device="cuda", generator=g) + 0.5) / 73
            self.w_scale = (torch.rand(N, device="cuda", generator=g) + 0.5) / 73 * K ** -0.5
        self.ws, self.nbytes = L.int8_workspace(M, K, N, r, n)
        self.ws.fill_(255)  # the workspace's contents need no initialisation

    def enqueue(self, segs=None, epi="own", y=None, stream=None, mode=L.LORA_MODE_AUTO):
        M, K, N, r, n = self.dims
        L.lora_linear_int8(self.x8, self.x_scale, self.W8, self.w_scale, self.A, self.B, self.scale,
                           self.ranks, self.ids, M, K, N, r, n, segs, self.epi() if epi == "own" else epi,
                           self.y if y is None else y, L.LORA_F32 if self.f32 else L.LORA_BF16, mode,
                           self.ws, self.nbytes, stream)

    def run(self, *args, y=None, **kw):
        self.enqueue(*args, y=y, **kw)
        torch.cuda.synchronize()
        return self.y if y is None else y

    def want(self):
        M, K, N, r, n = self.dims
        x, W = self.x8.double(), (self.W8.double() * self.w_scale.double()[:, None]).t().contiguous()
        z, S = x @ W, x.abs() @ W.abs()
        D = torch.zeros_like(S)
        for i in sorted(set(self.ids.tolist())):
            if not 0 <= i < n:
                continue
            rows = (self.ids == i).nonzero()[:, 0]
            k = r if self.ranks is None else int(self.ranks[i])
            a, b, s = self.A[i, :, :k].double(), self.B[i, :k].double(), float(self.scale[i])
            z[rows] += s * ((x[rows] @ a) @ b)
            D[rows] += abs(s) * ((x[rows].abs() @ a.abs()) @ b.abs())
        dz = 19 * 2.0 ** -24 * S + (max(K, 64) / 8 + 64) * 2.0 ** -24 * D
        if not self.f32:
            dz = dz + 2.0 ** -16 * D
        s = self.x_scale.double()[:, None]
        return epilogue64(z * s, dz * s + 2 * 2.0 ** -24 * (z * s).abs(), self.act, self.bias, self.mul,
                          self.residual, self.f32)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("k", range(3))
def test_matches_64_bits(shape, k):
    at = SHAPES.index(shape)
    opt = [dict(act=ACTS[at % 5], bias=True, mul=True, residual=True),
           dict(act=ACTS[(at + 2) % 5], bias=at % 2 == 0, residual=True, f32=True, codes="any"),
           dict(act=ACTS[(at + 3) % 5], mul=True, f32=at % 3 == 0, codes="any", ranks=None)][k]
    log(f"linear_int8 {shape} {opt}")
    c = Call(300 + at, *shape, **opt)
    c.check(c.run(), f"{shape} {opt}")


# The borders of the launch sequences: 64-row tiles that are one round of CUs and one more, splits of K that a
# quarter more workgroups than CUs makes, 2048 rows and one more, K slices and whole tiles behind them
BORDERS = [(128, 2048, 11008, 5, 16), (129, 512, 10880, 5, 16), (130, 512, 11008, 5, 16), (256, 1040, 8192, 9, 8),
           (333, 1040, 2760, 30, 24), (2048, 272, 1024, 40, 16), (2049, 272, 1024, 40, 16), (2048, 160, 1032, 3, 8),
           (1024, 4112, 2760, 64, 64), (2100, 4096, 264, 6, 16), (1100, 6160, 2056, 4, 5), (2048, 128, 8, 2048, 64),
           # adapter tiles beside W's: blocks of 16 rows, chunks of 512 k, 48 tiles and one more
           (17, 512, 264, 17, 24), (128, 528, 1032, 300, 64), (768, 1040, 512, 8, 16), (769, 1040, 512, 8, 16),
           (96, 144, 128, 40, 56), (192, 4608, 136, 30, 32), (193, 4624, 136, 30, 32), (3, 65552, 136, 5, 48)]


@pytest.mark.parametrize("shape", BORDERS, ids=lambda c: "x".join(map(str, c)))
def test_borders_of_the_sequences(shape):
    at = BORDERS.index(shape)
    log(f"linear_int8 border {shape}")
    for f32 in (False, True):
        c = Call(700 + at, *shape, act=ACTS[at % 5], bias=True, residual=at % 2 == 0, mul=at % 3 == 0, f32=f32,
                 codes="any")
        c.check(c.run(), f"{shape} f32={f32}")


@pytest.mark.parametrize("M,K,N", BATCHES)
def test_integer_sums_are_exact(M, K, N):
    """Scales 1, no adapters, fp32: every product sum below 2^24 is returned as it is."""
    c = Call(5, M, K, N, 3, 8, f32=True, ids=np.full(M, -1))
    c.x8.copy_(torch.randint(-15, 16, (M, K), device="cuda"))
    c.W8[:, ::7] = -128
    c.x_scale.fill_(1)
    c.w_scale.fill_(1)
    want = c.x8.double() @ c.W8.double().t()
    assert want.abs().max() < 2 ** 24 and K * 15 * 128 < 2 ** 24
    assert torch.equal(c.run(epi=None).double(), want)


@pytest.mark.parametrize("M", [1, 100, 150, 200, 300])
def test_the_largest_sums(M):
    """-128 times -128 at the longest d_in: the last int32 below 2^31."""
    K, N = L.LORA_INT8_MAX_D_IN, 264
    c = Call(6, M, K, N, 2, 4, f32=True, ids=np.full(M, -1))
    c.x8.fill_(-128)
    c.W8.fill_(-128)
    c.W8[3] = 127
    c.x_scale.fill_(1)
    c.w_scale.fill_(1)
    y = c.run(epi=None).double()
    keep = torch.arange(N, device="cuda") != 3
    assert (y[:, keep] == K * 2 ** 14).all()
    assert ((y[:, 3] + K * 128 * 127).abs() <= 19 * 2.0 ** -24 * K * 2 ** 14).all()


@pytest.mark.parametrize("M,K,N", BATCHES)
def test_no_epilogue(M, K, N):
    log(f"linear_int8 without epilogue M={M} K={K}")
    for f32 in (False, True):
        c = Call(7, M, K, N, 6, 16, f32=f32)
        want = c.run(epi=None).clone()
        c.check(want, "no epilogue")
        c.y.fill_(7)
        assert torch.equal(c.run(), want)


@pytest.mark.parametrize("M,K,N", BATCHES)
@pytest.mark.parametrize("which", ["residual", "mul"])
def test_in_place(M, K, N, which):
    for f32 in (False, True):
        c = Call(9, M, K, N, 6, 16, act="silu", bias=True, f32=f32, **{which: True})
        want = c.run().clone()
        buf = getattr(c, which).clone()
        setattr(c, which, buf)
        assert torch.equal(c.run(y=buf), want)


@pytest.mark.parametrize("M,K,N", BATCHES)
def test_base_rows_and_bad_ids(M, K, N):
    opt = dict(act="gelu", bias=True, residual=True)
    c = Call(13, M, K, N, 5, 16, ids=np.full(M, -1), **opt)
    c.check(c.run(), "all base")
    ids = np.arange(M) % 7 - 1  # 5 is outside the pool
    ids[3] = -2
    ids[4] = 2 ** 31 - 1
    c = Call(13, M, K, N, 5, 16, ids=ids, **opt)
    c.check(c.run(), "bad ids")


@pytest.mark.parametrize("n", [6, 40, 300])
@pytest.mark.parametrize("M,K,N", BATCHES)
def test_unused_adapters_do_not_leak(M, K, N, n):
    c = Call(15, M, K, N, n, 16, act="silu", mul=True, ids=np.arange(M) % 4 - 1)
    want = c.want()
    c.A[3:] = float("nan")
    c.B[3:] = float("inf")
    c.scale[3:] = float("nan")
    assert_within(c.run(), *want, f"M={M}")


@pytest.mark.parametrize("M,K,N", BATCHES)
def test_a_nan_scale_stays_in_its_row_or_column(M, K, N):
    """Rows that lora_quant_int8 gives no scale: integers 0, scale NaN."""
    c = Call(17, M, K, N, 4, 16, bias=True)
    base = c.run().clone()
    c.x8[2] = 0
    c.x_scale[2] = float("nan")
    c.w_scale[N - 1] = float("nan")
    got = c.run()
    assert torch.isnan(got[2]).all() and torch.isnan(got[:, N - 1]).all()
    keep = torch.arange(M, device="cuda") != 2
    assert torch.equal(got[keep, :N - 1], base[keep, :N - 1])


@pytest.mark.parametrize("M,K,N", BATCHES)
def test_an_adapter_with_nan_spoils_its_own_rows_alone(M, K, N):
    n, r = 6, 16
    c = Call(37, M, K, N, n, r, act="silu", bias=True, ids=np.arange(M) * 5 % (n + 1) - 1, ranks=None)
    base = c.run().clone()
    c.B[1, 0, 3] = float("nan")
    c.B[2, r - 1, N - 1] = float("inf")
    c.A[3, K - 1, 0] = float("nan")
    got = c.run()
    hit = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    hit[c.ids == 1, 3] = True
    hit[c.ids == 2, N - 1] = True
    hit[c.ids == 3] = True
    assert torch.equal(got[~hit], base[~hit])
    assert torch.isnan(got[c.ids == 1, 3]).all() and torch.isnan(got[c.ids == 3]).all()
    assert not torch.isfinite(got[c.ids == 2, N - 1]).any()


@pytest.mark.parametrize("M,K,N", BATCHES)
def test_given_segments_checked_mode_streams_and_rows_behind(M, K, N):
    c = Call(19, M, K, N, 6, 16, act="gelu_tanh", bias=True, residual=True)
    want = c.run().clone()
    seg = L.Segments(M, 6)
    L.lora_build_segments(c.ids, M, 6, seg)
    c.y.fill_(7)
    assert torch.equal(c.run(segs=seg), want)
    c.y.fill_(7)
    assert torch.equal(c.run(mode=L.LORA_MODE_CHECKED), want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.y.fill_(7)
    torch.cuda.synchronize()
    assert torch.equal(c.run(stream=st), want)
    buf = torch.full((M + 9, N), 5.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(c.run(y=buf)[:M], want) and (buf[M:] == 5).all()
    c.ids[1] = 6
    with pytest.raises(L.LoraError) as e:
        c.run(mode=L.LORA_MODE_CHECKED)
    assert e.value.status == 8


@pytest.mark.parametrize("M,K,N", BATCHES)
def test_graph_replays(M, K, N):
    c = Call(29, M, K, N, 6, 16, act="silu", bias=True, mul=True, residual=True)
    want = c.run().clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.enqueue()
    for rep in range(3):
        c.y.fill_(0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.y, want), rep
        assert torch.equal(c.run(), want)


def test_operands_past_4_gib():
    """64-bit addresses: x and W in +-1, scales 1, so that every fp32 sum is exact."""
    for M, K, N in ((300000, 14400, 264), (33000, 131056, 264)):
        if torch.cuda.mem_get_info()[0] < 4 * M * K + (16 << 30):
            pytest.skip("not enough memory")
        log(f"linear_int8 past 4 GiB {M} {K}")
        g = torch.Generator(device="cuda").manual_seed(M)
        c = Call.__new__(Call)
        c.dims, c.f32, c.act = (M, K, N, 8, 3), True, "none"
        c.x8 = torch.empty(M, K, dtype=torch.int8, device="cuda").random_(0, 2, generator=g).mul_(2).sub_(1)
        c.W8 = torch.empty(N, K, dtype=torch.int8, device="cuda").random_(0, 2, generator=g).mul_(2).sub_(1)
        c.x_scale, c.w_scale = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
        c.A = (1.0 - 2.0 * torch.randint(0, 2, (3, K, 8), device="cuda", generator=g)).bfloat16()
        c.B = (0.5 - torch.randint(0, 2, (3, 8, N), device="cuda", generator=g)).bfloat16()
        c.scale, c.ranks, c.bias, c.mul, c.residual = torch.ones(3, device="cuda"), None, None, None, None
        c.ids = torch.randint(-1, 3, (M,), device="cuda", generator=g, dtype=torch.int32)
        c.y = torch.full((M, N), 7.0, device="cuda")
        c.ws, c.nbytes = L.int8_workspace(M, K, N, 8, 3)
        c.run()
        edge = (1 << 32) // K
        rows = torch.tensor([0, 1, M // 2, edge - 1, edge, edge + 1, M - 129, M - 1], device="cuda")
        x = c.x8[rows].double()
        want = x @ c.W8.double().t().contiguous()
        for k, i in enumerate(c.ids[rows].tolist()):
            if i >= 0:
                want[k] += (x[k] @ c.A[i].double()) @ c.B[i].double()
        assert torch.equal(c.y[rows].double(), want)
        del c, x
        torch.cuda.empty_cache()


@pytest.mark.parametrize("M,K,N", [(512, 272, 1032), (2048, 160, 264), (2048, 128, 1024)])
def test_the_largest_adapter_table(M, K, N):
    """Segments of 16384 adapters in one workgroup beside the GEMM, ids that use a few and the last of them."""
    n, r = L.LORA_MAX_ADAPTERS, 8
    c = Call(23, M, K, N, n, r, act="silu", bias=True, mul=True)
    c.check(c.run(), f"{M} {K} {N}")
    want = c.run().clone()
    seg = L.Segments(M, n)
    L.lora_build_segments(c.ids, M, n, seg)
    c.y.fill_(7)
    assert torch.equal(c.run(segs=seg), want)


# With segments beside the GEMM (many adapter tiles, or a stride that is no multiple of 8), and adapter tiles for
# more than 128 rows
WAYS = [(333, 1040, 2760, 30, 24), (100, 512, 264, 6, 5), (700, 256, 264, 40, 64), (300, 528, 264, 6, 13),
        (257, 1040, 264, 12, 16), (17, 656, 136, 17, 40)]


@pytest.mark.parametrize("shape", WAYS, ids=lambda c: "x".join(map(str, c)))
def test_ways_of_wide_batches(shape):
    """Given segments, a graph whose ids change between its replays, two calls at once, NaN in an adapter."""
    M, K, N, n, r = shape
    a = Call(31, *shape, act="silu", bias=True, mul=True, residual=True)
    b = Call(32, *shape, residual=True, f32=True)
    want_a, want_b = a.run().clone(), b.run().clone()
    a.check(want_a, f"{shape}"), b.check(want_b, f"{shape} f32")
    seg = L.Segments(M, n)
    L.lora_build_segments(a.ids, M, n, seg)
    a.y.fill_(7)
    assert torch.equal(a.run(segs=seg), want_a)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a.y.fill_(7), b.y.fill_(7)
        torch.cuda.synchronize()
        a.enqueue(stream=s1), b.enqueue(stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a.y, want_a) and torch.equal(b.y, want_b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.enqueue()
    ids = a.ids.clone()
    for rep in range(3):
        a.ids.copy_(torch.roll(ids, rep * 5 + 1) if rep < 2 else ids)
        a.y.fill_(7)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = a.y.clone()
        assert torch.equal(got, a.run()), rep
    assert torch.equal(got, want_a)
    i = int(b.ids[b.ids >= 0][0])
    b.B[i, 0, 3] = float("nan")
    got, hit = b.run(), b.ids == i
    assert torch.equal(got[~hit], want_b[~hit]) and torch.isnan(got[hit, 3]).all()
