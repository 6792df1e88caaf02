"""lora_linear_act against the layer and its epilogue in 64 bits (bounds: epilogue_util)."""

import numpy as np
import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

from .epilogue_util import ACTS, assert_within, epilogue64, layer64
from .gpu_util import log

pytestmark = pytest.mark.gpu

DEC, PRE, AUTO = L.LORA_MODE_DECODE, L.LORA_MODE_PREFILL, L.LORA_MODE_AUTO


class Call:
    """One layer's inputs and its lora_linear_act call."""

    def __init__(self, seed, M, K, N, n, r, act="none", bias=False, mul=False, residual=False,
                 f32=False, mode=AUTO, ids=None, ranks="mixed"):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*s, std=1.0):
            return torch.empty(s, device="cuda").normal_(0, std, generator=g)

        self.dims = (M, K, N, r, n)
        self.mode, self.f32, self.act = mode, f32, act
        out = torch.float32 if f32 else torch.bfloat16
        rk = torch.randint(1, r + 1, (n,), device="cuda", generator=g, dtype=torch.int32)
        self.ranks = rk if ranks == "mixed" else None
        kept = torch.arange(r, device="cuda") < (rk[:, None] if ranks == "mixed" else torch.full_like(rk, r)[:, None])
        self.x = normal(M, K).bfloat16()
        self.W = normal(K, N, std=K ** -0.5).bfloat16()
        self.A = (normal(n, K, r, std=K ** -0.5) * kept[:, None, :]).bfloat16()
        self.B = (normal(n, r, N, std=0.5 * r ** -0.5) * kept[:, :, None]).bfloat16()
        self.scale = (16.0 / rk.float()).contiguous()
        if ids is None:
            self.ids = torch.randint(-1, n, (M,), device="cuda", generator=g, dtype=torch.int32)
        else:
            self.ids = torch.as_tensor(ids, dtype=torch.int32, device="cuda").contiguous()
        self.bias = normal(N).bfloat16() if bias else None
        self.mul = normal(M, N).to(out) if mul else None
        self.residual = normal(M, N).to(out) if residual else None
        self.y = torch.full((M, N), 7.0, dtype=out, device="cuda")
        self.ws, self.nbytes = L.workspace(M, K, N, r, n)

    def epi(self):
        return L.lora_epilogue(ACTS.index(self.act), self.bias, self.mul, self.residual)

    def run(self, segs=None, epi="own", y=None, stream=None, mode=None):
        M, K, N, r, n = self.dims
        L.lora_linear_act(self.x, self.W, self.A, self.B, self.scale, self.ranks, self.ids, M, K, N,
                          r, n, segs, self.epi() if epi == "own" else epi,
                          self.y if y is None else y, L.LORA_F32 if self.f32 else L.LORA_BF16,
                          self.mode if mode is None else mode, self.ws, self.nbytes, stream)
        torch.cuda.synchronize()
        return self.y if y is None else y

    def want(self):
        z, dz = layer64(self.x.double(), self.W.double(), self.A, self.B, self.scale, self.ranks, self.ids)
        return epilogue64(z, dz, self.act, self.bias, self.mul, self.residual, self.f32)

    def check(self, got, what):
        assert_within(got, *self.want(), what)


# (M, K, N, n, r, mode): every launch sequence and its edges
SEQUENCES = [
    # small decode: one row, odd rows, adapters by id and by row, ragged columns
    (1, 128, 8, 1, 1, DEC), (1, 4096, 4096, 8, 16, AUTO), (5, 256, 1032, 3, 8, DEC),
    (33, 1024, 520, 90, 16, DEC), (64, 4096, 1000, 32, 64, AUTO), (128, 512, 2056, 20, 24, DEC),
    (31, 288, 136, 4, 12, DEC),  # r_max not a multiple of 8: the three-launch sequence
    # medium decode
    (129, 512, 512, 7, 16, DEC), (200, 1024, 520, 40, 32, AUTO), (256, 4096, 264, 256, 64, DEC),
    (131, 160, 1096, 300, 5, DEC),
    # stream-K
    (257, 4096, 2056, 50, 64, DEC), (509, 11008, 1024, 100, 24, AUTO), (767, 4096, 512, 9, 8, AUTO),
    (1024, 2048, 520, 600, 16, DEC),
    # d_in not a multiple of 32 or 128: plain split-K slices
    (1, 1032, 520, 4, 16, DEC), (64, 4104, 1000, 32, 16, AUTO), (200, 1160, 520, 40, 33, DEC),
    (300, 4128, 1032, 50, 64, DEC), (700, 2088, 136, 5, 8, AUTO),
    # too short to split
    (7, 8, 8, 2, 1, DEC), (3, 200, 72, 5, 3, AUTO), (300, 64, 520, 4, 16, DEC),
    # prefill: 128 x 128 and 256 x 256 tiles, ragged rows and columns, odd d_in
    (768, 512, 520, 8, 16, AUTO), (1500, 1032, 264, 30, 64, AUTO), (3000, 264, 2056, 5, 8, AUTO),
    (4100, 520, 3080, 3, 16, AUTO), (12, 96, 40, 4, 16, PRE), (2000, 256, 6408, 700, 40, PRE),
    # decode asked for where only a large-tile launch runs
    (1300, 4096, 4104, 4, 16, DEC), (900, 256, 8200, 4, 16, DEC),
    # AUTO's choice between splitting K and whole tiles, both sides of it below and above 768 rows
    (300, 512, 4096, 4, 16, AUTO), (300, 512, 4096, 300, 64, AUTO), (768, 4096, 1024, 4, 16, AUTO),
    (1024, 256, 2056, 1024, 40, AUTO), (1300, 1032, 1032, 700, 64, AUTO), (1300, 4104, 2056, 3, 8, AUTO),
    # a few more tiles than one round of 256 x 256 ones
    (4500, 128, 4096, 9, 16, PRE),
    # small tiles over one, two, an odd number and very many runs, at each number of rank chunks
    (140, 128, 136, 1, 64, PRE), (129, 128, 136, 2, 64, PRE), (900, 128, 520, 33, 32, PRE),
    (900, 136, 520, 51, 8, PRE), (300, 128, 264, 300, 48, PRE), (131, 64, 72, 3, 17, PRE),
]


@pytest.mark.parametrize("seq", SEQUENCES, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("k", range(3))
def test_matches_64_bits(seq, k):
    M, K, N, n, r, mode = seq
    # three epilogues per sequence, all five activations and both types over the list
    at = SEQUENCES.index(seq)
    opt = [dict(act=ACTS[at % 5], bias=True, mul=True, residual=True),
           dict(act=ACTS[(at + 2) % 5], bias=at % 2 == 0, residual=True, f32=True),
           dict(act=ACTS[(at + 3) % 5], mul=True, f32=at % 3 == 0)][k]
    log(f"linear_act {seq} {opt}")
    c = Call(100 + at, M, K, N, n, r, mode=mode, **opt)
    c.check(c.run(), f"{seq} {opt}")


@pytest.mark.parametrize("M,K,N,mode", [(20, 512, 264, DEC), (200, 512, 264, DEC), (300, 2048, 264, DEC),
                                        (300, 16384, 264, DEC), (300, 1032, 264, DEC),
                                        (800, 512, 264, PRE)])
def test_no_epilogue_is_lora_linear(M, K, N, mode):
    """NULL gives lora_linear's bits; so does an epilogue of nothing where the launches match."""
    log(f"linear_act without epilogue M={M} K={K}")
    for f32 in (False, True):
        c = Call(7, M, K, N, 6, 16, mode=mode, f32=f32)
        y = torch.empty_like(c.y)
        _, _, _, r, n = c.dims
        L.lora_linear(c.x, c.W, c.A, c.B, c.scale, c.ranks, c.ids, M, K, N, r, n, None, y,
                      L.LORA_F32 if f32 else L.LORA_BF16, mode, c.ws, c.nbytes)
        assert torch.equal(c.run(epi=None), y)
        c.y.fill_(7)
        if (M, K) in ((300, 2048), (300, 1032)):
            # split-K slices: lora_linear rounds x W before its expand adds the delta, the
            # epilogue's pass rounds their sum once
            c.check(c.run(), "empty epilogue")
        else:
            assert torch.equal(c.run(), y)


@pytest.mark.parametrize("M,K,N,mode", [(1, 512, 264, DEC), (77, 1024, 1032, DEC), (200, 512, 264, DEC),
                                        (300, 2048, 520, DEC), (300, 16384, 264, DEC),
                                        (300, 1032, 264, DEC), (777, 512, 264, PRE),
                                        (4100, 128, 3080, PRE)])
@pytest.mark.parametrize("which", ["residual", "mul"])
def test_in_place(M, K, N, mode, which):
    """residual or mul may be y itself: the bits of separate buffers."""
    log(f"linear_act in place {which} M={M} K={K} N={N}")
    for f32 in (False, True):
        c = Call(9, M, K, N, 6, 16, act="silu", bias=True, mode=mode, f32=f32, **{which: True})
        want = c.run().clone()
        buf = getattr(c, which).clone()
        setattr(c, which, buf)
        assert torch.equal(c.run(y=buf), want)


# one batch per launch sequence (d_out 264)
BATCHES = ((20, 256, DEC), (150, 256, DEC), (300, 2048, DEC), (300, 16384, DEC), (300, 1032, DEC),
           (800, 256, PRE))


def test_base_rows_and_bad_ids():
    """Rows without an adapter, alone or in a batch, and ids outside the pool take z = x W."""
    for M, K, mode in BATCHES:
        log(f"base rows M={M} K={K}")
        opt = dict(act="gelu", bias=True, residual=True, mode=mode)
        c = Call(13, M, K, 264, 5, 16, ids=np.full(M, -1), **opt)
        c.check(c.run(), f"all base M={M}")
        ids = np.arange(M) % 7 - 1  # 5 is outside the pool
        ids[3] = -2
        ids[4] = 2 ** 31 - 1
        c = Call(13, M, K, 264, 5, 16, ids=ids, **opt)
        c.check(c.run(), f"bad ids M={M}")


def test_unused_adapters_do_not_leak():
    """NaN and infinities in adapters no row uses, and outside an adapter's rank rows' batch,
    stay out of every row."""
    for M, K, n, mode in ((9, 256, 6, DEC), (9, 256, 40, DEC), (150, 256, 6, DEC),
                          (300, 2048, 6, DEC), (300, 16384, 6, DEC), (300, 1032, 6, DEC), (800, 256, 6, PRE)):
        log(f"unused adapters M={M} n={n}")
        c = Call(15, M, K, 264, n, 16, act="silu", mul=True, mode=mode, ids=np.arange(M) % 4 - 1)
        want = c.want()
        c.A[3:] = float("nan")
        c.B[3:] = float("inf")
        c.scale[3:] = float("nan")
        assert_within(c.run(), *want, f"M={M}")


def test_special_values_follow_the_formula():
    """NaN and infinities of an operand touch their own element alone."""
    for M, K, mode in ((9, 256, DEC), (150, 256, DEC), (300, 2048, DEC), (300, 16384, DEC), (800, 256, PRE)):
        for act in ACTS:
            c = Call(17, M, K, 264, 4, 16, act=act, bias=True, mul=True, residual=True, mode=mode)
            base = c.run().clone()
            c.residual[0, 5] = float("nan")
            c.residual[1, 6] = float("inf")
            c.mul[2, 7] = float("nan")
            c.mul[M - 1, 263] = float("-inf")
            got = c.run()
            hit = torch.zeros(M, 264, dtype=torch.bool, device="cuda")
            hit[0, 5] = hit[1, 6] = hit[2, 7] = hit[M - 1, 263] = True
            assert torch.equal(got[~hit], base[~hit])
            assert torch.isnan(got[0, 5]) and got[1, 6] == float("inf") and torch.isnan(got[2, 7])
            assert not torch.isfinite(got[M - 1, 263]) or act == "relu"
            # large inputs of an activation: no NaN from its exponentials
            c = Call(17, M, K, 264, 4, 16, act=act, bias=True, mode=mode)
            c.bias[:132] = 3e4
            c.bias[132:] = -3e4
            c.check(c.run(), f"{act} far out")


def test_given_segments_checked_mode_and_streams():
    for M, K, mode in BATCHES:
        c = Call(19, M, K, 264, 6, 16, act="gelu_tanh", bias=True, residual=True, mode=mode)
        want = c.run().clone()
        seg = L.Segments(M, 6)
        L.lora_build_segments(c.ids, M, 6, seg)
        c.y.fill_(7)
        assert torch.equal(c.run(segs=seg), want)
        c.y.fill_(7)
        assert torch.equal(c.run(mode=mode | L.LORA_MODE_CHECKED), want)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        c.y.fill_(7)
        torch.cuda.synchronize()
        assert torch.equal(c.run(stream=st), want)
        c.ids[1] = 6
        with pytest.raises(L.LoraError) as e:
            c.run(mode=mode | L.LORA_MODE_CHECKED)
        assert e.value.status == 8


def test_rows_behind_the_batch_are_kept():
    for M, K, mode in BATCHES:
        c = Call(23, M, K, 264, 6, 16, act="silu", mul=True, mode=mode)
        buf = torch.full((M + 9, 264), 5.0, dtype=torch.bfloat16, device="cuda")
        c.check(c.run(y=buf)[:M], f"M={M}")
        assert (buf[M:] == 5).all()


@pytest.mark.parametrize("M,K,mode", [(20, 256, DEC), (150, 256, DEC), (300, 2048, DEC),
                                      (300, 16384, DEC), (300, 1032, DEC), (800, 256, PRE)])
def test_graph_replays(M, K, mode):
    log(f"linear_act graph M={M} K={K}")
    c = Call(29, M, K, 264, 6, 16, act="silu", bias=True, mul=True, residual=True, mode=mode)
    want = c.run().clone()

    def call():
        _, _, N, r, n = c.dims
        L.lora_linear_act(c.x, c.W, c.A, c.B, c.scale, c.ranks, c.ids, M, K, N, r, n, None, c.epi(),
                          c.y, L.LORA_BF16, mode, c.ws, c.nbytes)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(3):
        c.y.fill_(0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.y, want), rep
        call()
        torch.cuda.synchronize()


@pytest.mark.parametrize("M,K,N,n,r,mode", [
    (9, 256, 264, 6, 16, DEC), (9, 256, 264, 40, 8, DEC), (150, 256, 264, 6, 16, DEC),
    (300, 16384, 264, 6, 16, DEC), (300, 1032, 264, 6, 16, DEC), (800, 256, 264, 6, 16, PRE),
    (800, 256, 264, 6, 64, PRE), (4100, 128, 3080, 40, 32, PRE), (3000, 264, 2056, 9, 8, PRE)])
def test_an_adapter_with_nan_spoils_its_own_rows_alone(M, K, N, n, r, mode):
    log(f"NaN adapter M={M} K={K} n={n} r={r}")
    ids = np.arange(M) * 7 % (n + 1) - 1
    c = Call(37, M, K, N, n, r, act="silu", bias=True, mode=mode, ids=ids, ranks=None)
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
    # (silu of minus infinity is NaN by its formula, of plus infinity infinity)
    assert not torch.isfinite(got[c.ids == 2, N - 1]).any()


@pytest.mark.parametrize("M,K,N,n,r", [(800, 256, 520, 700, 16), (1300, 520, 264, 121, 3), (4100, 128, 3080, 512, 8),
                                       (4100, 128, 3080, 90, 64), (1024, 264, 1032, 64, 32), (777, 136, 264, 1, 40)])
def test_prefill_with_many_adapters(M, K, N, n, r):
    """Tiles of many short runs, each rank bucket."""
    log(f"prefill M={M} n={n} r={r}")
    for f32 in (False, True):
        c = Call(41, M, K, N, n, r, act="gelu", residual=True, f32=f32, mode=PRE)
        c.check(c.run(), f"M={M} n={n} r={r}")
