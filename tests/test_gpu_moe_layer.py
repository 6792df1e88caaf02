"""lora_moe_layer against its formula in 64 bits.

Tolerances, worst case element by element.  A projection of k inputs: c(k) = (k / 8 + 64 + 16) 2^-24 of the
sum of its absolute products, base and delta (MFMA chains with at least eight products per rounding,
the expand's r_max products, at most 16 splits).  The activations' slopes are at most 1.13 and their own
error |z| 2^-20 (tests/epilogue_util.py).  h adds its rounding: 2^-8 of itself with y in bf16, 2^-24 with
y in fp32 (three bf16 parts).  What dh makes of y is |dh| through the absolute weights.  Then a product and
a sum per slot, the residual, and y's rounding: 2^-8 or 2^-24.

That bound is loose for y in bf16 (the roundings of h seldom agree), so the integer cases, whose every sum
and hidden value is exact, have to be equal."""

import numpy as np
import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

from .epilogue_util import ACTS, act64, assert_within
from .gpu_util import log

pytestmark = pytest.mark.gpu


def c_of(k):
    return (k / 8 + 80) * 2.0 ** -24


class Layer:
    """One layer's inputs and its lora_moe_layer call."""

    def __init__(self, seed, M, top_k, E, d, ff, n, r, act="silu", residual=True, f32=False, ids=None, topk=None,
                 weights=True, ranks="mixed", holes=0.15):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)

        def normal(*s, std=1.0):
            return torch.empty(s, device="cuda").normal_(0, std, generator=g)

        def ints(v):
            return torch.as_tensor(np.ascontiguousarray(v), dtype=torch.int32, device="cuda").contiguous()

        self.dims, self.act, self.f32 = (M, top_k, E, d, ff, r, n), act, f32
        self.type = torch.float32 if f32 else torch.bfloat16
        self.ids = ints(rng.integers(-1, n, M) if ids is None else ids)
        if topk is None:
            topk = np.stack([rng.permutation(max(E, top_k))[:top_k] % E for _ in range(M)]) if M else np.zeros((0, top_k))
            topk[rng.random((M, top_k)) < holes] = -1
        self.topk_ids = ints(topk)
        self.topk_w = torch.rand(M, top_k, device="cuda", generator=g) + 0.1 if weights else None
        rk = rng.integers(1, r + 1, n)
        self.ranks = ints(rk) if ranks == "mixed" else None
        full = rk if ranks == "mixed" else np.full(n, r)
        self.rank_of = full
        self.scale = torch.as_tensor(16.0 / full, dtype=torch.float32, device="cuda")
        kept = torch.arange(r, device="cuda") < torch.as_tensor(full, device="cuda")[:, None]
        self.x = normal(M, d).bfloat16()
        self.W, self.A, self.B = {}, {}, {}
        for p, (a, b) in dict(g=(d, ff), u=(d, ff), d=(ff, d)).items():
            self.W[p] = normal(E, a, b, std=a ** -0.5).bfloat16()
            self.A[p] = (normal(n, E, a, r, std=a ** -0.5) * kept[:, None, None, :]).bfloat16()
            self.B[p] = (normal(n, E, r, b, std=0.5 * r ** -0.5) * kept[:, None, :, None]).bfloat16()
        self.residual = normal(M, d).to(self.type) if residual else None
        self.y = torch.full((M, d), 7.0, dtype=self.type, device="cuda")
        self.ws, self.nbytes = L.moe_layer_workspace(M, top_k, E, d, ff, r, n)
        self.ws.fill_(255)  # the workspace's contents need no initialisation

    def enqueue(self, y=None, stream=None, mode=L.LORA_MODE_AUTO):
        M, k, E, d, ff, r, n = self.dims
        w = L.lora_moe_weights(*(t[p] for p in "gud" for t in (self.W, self.A, self.B)))
        L.lora_moe_layer(self.x, w, self.scale, self.ranks, self.ids, self.topk_ids, self.topk_w, self.residual, M, k,
                         E, d, ff, r, n, ACTS.index(self.act), self.y if y is None else y,
                         L.LORA_F32 if self.f32 else L.LORA_BF16, mode, self.ws, self.nbytes, stream)

    def run(self, y=None, **kw):
        self.enqueue(y, **kw)
        torch.cuda.synchronize()
        return self.y if y is None else y

    def project(self, p, e, v, dv, rows):
        """(z, |error|) of the rows v through expert e's projection p"""
        n = self.dims[6]
        W = self.W[p][e].double()
        z, S, dz = v @ W, v.abs() @ W.abs(), dv @ W.abs()
        for i in sorted(set(self.ids[rows].tolist())):
            if not 0 <= i < n:
                continue
            at = (self.ids[rows] == i).nonzero()[:, 0]
            k = int(self.rank_of[i])
            a, b, s = self.A[p][i, e, :, :k].double(), self.B[p][i, e, :k].double(), float(self.scale[i])
            z[at] += s * ((v[at] @ a) @ b)
            S[at] += abs(s) * ((v[at].abs() @ a.abs()) @ b.abs())
            dz[at] += abs(s) * ((dv[at] @ a.abs()) @ b.abs())
        return z, dz + c_of(v.shape[1]) * S

    def want(self):
        M, top_k, E, d, ff, r, n = self.dims
        x = self.x.double()
        y = torch.zeros(M, d, dtype=torch.float64, device="cuda")
        dy, size = torch.zeros_like(y), torch.zeros_like(y)
        half = 2.0 ** -24 if self.f32 else 2.0 ** -8
        for e in sorted(set(self.topk_ids.flatten().tolist())):
            if not 0 <= e < E:
                continue
            m, j = (self.topk_ids == e).nonzero(as_tuple=True)
            v = x[m]
            g, dg = self.project("g", e, v, torch.zeros_like(v), m)
            u, du = self.project("u", e, v, torch.zeros_like(v), m)
            a, da = act64(g, self.act), 1.13 * dg
            if self.act != "none":
                da = da + 2.0 ** -20 * g.abs()
            h = a * u
            dh = da * (u.abs() + du) + a.abs() * du
            dh = dh + (h.abs() + dh) * (half + 2.0 ** -23)
            z, dz = self.project("d", e, h, dh, m)
            w = torch.ones(len(m), 1, dtype=torch.float64, device="cuda") if self.topk_w is None else \
                self.topk_w[m, j].double()[:, None]
            y.index_add_(0, m, z * w)
            dy.index_add_(0, m, dz * w.abs())
            size.index_add_(0, m, (z * w).abs())
        if self.residual is not None:
            y, size = y + self.residual.double(), size + self.residual.double().abs()
        dy = dy + (top_k + 4) * 2.0 ** -24 * size
        return y, dy + (y.abs() + dy) * half + 1e-37

    def check(self, got, what):
        assert_within(got, *self.want(), what)


# M, top_k, E, d, ff, n, r
SHAPES = [
    (1, 1, 1, 128, 128, 1, 8), (1, 4, 32, 256, 400, 8, 16), (3, 2, 8, 144, 272, 3, 8), (1, 8, 64, 128, 1040, 1, 64),
    (5, 3, 5, 272, 128, 40, 24), (23, 2, 8, 1040, 560, 40, 24), (16, 4, 16, 512, 512, 2, 32),
    (33, 4, 4, 384, 1408, 33, 56), (64, 4, 32, 256, 384, 8, 16), (100, 2, 6, 2064, 144, 7, 40),
    (65, 1, 3, 160, 2880, 100, 16), (7, 64, 70, 128, 144, 4, 8), (300, 2, 4, 176, 208, 5, 16),
    (50, 2, 700, 128, 144, 3, 8), (33, 2, 128, 144, 128, 90, 64), (16, 4, 66, 128, 272, 20, 16),
    (17, 2, 6, 144, 272, 9, 16), (99, 3, 5, 272, 144, 11, 24), (241, 1, 8, 128, 400, 64, 64),
    (2, 2, 4096, 128, 128, 2, 8), (9, 3, 700, 144, 128, 3, 8), (130, 8, 9, 128, 256, 500, 8), (40, 5, 3, 128, 144, 2, 8),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
def test_matches_64_bits(shape, f32):
    at = SHAPES.index(shape)
    log(f"moe_layer {shape} f32={f32}")
    c = Layer(50 + at, *shape, act=ACTS[at % 5], residual=at % 3 != 1, f32=f32, weights=at % 4 != 2,
              ranks="mixed" if at % 2 else "full")
    c.check(c.run(), f"{shape} {f32}")


@pytest.mark.parametrize("shape", [(64, 4, 32, 2880, 2880, 8, 16), (1, 4, 32, 2880, 2880, 8, 16)])
def test_matches_64_bits_at_full_width(shape):
    log(f"moe_layer {shape}")
    for f32 in (True, False):
        c = Layer(3, *shape, f32=f32, holes=0.0)
        c.check(c.run(), f"{shape} {f32}")
        del c
        torch.cuda.empty_cache()


@pytest.mark.parametrize("shape", [(1, 2, 8, 128, 144, 2, 8), (37, 3, 6, 272, 400, 9, 16), (64, 4, 8, 1040, 656, 3, 24),
                                   (290, 4, 5, 256, 128, 12, 64)], ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
def test_integers_are_exact(shape, f32):
    """About four +-1 in every column of gate and up, few in the adapters: hidden values are integers up to
    256, and every sum is exact."""
    M, top_k, E, d, ff, n, r = shape
    log(f"moe_layer integers {shape} {f32}")
    c = Layer(11, *shape, act="relu", f32=f32)
    g = torch.Generator(device="cuda").manual_seed(12)

    def signs(t, share):
        keep = torch.rand(t.shape, device="cuda", generator=g) < share
        return (keep * (1.0 - 2.0 * torch.randint(0, 2, t.shape, device="cuda", generator=g))).bfloat16()

    c.x = torch.randint(-1, 2, c.x.shape, device="cuda", generator=g).bfloat16()
    for p, k in dict(g=d, u=d, d=ff).items():
        c.W[p], c.A[p], c.B[p] = signs(c.W[p], 4.0 / k), signs(c.A[p], 2.0 / k), signs(c.B[p], 0.5 / r)
    c.ranks, c.rank_of = None, np.full(n, r)
    c.scale = 1.0 - 2.0 * torch.randint(0, 2, (n,), device="cuda", generator=g).float()
    c.topk_w = 2.0 ** torch.randint(-2, 2, (M, top_k), device="cuda", generator=g).float()
    if c.residual is not None:
        c.residual = torch.randint(-50, 50, (M, d), device="cuda", generator=g).to(c.type)
    y = torch.zeros(M, d, dtype=torch.float64, device="cuda")
    for e in range(E):
        m, j = (c.topk_ids == e).nonzero(as_tuple=True)
        if len(m) == 0:
            continue
        zero = torch.zeros(len(m), d, dtype=torch.float64, device="cuda")
        h = torch.relu(c.project("g", e, c.x[m].double(), zero, m)[0]) * c.project("u", e, c.x[m].double(), zero, m)[0]
        assert h.abs().max() <= 256
        z = c.project("d", e, h, torch.zeros_like(h), m)[0]
        y.index_add_(0, m, z * c.topk_w[m, j].double()[:, None])
    if c.residual is not None:
        y += c.residual.double()
    assert (y.abs().max() < 2 ** 20) and y.abs().max() > 0
    assert torch.equal(c.run(), y.to(c.type))


CALLS = [(1, 4, 32, 128, 144, 3, 16), (30, 2, 4, 272, 144, 5, 8), (90, 3, 7, 128, 400, 60, 24)]


@pytest.mark.parametrize("shape", CALLS, ids=lambda c: "x".join(map(str, c)))
def test_tokens_without_experts_bad_ids_and_repeats(shape):
    M, top_k, E = shape[:3]
    rng = np.random.default_rng(4)
    for f32 in (False, True):
        # no expert at all: the residual, or zeros
        for residual in (True, False):
            c = Layer(21, *shape, f32=f32, residual=residual, topk=np.full((M, top_k), -1))
            assert torch.equal(c.run(), c.residual if residual else torch.zeros_like(c.y))
        # ids and experts outside their range, a token that names one expert in every slot
        topk = rng.integers(-1, E, (M, top_k))
        topk[0, :] = 0
        topk[-1, -1] = E
        topk[M // 2, 0] = 2 ** 31 - 1
        topk[M // 3, 0] = -2 ** 31
        ids = rng.integers(-1, shape[5], M)
        ids[M // 2], ids[-1] = shape[5], -7
        c = Layer(22, *shape, f32=f32, topk=topk, ids=ids)
        c.check(c.run(), f"bad ids {shape}")
        c = Layer(23, *shape, f32=f32, ids=np.full(M, -1))
        c.check(c.run(), f"bare base {shape}")


@pytest.mark.parametrize("shape", CALLS, ids=lambda c: "x".join(map(str, c)))
def test_what_no_token_names_does_not_leak(shape):
    M, top_k, E, d, ff, n, r = shape
    rng = np.random.default_rng(5)
    for f32 in (False, True):
        c = Layer(31, *shape, f32=f32, topk=2 * rng.integers(0, (E + 1) // 2, (M, top_k)), ids=rng.integers(-1, 2, M))
        want = c.run().clone()
        for p in "gud":
            c.W[p][1::2] = float("nan")
            c.A[p][:, 1::2] = float("nan")
            c.B[p][:, 1::2] = float("inf")
            c.A[p][2:], c.B[p][2:] = float("nan"), float("nan")
        c.scale[2:] = float("nan")
        c.y.fill_(3)
        assert torch.equal(c.run(), want)


def test_nan_and_infinity_stay_in_their_token():
    shape = (40, 2, 4, 128, 144, 5, 16)
    for value in (float("nan"), float("inf")):
        for f32 in (False, True):
            c = Layer(33, *shape, f32=f32, holes=0.0)
            want = c.run().clone()
            c.x[7, 100] = value
            got = c.run()
            keep = torch.arange(40, device="cuda") != 7
            assert torch.equal(got[keep], want[keep]) and torch.isnan(got[7]).all()
            # an adapter's: the tokens that carry it
            c = Layer(33, *shape, f32=f32, holes=0.0)
            c.B["u"][1, :, 0, 5] = float("nan")
            got = c.run()
            hit = c.ids == 1
            assert hit.any() and torch.equal(got[~hit], want[~hit]) and torch.isnan(got[hit]).all()


@pytest.mark.parametrize("shape", CALLS, ids=lambda c: "x".join(map(str, c)))
def test_in_place_streams_checked_mode_rows_behind_and_graph(shape):
    M = shape[0]
    for f32 in (False, True):
        c = Layer(41, *shape, f32=f32)
        want = c.run().clone()
        c.check(want, str(shape))
        for _ in range(2):  # the same bits again
            c.y.fill_(1)
            assert torch.equal(c.run(), want)
        c.y.fill_(1)
        assert torch.equal(c.run(mode=L.LORA_MODE_CHECKED | L.LORA_MODE_DECODE), want)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        c.y.fill_(1)
        torch.cuda.synchronize()
        assert torch.equal(c.run(stream=st), want)
        buf = torch.full((M + 5, shape[3]), 5.0, dtype=c.type, device="cuda")
        assert torch.equal(c.run(y=buf)[:M], want) and (buf[M:] == 5).all()
        keep, c.residual = c.residual, c.residual.clone()
        assert torch.equal(c.run(y=c.residual), want)
        c.residual = keep
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.enqueue()
        for _ in range(3):
            c.y.fill_(0)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.y, want)
            assert torch.equal(c.run(), want)
        bad = c.topk_ids.clone()
        c.topk_ids[0, 0] = shape[2]
        with pytest.raises(L.LoraError) as e:
            c.run(mode=L.LORA_MODE_CHECKED)
        assert e.value.status == 8
        c.topk_ids = bad
        c.ids[0] = shape[5]
        with pytest.raises(L.LoraError) as e:
            c.run(mode=L.LORA_MODE_CHECKED)
        assert e.value.status == 8


def test_two_calls_at_once_on_their_own_workspaces():
    a, b = (Layer(s, 30, 2, 4, 272, 144, 5, 8) for s in (61, 62))
    want_a, want_b = a.run().clone(), b.run().clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.y.fill_(0), b.y.fill_(0)
        torch.cuda.synchronize()
        a.enqueue(stream=s1)
        b.enqueue(stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a.y, want_a) and torch.equal(b.y, want_b)


def test_the_largest_batch():
    """LORA_MOE_MAX_PAIRS pairs; one expert takes most of them."""
    M, top_k, E = 2048, 4, 5
    log("moe_layer largest batch")
    topk = np.random.default_rng(1).integers(0, E, (M, top_k))
    topk[:, 0] = 2
    for f32 in (False, True):
        c = Layer(71, M, top_k, E, 128, 144, 20, 8, f32=f32, topk=topk)
        c.check(c.run(), "largest batch")


def test_weights_past_4_gib():
    """64-bit addresses in W and the adapters of the last experts."""
    M, top_k, E, d, ff, n, r = 3, 2, 600, 2048, 2048, 3, 64
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("not enough memory")
    log("moe_layer past 4 GiB")
    c = Layer.__new__(Layer)
    small = Layer(81, M, top_k, 2, d, ff, n, r, f32=True, topk=[[0, 1], [1, 0], [1, 1]], ids=[2, 0, -1])
    want = small.run().clone()
    c.__dict__.update(small.__dict__)
    c.dims = (M, top_k, E, d, ff, r, n)
    c.W, c.A, c.B = {}, {}, {}
    for p in "gud":
        c.W[p] = torch.empty((E,) + small.W[p].shape[1:], dtype=torch.bfloat16, device="cuda")
        c.W[p][1], c.W[p][E - 1] = small.W[p][0], small.W[p][1]
        for t, s in ((c.A, small.A), (c.B, small.B)):
            t[p] = torch.empty((n, E) + s[p].shape[2:], dtype=torch.bfloat16, device="cuda")
            t[p][:, 1], t[p][:, E - 1] = s[p][:, 0], s[p][:, 1]
    assert c.W["g"].numel() > 1 << 31
    c.topk_ids = torch.tensor([[1, E - 1], [E - 1, 1], [E - 1, E - 1]], dtype=torch.int32, device="cuda")
    c.ws, c.nbytes = L.moe_layer_workspace(M, top_k, E, d, ff, r, n)
    got = c.run(y=torch.empty_like(want))
    # (more experts, the same pairs: the split of K may differ, not the sums' sizes)
    y, bound = small.want()
    assert ((got.double() - y).abs() <= bound).all()
