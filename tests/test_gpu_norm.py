"""lora_rmsnorm against its formula in 64 bits.

Tolerances.  n is computed in fp32 from h (one rounding of the exact sum), a sum of squares in
chains of at most c = d / 8192 * 8 + 86 additions (a lane's elements, the wave's six steps, the
row's 16 waves), a square root, a division and two products: relative error at most
(c / 2 + 8) 2^-24 = t.  y adds half a bf16 step, 2^-8.  A code adds half an E4M3 step: 2^-4 of
the value, or 2^-10 (half the smallest subnormal) in units of the scale.
"""

import numpy as np
import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

from .gpu_util import log

pytestmark = pytest.mark.gpu

EPS = 1e-5
NAN_FILL = 0x7F  # an E4M3 NaN


def formula(x, res, w, eps=EPS):
    """(n in float64, bf16 sum): h is the fp32 sum."""
    h = x.float() if res is None else x.float() + res.float()
    s = h.bfloat16()
    h = h.double()
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return (n if w is None else n * w.double()), s


def slack(d):
    return (d / 8192 * 8 / 2 + 51) * 2.0 ** -24


def run(x, res, w, want="sum y y8", eps=EPS, stream=None):
    M, d = x.shape
    sum_ = torch.full_like(x, 7.0) if "sum" in want else None
    y = torch.full_like(x, 7.0) if "y" in want.split() else None
    y8 = torch.full((M, d), NAN_FILL, dtype=torch.uint8, device="cuda") if "y8" in want else None
    sc = torch.full((M,), 7.0, device="cuda") if "y8" in want else None
    L.lora_rmsnorm(x, res, w, eps, M, d, sum_, y, y8, sc, stream)
    torch.cuda.synchronize()
    return sum_, y, (None if y8 is None else y8.view(torch.float8_e4m3fn)), sc


def check(got, x, res, w, eps=EPS):
    sum_, y, y8, sc = got
    n, s = formula(x, res, w, eps)
    t = slack(x.shape[1])
    if sum_ is not None:
        assert torch.equal(sum_.view(torch.int16), s.view(torch.int16))
    if y is not None:
        # (below the normal range of bf16 a step is 2^-133)
        assert ((y.double() - n).abs() <= n.abs() * (2.0 ** -8 * 1.01 + t) + 2.0 ** -134).all()
    if y8 is not None:
        s64 = n.abs().amax(1).clamp_min(2.0 ** -60) / 448.0
        assert ((sc.double() - s64).abs() <= s64 * (t + 2.0 ** -22)).all()
        q = n / s64[:, None]
        assert torch.isfinite(y8.float()).all()
        off = (y8.double() - q).abs()
        assert (off <= torch.maximum(q.abs() * 2.0 ** -4, torch.full_like(q, 2.0 ** -10)) * (1 + 2.0 ** -12)
                + q.abs() * 2 * t).all(), float(off.max())


def inputs(M, d, res, w, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.empty(s, device="cuda").normal_(0, std, generator=g).bfloat16()

    return r(M, d), (r(M, d) if res else None), (r(d) if w else None)


SHAPES = [(1, 8), (5, 24), (3, 512), (2, 520), (9, 1024), (7, 1032), (4, 2048), (6, 2056),
          (129, 4096), (64, 4104), (33, 8192), (3, 8200), (17, 11008), (3, 16384), (2, 16392),
          (1, 40968), (1023, 256), (2500, 1536), (3000, 4096), (2200, 11008)]


@pytest.mark.parametrize("M,d", SHAPES)
@pytest.mark.parametrize("res,w,want", [(True, True, "sum y y8"), (False, True, "y"),
                                        (True, False, "y8"), (False, False, "sum y8")])
def test_matches_formula(M, d, res, w, want):
    log(f"rmsnorm M={M} d={d} residual={res} weight={w} outputs={want}")
    x, r, wt = inputs(M, d, res, w, 1000 + M + d)
    check(run(x, r, wt, want), x, r, wt)


@pytest.mark.parametrize("d", [64, 1032, 4096, 11008, 16400])
@pytest.mark.parametrize("std", [1e-30, 1e-12, 1e-3, 1e4, 1e25])
def test_small_and_large_magnitudes(d, std):
    """Rows whose squares underflow (eps decides) and rows whose squares overflow fp32."""
    log(f"rmsnorm d={d} std={std}")
    x, r, wt = inputs(3, d, True, False, 11, std)
    check(run(x, r, wt), x, r, wt)


@pytest.mark.parametrize("d", [64, 1032, 4096, 11008, 16400])
@pytest.mark.parametrize("x2,w2,eps", [(100, 60, EPS), (100, -60, EPS), (3, 125, EPS), (66, 0, 1e38),
                                       (62.5, 0, 3e38), (-40, 0, 3e38)])
def test_ends_of_the_range(d, x2, w2, eps):
    """Finite n whose h w overflows fp32, and an eps that counts next to squares that do."""
    log(f"rmsnorm d={d} x 2^{x2} w 2^{w2} eps {eps}")
    x, _, wt = inputs(3, d, False, True, 12, 2.0 ** x2)
    wt = (wt.double() * 2.0 ** (w2 - x2)).bfloat16()
    got = run(x, None, wt, eps=eps)
    # rows whose n itself leaves fp32 (8 sigma at w 2^125): y is infinite there, no scale exists
    n = formula(x, None, wt, eps)[0].abs()
    lim, t = 2.0 ** 128, slack(d)
    off = n.amax(1) >= lim * (1 - t)
    keep = ~off
    check((got[0][keep], got[1][keep], got[2][keep], got[3][keep]), x[keep], None, wt, eps)
    y, no = got[1][off], n[off]
    assert torch.isinf(y[no >= lim * (1 + t)]).all()
    fine = no < lim * (1 - 2.0 ** -8)
    err = (y.double().abs() - no)[fine].abs()
    assert (err <= no[fine] * (2.0 ** -8 * 1.01 + t)).all()
    sure = n.amax(1) >= lim * (1 + t)
    assert torch.isnan(got[3][sure]).all() and torch.isnan(got[2][sure].float()).all()


@pytest.mark.parametrize("d", [512, 1024, 4096, 11008, 16392])
def test_special_rows(d):
    """Zero rows, infinities and NaN touch their own row alone."""
    log(f"special rows d={d}")
    x, r, wt = inputs(9, d, True, True, 5)
    wt = wt.abs() + 0.5
    x[1] = 0
    r[1] = 0
    x[2, 3] = float("inf")
    x[4, d - 1] = float("nan")
    x[6, 0] = float("-inf")
    x[7, :] = 0
    r[7, :] = 0
    x[7, d // 2] = 3.0
    sum_, y, y8, sc = run(x, r, wt)
    ok = [0, 1, 3, 5, 7, 8]
    check((sum_[ok], y[ok], y8[ok], sc[ok]), x[ok], r[ok], wt)
    assert (y[1] == 0).all() and (y8[1].float() == 0).all()
    n, s = formula(x, r, wt)
    assert torch.equal(torch.isnan(y), torch.isnan(n.bfloat16()))
    assert torch.equal(y[2].nan_to_num(9.0), n[2].bfloat16().nan_to_num(9.0))
    for m in (2, 4, 6):
        assert torch.isnan(sc[m]) and torch.isnan(y8[m].float()).all()
    assert torch.equal(torch.isnan(sum_), torch.isnan(s))


@pytest.mark.parametrize("M,d", [(3, 512), (5, 4096), (3000, 4096), (2, 16400)])
def test_in_place(M, d):
    """sum and y written over residual and x give the separate buffers' bits."""
    x, r, wt = inputs(M, d, True, True, 21)
    a = run(x, r, wt)
    x2, r2 = x.clone(), r.clone()
    y8, sc = torch.empty(M, d, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(M, device="cuda")
    L.lora_rmsnorm(x2, r2, wt, EPS, M, d, r2, x2, y8, sc)
    torch.cuda.synchronize()
    assert torch.equal(r2, a[0]) and torch.equal(x2, a[1])
    assert torch.equal(y8.view(torch.uint8), a[2].view(torch.uint8)) and torch.equal(sc, a[3])


@pytest.mark.parametrize("d", [64, 2056, 11008])
def test_writes_only_its_rows(d):
    """Buffers longer than M rows keep what lies behind."""
    M = 5
    x, r, wt = inputs(M + 3, d, True, True, 31)
    y = torch.full((M + 3, d), 9.0, dtype=torch.bfloat16, device="cuda")
    s = torch.full_like(y, 9.0)
    y8 = torch.full((M + 3, d), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.full((M + 3,), 9.0, device="cuda")
    L.lora_rmsnorm(x, r, wt, EPS, M, d, s, y, y8, sc)
    torch.cuda.synchronize()
    check((s[:M], y[:M], y8[:M].view(torch.float8_e4m3fn), sc[:M]), x[:M], r[:M], wt)
    assert (y[M:] == 9).all() and (s[M:] == 9).all() and (y8[M:] == 0x55).all() and (sc[M:] == 9).all()


def test_every_batch_size_of_one_matrix():
    """Slices of one matrix (the launch depends on the number of rows) hold the formula."""
    x, r, wt = inputs(4500, 4096, True, True, 41)
    for m0, M in ((0, 1), (17, 5), (100, 300), (0, 1500), (0, 4500)):
        check(run(x[m0:m0 + M], r[m0:m0 + M], wt), x[m0:m0 + M], r[m0:m0 + M], wt)


def test_offsets_past_32_bits():
    M, d = 530000, 4096  # 2.17e9 elements
    log(f"rmsnorm M={M} d={d}")
    x = torch.empty(M, d, dtype=torch.bfloat16, device="cuda")
    tail, _, wt = inputs(40, d, False, True, 51)
    x.zero_()
    x[-40:] = tail
    x[:3] = tail[:3]
    _, y, y8, sc = run(x, None, wt, "y y8")
    check((None, y[-40:], y8[-40:], sc[-40:]), tail, None, wt)
    check((None, y[:3], y8[:3], sc[:3]), tail[:3], None, wt)


def test_other_stream_and_graph():
    x, r, wt = inputs(70, 4096, True, True, 61)
    want = run(x, r, wt)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = run(x, r, wt, stream=st)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    out = (torch.empty_like(x), torch.empty_like(x),
           torch.empty(70, 4096, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(70, device="cuda"))

    def call():
        L.lora_rmsnorm(x, r, wt, EPS, 70, 4096, *out)

    with torch.cuda.stream(st):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(3):
        for o in out:
            o.view(torch.uint8).fill_(0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), rep
        call()
        torch.cuda.synchronize()


@pytest.mark.parametrize("d", [64, 512, 1024, 1032, 4096, 11008, 16384, 16392])
@pytest.mark.parametrize("kind", ["nan", "inf times zero", "inf", "none"])
def test_special_weights(d, kind):
    """n that is NaN or infinite in one column leaves its row without a scale: NaN in y_scale and
    every code, as max|n| of the formula; y is spoilt in that column alone."""
    log(f"special weights d={d} {kind}")
    x, r, wt = inputs(5, d, True, True, 71)
    base = run(x, r, wt)
    at = d - 3
    hit = [0, 1, 2, 3, 4]
    if kind == "nan":
        wt[at] = float("nan")
    elif kind == "inf":
        wt[at] = float("-inf")
        x[:, at], r[:, at] = 2.0, 1.0
    elif kind == "inf times zero":
        wt[at] = float("inf")
        x[:, at], r[:, at] = 1.0, -1.0
    else:
        hit = []
    n, _ = formula(x, r, wt)
    _, y, y8, sc = run(x, r, wt)
    assert torch.equal(torch.isnan(y), torch.isnan(n)) and torch.equal(torch.isinf(y), torch.isinf(n))
    assert torch.isnan(sc[hit]).all() and torch.isnan(y8[hit].float()).all()
    if not hit:
        assert torch.equal(sc, base[3]) and torch.equal(y8.view(torch.uint8), base[2].view(torch.uint8))


@pytest.mark.parametrize("d", [8, 12296])
def test_most_rows(d):
    """LORA_MAX_ROWS rows in place, also of a d whose blocks hold 1024 threads (2^32 in all)."""
    M = L.LORA_MAX_ROWS
    if torch.cuda.mem_get_info()[0] < M * d * 2 + (8 << 30):
        pytest.skip("not enough memory")
    log(f"rmsnorm M={M} d={d}")
    x = torch.zeros(M, d, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, 2 ** 21 - 1, 2 ** 21, 2 ** 21 + 1, M - 2, M - 1]
    tail, _, wt = inputs(len(at), d, False, True, 81)
    for i, m in enumerate(at):
        x[m] = tail[i]
    sc = torch.full((M,), 7.0, device="cuda")
    y8 = torch.full((M * d,), 0x55, dtype=torch.uint8, device="cuda") if d == 8 else None
    L.lora_rmsnorm(x, None, wt, EPS, M, d, None, x, y8, None if y8 is None else sc)
    torch.cuda.synchronize()
    if y8 is not None:
        y8 = y8.view(M, d).view(torch.float8_e4m3fn)
        check((None, x[at], y8[at], sc[at]), tail, None, wt)
        assert (sc == 2.0 ** -60 / 448).sum() == M - len(at)
    else:
        check((None, x[at], None, None), tail, None, wt)
    assert (x[3:2 ** 21 - 1] == 0).all()
    del x, y8, sc
    torch.cuda.empty_cache()
