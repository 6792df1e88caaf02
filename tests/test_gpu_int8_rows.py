"""lora_rmsnorm_int8 and lora_quant_int8 against their formulas in 64 bits.

The integers are exact: rint(127 p / max|p|) of the fp32 p = h * weight (h the fp32 sum), so they
have to be equal.  y_scale of lora_quant_int8 is one fp32 division of a bf16 value: equal too.
Behind the norm it carries the statistics' error, t of test_gpu_norm: a sum of squares in chains of
at most c = d / 8192 * 8 + 86 additions, a square root, a division and two products, (c / 2 + 8)
2^-24; the scale's own product and division add 2^-23.  y adds half a bf16 step, 2^-8.
"""

import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

from .gpu_util import log

pytestmark = pytest.mark.gpu

EPS = 1e-5


def slack(d):
    return (d / 8192 * 8 / 2 + 51) * 2.0 ** -24


def codes64(p, top):
    return torch.round(127.0 * p.double() / top.double().clamp_min(2.0 ** -60)[:, None]).to(torch.int8)


def run(x, res=None, w=None, norm=True, want="sum y", eps=EPS, stream=None):
    M, d = x.shape
    y8 = torch.full((M, d), 99, dtype=torch.int8, device="cuda")
    sc = torch.full((M,), 7.0, device="cuda")
    sum_ = torch.full_like(x, 7.0) if norm and "sum" in want else None
    y = torch.full_like(x, 7.0) if norm and "y" in want else None
    if norm:
        L.lora_rmsnorm_int8(x, res, w, eps, M, d, sum_, y, y8, sc, stream)
    else:
        L.lora_quant_int8(x, M, d, y8, sc, stream)
    torch.cuda.synchronize()
    return sum_, y, y8, sc


def check_norm(got, x, res, w, eps=EPS):
    sum_, y, y8, sc = got
    h = x.float() if res is None else x.float() + res.float()
    p = h if w is None else h * w.float()
    n = h.double() / torch.sqrt((h.double() ** 2).mean(1, keepdim=True) + eps)
    n = n if w is None else n * w.double()
    t = slack(x.shape[1])
    assert torch.equal(y8, codes64(p, p.abs().amax(1)))
    s64 = n.abs().amax(1).clamp_min(2.0 ** -60) / 127.0
    assert ((sc.double() - s64).abs() <= s64 * (t + 2.0 ** -22)).all()
    if sum_ is not None:
        assert torch.equal(sum_.view(torch.int16), h.bfloat16().view(torch.int16))
    if y is not None:
        assert ((y.double() - n).abs() <= n.abs() * (2.0 ** -8 * 1.01 + t) + 2.0 ** -134).all()


def check_plain(got, x):
    _, _, y8, sc = got
    top = x.float().abs().amax(1)
    assert torch.equal(y8, codes64(x, top))
    assert torch.equal(sc, (top.double().clamp_min(2.0 ** -60) / 127.0).float())


def inputs(M, d, res, w, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.empty(s, device="cuda").normal_(0, std, generator=g).bfloat16()

    return r(M, d), (r(M, d) if res else None), (r(d) if w else None)


SHAPES = [(1, 8), (5, 24), (3, 512), (2, 520), (9, 1024), (1500, 1000), (4, 2048), (6, 2056), (129, 4096),
          (64, 4104), (33, 8192), (3, 8200), (17, 11008), (3, 16384), (2, 16392), (1, 40968)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
@pytest.mark.parametrize("res,w", [(True, True), (False, True), (True, False), (False, False)])
def test_norm(shape, res, w):
    log(f"rmsnorm_int8 {shape} {res} {w}")
    x, r, g = inputs(*shape, res, w, sum(shape))
    check_norm(run(x, r, g), x, r, g)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
@pytest.mark.parametrize("std", [1.0, 1e-12, 1e30])
def test_quant(shape, std):
    log(f"quant_int8 {shape} {std}")
    x, _, _ = inputs(*shape, False, False, sum(shape), std)
    check_plain(run(x, norm=False), x)


def test_ties_go_to_the_even_integer():
    # max 2^k * 127: every odd multiple of half a step is a tie; also in bf16's own grid
    v = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 63.5, -63.5, 100.5, 3.5, 126.5] * 8)
    for scale in (1.0, 2.0 ** 40, 2.0 ** -50, 2.0 ** 120):
        x = (v * scale).bfloat16()[None].cuda()
        assert torch.equal(x.double().cpu()[0], v.double() * scale)
        _, _, y8, _ = run(x, norm=False)
        want = torch.round(v).to(torch.int8)
        assert torch.equal(y8.cpu()[0], want)
        check_plain(run(x, norm=False), x)
    # every bf16 value of two binades against every maximum of one
    tops = (1.0 + torch.arange(128) / 128.0).double()
    x = torch.cat([tops[:, None] * 0 + tops, tops[:, None] * 0 - tops / 2, tops[:, None] * 0 + tops / 32], 1)
    x = torch.where(x.abs() > tops[:, None], torch.zeros_like(x), x)
    x = torch.cat([x, tops[:, None], torch.zeros(128, 7).double()], 1).bfloat16().cuda()
    check_plain(run(x, norm=False), x)
    check_norm(run(x), x, None, None)


def test_zero_and_tiny_rows():
    x = torch.zeros(4, 520, dtype=torch.bfloat16, device="cuda")
    x[1] = 2.0 ** -130  # below the floor
    x[2, 3] = 2.0 ** -60
    _, _, y8, sc = run(x, norm=False)
    assert (y8[[0, 1, 3]] == 0).all() and int(y8[2, 3]) == 127 and int(y8[2].abs().sum()) == 127
    assert torch.equal(sc, torch.full_like(sc, float(torch.tensor(2.0 ** -60 / 127, dtype=torch.float64))))
    sum_, y, y8, sc = run(x)
    assert (y8[[0, 3]] == 0).all() and (y[0] == 0).all()
    assert torch.equal(sc[[0, 3]], torch.full_like(sc[:2], 2.0 ** -60 / 127))
    # a row of zeros beside others, with eps alone under the root
    x2, r, w = inputs(5, 1032, False, True, 3)
    x2[2] = 0
    got = run(x2, None, w)
    assert (got[2][2] == 0).all() and torch.isfinite(got[3]).all()


@pytest.mark.parametrize("d", [512, 2048, 4096, 40968])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_rows_without_a_scale(d, value):
    x, r, w = inputs(6, d, True, True, d)
    x[2, d - 1] = value
    good = [0, 1, 3, 4, 5]
    for norm in (True, False):
        _, _, y8, sc = run(x, r if norm else None, w if norm else None, norm=norm)
        assert torch.isnan(sc[2]) and (y8[2] == 0).all() and torch.isfinite(sc[good]).all()
        _, _, ref, rsc = run(x[good].contiguous(), r[good].contiguous() if norm else None,
                             w if norm else None, norm=norm)
        assert torch.equal(y8[good], ref) and torch.equal(sc[good], rsc)
    # an infinite or NaN weight reaches every row's scale
    w[1] = value
    _, _, y8, sc = run(x[good].contiguous(), None, w)
    assert torch.isnan(sc).all() and (y8 == 0).all()


@pytest.mark.parametrize("d", [512, 4096, 40968])
def test_products_beyond_fp32(d):
    """h w overflows where n does not: the integers are those of n."""
    x, _, w = inputs(3, d, False, True, d + 1)
    x = (x.float() * 2.0 ** 100).bfloat16()
    w = (w.float() * 2.0 ** 40).bfloat16()
    _, y, y8, sc = run(x, None, w)
    h = x.double()
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * w.double()
    q = 127.0 * n / n.abs().amax(1, keepdim=True)
    assert ((y8.double() - q).abs() <= 0.5 + 127 * 4 * slack(d)).all()
    assert ((sc.double() * 127 / n.abs().amax(1) - 1).abs() <= slack(d) + 2.0 ** -22).all()
    assert torch.isfinite(y.float()).all()


def test_in_place_sum_and_outputs_of_one_kind():
    x, r, w = inputs(37, 1032, True, True, 9)
    want = run(x, r, w)
    a, b = x.clone(), r.clone()
    y8, sc = torch.empty(37, 1032, dtype=torch.int8, device="cuda"), torch.empty(37, device="cuda")
    L.lora_rmsnorm_int8(a, b, w, EPS, 37, 1032, b, a, y8, sc)
    torch.cuda.synchronize()
    for g, e in zip((b, a, y8, sc), want):
        assert torch.equal(g, e)
    assert torch.equal(run(x, r, w, want="")[2], want[2])


def test_rows_behind_the_last_are_left():
    x, r, w = inputs(9, 264, True, True, 4)
    y8 = torch.full((9, 264), 55, dtype=torch.int8, device="cuda")
    sc = torch.full((9,), 5.0, device="cuda")
    L.lora_quant_int8(x, 6, 264, y8, sc)
    torch.cuda.synchronize()
    assert (y8[6:] == 55).all() and (sc[6:] == 5.0).all()
    check_plain((None, None, y8[:6], sc[:6]), x[:6])


def test_side_stream_and_graph():
    x, r, w = inputs(70, 2056, True, True, 5)
    want_n, want_q = run(x, r, w), run(x, norm=False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(x, r, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want_n))
    y8, sc = torch.empty_like(want_n[2]), torch.empty_like(want_n[3])
    q8, qc = torch.empty_like(y8), torch.empty_like(sc)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lora_rmsnorm_int8(x, r, w, EPS, 70, 2056, None, None, y8, sc)
        L.lora_quant_int8(x, 70, 2056, q8, qc)
    for _ in range(3):
        y8.zero_(), q8.zero_(), sc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y8, want_n[2]) and torch.equal(sc, want_n[3])
        assert torch.equal(q8, want_q[2]) and torch.equal(qc, want_q[3])
        torch.ones(1000, device="cuda").sum()


def test_rows_past_2_31_elements():
    M, d = 66000, 32776  # 2.16e9 elements
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough memory")
    log("quant_int8 past 2^31 elements")
    x = torch.empty(M, d, dtype=torch.bfloat16, device="cuda").normal_()
    y8, sc = torch.empty(M, d, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    L.lora_quant_int8(x, M, d, y8, sc)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, M // 2, (1 << 31) // d, (1 << 31) // d + 1, M - 1], device="cuda")
    check_plain((None, None, y8[rows], sc[rows]), x[rows])
