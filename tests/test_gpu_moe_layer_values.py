"""lora_moe_layer on values that show its arithmetic: infinities in the down projection, hidden values of 16 bits."""

import numpy as np
import pytest
import torch

from .gpu_util import log
from .test_gpu_moe_layer import Layer

pytestmark = pytest.mark.gpu

# M, top_k, E, d, ff, n, r: blocks of 16, 32 and 64 rows, one split of K and many
SHAPES = [(1, 4, 32, 256, 400, 3, 16), (6, 1, 2, 128, 2064, 2, 8), (30, 2, 4, 272, 144, 5, 8),
          (90, 3, 7, 128, 400, 60, 24), (300, 2, 4, 176, 208, 5, 64)]


@pytest.mark.parametrize("where", ["W", "A", "both"])
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "x".join(map(str, c)))
def test_infinite_down_weights_follow_the_formula(shape, f32, where):
    """A finite hidden value times an infinity is an infinity of its sign, whatever bits the value has; NaN
    only where infinities of both signs (or one and a zero) meet.  Elements without one keep their bound."""
    M, top_k, E, d, ff, n, r = shape
    log(f"moe_layer infinities {shape} f32={f32} {where}")
    c = Layer(91, *shape, act="gelu", f32=f32, holes=0.0, ids=n - 1 - np.arange(M) % (n + 1))
    inf = float("inf")
    if where != "A":
        for e in range(E):
            c.W["d"][e, (7 * e + 3) % ff, 5] = inf
            c.W["d"][e, ff - 1, 64 + e % 32] = -inf
            c.W["d"][e, 0, d - 1], c.W["d"][e, ff // 2, d - 1] = inf, inf
    if where != "W":
        c.A["d"][n - 1, :, ff // 3, 0] = inf
        if n > 1:
            c.A["d"][0, E // 2, 1, 0] = -inf
    got = c.run().double()
    want, bound = c.want()
    fine = want.isfinite()
    assert not fine.all() and want.isinf().any()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[want.isinf()], want[want.isinf()])
    assert bool(((got - want).abs() <= bound)[fine].all())


BITS = [(1, 4, 32, 128, 144, 3, 16), (30, 2, 4, 272, 144, 5, 8), (90, 3, 7, 128, 400, 60, 24), (200, 1, 6, 128, 1040, 9, 40),
        (150, 2, 3, 256, 128, 4, 64)]


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", BITS, ids=lambda c: "x".join(map(str, c)))
def test_hidden_values_keep_sixteen_bits(shape, f32):
    """Hidden values g u and g (u + 1), integers up to 255 256 < 2^16, meet down weights 1 and -1: their
    difference g is what is left.  Every product and sum is an integer below 2^24, so the results are exact up to y's
    rounding (two bf16 values hold any integer of 16 bits: eight of them, and a rest of at most 2^7)."""
    M, top_k, E, d, ff, n, r = shape
    log(f"moe_layer hidden bits {shape} f32={f32}")
    c = Layer(95, *shape, act="none", f32=f32, holes=0.0, residual=False)
    rng = np.random.default_rng(96)
    g = torch.Generator(device="cuda").manual_seed(97)
    x = np.zeros((M, d))
    x[np.arange(M), rng.integers(0, d, M)] = rng.choice([-1.0, 1.0], M)  # one element: g and u are W's
    c.x = torch.as_tensor(x, device="cuda").bfloat16()
    odd = torch.arange(ff, device="cuda") % 2

    def whole(lo, hi, *s):
        return torch.randint(lo, hi + 1, s, device="cuda", generator=g).double()

    def pairs(t):
        """The rows 2 i of t, and behind each its negative"""
        return t.repeat_interleave(2, -2) * (1.0 - 2.0 * odd)[:, None]

    c.W["g"] = whole(-255, 255, E, d, ff // 2).repeat_interleave(2, -1).bfloat16()
    c.W["u"] = (whole(0, 255, E, d, ff // 2).repeat_interleave(2, -1) + odd).bfloat16()
    some = torch.rand(E, ff // 2, d, device="cuda", generator=g) < 6.0 / ff
    c.W["d"] = pairs(some * (1.0 - 2.0 * whole(0, 1, E, ff // 2, d))).bfloat16()
    c.B["g"], c.B["u"] = torch.zeros_like(c.B["g"]), torch.zeros_like(c.B["u"])
    some = torch.rand(n, E, ff // 2, r, device="cuda", generator=g) < 4.0 / ff
    c.A["d"] = pairs(some * (1.0 - 2.0 * whole(0, 1, n, E, ff // 2, r))).bfloat16()
    c.B["d"] = whole(-1, 1, n, E, r, d).bfloat16()
    c.ranks, c.rank_of = None, np.full(n, r)
    c.scale = 1.0 - 2.0 * whole(0, 1, n).float()
    c.topk_w = 2.0 ** whole(-1, 1, M, top_k).float()
    y = torch.zeros(M, d, dtype=torch.float64, device="cuda")
    top = 0.0
    for e in range(E):
        m, j = (c.topk_ids == e).nonzero(as_tuple=True)
        if len(m) == 0:
            continue
        v = c.x[m].double()
        h = (v @ c.W["g"][e].double()) * (v @ c.W["u"][e].double())
        z, _ = c.project("d", e, h, torch.zeros_like(h), m)
        top = max(top, float((h.abs() @ c.W["d"][e].double().abs()).max()), float(h.abs().max()))
        y.index_add_(0, m, z * c.topk_w[m, j].double()[:, None])
    assert 255 < top < 2 ** 24 and 0 < y.abs().max() < 2 ** 23
    assert torch.equal(c.run(), y.to(c.type))
