"""lora_moe_layer on values at the ends: infinities in the down projection."""

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
