"""lora_rope against its formula in 64 bits.

Tolerances.  The turns and their fraction are 64-bit here and there.  The kernel's cosines and sines:
the angle (at most pi / 4) is rounded twice, 2 * 0.79 * 2^-24; their polynomials are within 2e-9 and a
few roundings of values up to 1; the factor is one more: 6 * 2^-24 of the factor together.  Each output
is a fused product and sum, 2 more roundings of |a| + |b|: |error| <= 8 * 2^-24 factor (|a| + |b|), and
the output's rounding: 2^-8 of itself in bf16, 2^-24 in fp32.  What passes through is equal.
"""

import math

import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

from .gpu_util import log

pytestmark = pytest.mark.gpu

T = {L.LORA_BF16: torch.bfloat16, L.LORA_F32: torch.float32}


def reference(x, positions, freqs, rot, layout, factor, inverse):
    """(y, bound) of x[M, heads, D]"""
    x = x.double()
    t = positions.double()[:, None] * freqs
    t = 2 * math.pi * (t - torch.floor(t))
    c, s = torch.cos(t)[:, None] * factor, torch.sin(t)[:, None] * (-factor if inverse else factor)
    y, size = x.clone(), torch.zeros_like(x)
    i = torch.arange(rot // 2, device=x.device)
    ia, ib = (i, i + rot // 2) if layout == L.LORA_ROPE_HALF else (2 * i, 2 * i + 1)
    a, b = x[:, :, ia], x[:, :, ib]
    y[:, :, ia], y[:, :, ib] = a * c - b * s, a * s + b * c
    size[:, :, ia] = size[:, :, ib] = factor * (a.abs() + b.abs())
    return y, 8 * 2.0 ** -24 * size


def check(got, x, positions, freqs, rot, layout, factor, inverse):
    want, bound = reference(x, positions, freqs, rot, layout, factor, inverse)
    step = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    off = (got.double() - want).abs()
    assert (off <= bound + (want.abs() + bound) * step + 1e-40).all(), float((off - bound).max())
    assert torch.equal(got[:, :, rot:], x[:, :, rot:])


def make(seed, M, hq, hk, D, dtype, pad=8):
    """q and k as slices of rows of q, k and something else"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    row = (hq + hk) * D + pad
    qk = torch.empty(M, row, device="cuda").normal_(0, 1, generator=g).to(T[dtype])
    return qk, qk[:, :hq * D], qk[:, hq * D:(hq + hk) * D], row


# M, q heads, k heads, head_dim, rot_dim
SHAPES = [(1, 1, 0, 8, 8), (1, 32, 8, 128, 128), (3, 2, 1, 64, 32), (7, 5, 5, 104, 52), (33, 12, 3, 96, 96),
          (5, 3, 1, 80, 2), (2, 1, 1, 256, 254), (17, 9, 0, 72, 24), (4, 2, 2, 1024, 1024), (257, 16, 2, 128, 64),
          (2, 1024, 1, 8, 6), (65, 71, 1, 64, 64), (1021, 6, 1, 40, 40)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("layout", [L.LORA_ROPE_HALF, L.LORA_ROPE_INTERLEAVED], ids=["half", "inter"])
@pytest.mark.parametrize("dtype", [L.LORA_BF16, L.LORA_F32], ids=["bf16", "f32"])
def test_rope(shape, layout, dtype):
    M, hq, hk, D, rot = shape
    log(f"rope {shape} {layout} {dtype}")
    for inverse, in_place in ((0, False), (1, True)):
        qk, q, k, row = make(sum(shape), M, hq, hk, D, dtype)
        before = qk.clone()
        freqs, factor = L.lora_rope_freqs(rot, 10000.0, L.LORA_ROPE_YARN, 4.0, 256.0)
        pos = torch.randint(-50, 100000, (M,), device="cuda", dtype=torch.int32)
        if in_place:
            qo, ko, so, sk = q, k, row, row
        else:
            big = torch.full((M, hq * D + 16), 7.0, device="cuda", dtype=T[dtype])
            qo, ko, so, sk = big[:, :hq * D], torch.full((M, max(hk, 1) * D), 7.0, device="cuda", dtype=T[dtype]), hq * D + 16, max(hk, 1) * D
        L.lora_rope(q, k if hk else None, pos, freqs, M, hq, hk, D, rot, row, row, layout, factor, inverse, qo, so,
                    ko if hk else None, sk, dtype)
        torch.cuda.synchronize()
        x = before[:, :(hq + hk) * D].reshape(M, hq + hk, D)
        check(qo.reshape(M, hq, D), x[:, :hq], pos, freqs, rot, layout, factor, inverse)
        if hk:
            check(ko.reshape(M, hk, D), x[:, hq:], pos, freqs, rot, layout, factor, inverse)
        if in_place:
            assert torch.equal(qk[:, (hq + hk) * D:], before[:, (hq + hk) * D:])
        else:
            assert torch.equal(qk, before) and (big[:, hq * D:] == 7.0).all()


@pytest.mark.parametrize("layout", [L.LORA_ROPE_HALF, L.LORA_ROPE_INTERLEAVED])
def test_positions_at_the_ends(layout):
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 999999, 131072], dtype=torch.int32, device="cuda")
    M = len(pos)
    qk, q, k, row = make(5, M, 2, 1, 64, L.LORA_F32)
    freqs, factor = L.lora_rope_freqs(64)
    qo, ko = torch.empty(M, 128, device="cuda"), torch.empty(M, 64, device="cuda")
    L.lora_rope(q, k, pos, freqs, M, 2, 1, 64, 64, row, row, layout, factor, 0, qo, 128, ko, 64, L.LORA_F32)
    torch.cuda.synchronize()
    check(qo.view(M, 2, 64), q.reshape(M, 2, 64), pos, freqs, 64, layout, factor, 0)
    assert torch.equal(qo[0], q[0])  # position 0 turns nothing


def test_there_and_back_is_the_gradient():
    """inverse is the transpose: <R x, g> = <x, R^T g>, and differences along a direction."""
    M, D, rot = 19, 96, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x, gy, v = (torch.empty(M, 3 * D, device="cuda").normal_(0, 1, generator=g) for _ in range(3))
    freqs, factor = L.lora_rope_freqs(rot, 10000.0, L.LORA_ROPE_YARN, 8.0, 64.0)
    pos = torch.arange(M, device="cuda", dtype=torch.int32) * 77

    def f(t, inverse):
        y = torch.empty_like(t)
        L.lora_rope(t, None, pos, freqs, M, 3, 0, D, rot, 3 * D, 0, L.LORA_ROPE_INTERLEAVED, factor, inverse, y, 3 * D,
                    None, 0, L.LORA_F32)
        return y.double()

    gx = f(gy, 1)
    size = factor * float((x.abs().double() * gy.abs().double()).sum()) * 2
    assert abs(float((f(x, 0) * gy.double()).sum() - (x.double() * gx).sum())) <= 20 * 2.0 ** -24 * size
    h = 2.0 ** -4
    slope = ((f(x + h * v, 0) - f(x - h * v, 0)) * gy.double()).sum() / (2 * h)
    size = factor * float(((x.abs() + v.abs()).double() * gy.abs().double()).sum()) * 4 / h
    assert abs(float(slope - (v.double() * gx).sum())) <= 20 * 2.0 ** -24 * size


def test_nan_and_infinity_stay_in_their_pair():
    M, D = 4, 64
    for value in (float("nan"), float("inf")):
        qk, q, k, row = make(6, M, 2, 0, D, L.LORA_BF16)
        ref = torch.empty(M, 2 * D, dtype=torch.bfloat16, device="cuda")
        got = torch.empty_like(ref)
        freqs, _ = L.lora_rope_freqs(D)
        pos = torch.arange(M, device="cuda", dtype=torch.int32)
        args = (None, pos, freqs, M, 2, 0, D, D, row, 0, L.LORA_ROPE_HALF, 1.0, 0)
        L.lora_rope(q, *args, ref, 2 * D, None, 0, L.LORA_BF16)
        qk[2, 5] = value
        L.lora_rope(q, *args, got, 2 * D, None, 0, L.LORA_BF16)
        torch.cuda.synchronize()
        hit = torch.zeros(M, 2 * D, dtype=torch.bool, device="cuda")
        hit[2, 5] = hit[2, 5 + D // 2] = True
        assert torch.equal(got[~hit], ref[~hit]) and not torch.isfinite(got[hit].float()).any()


def test_rows_behind_the_last_are_left_and_streams_and_graph():
    M, hq, hk, D = 45, 8, 2, 128
    qk, q, k, row = make(8, M, hq, hk, D, L.LORA_BF16)
    freqs, factor = L.lora_rope_freqs(D)
    pos = torch.arange(M, device="cuda", dtype=torch.int32) + 4000
    qo = torch.full((M, hq * D), 7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((M, hk * D), 7.0, dtype=torch.bfloat16, device="cuda")

    def call(m):
        L.lora_rope(q, k, pos, freqs, m, hq, hk, D, D, row, row, L.LORA_ROPE_HALF, factor, 0, qo, hq * D, ko, hk * D,
                    L.LORA_BF16)

    call(40)
    torch.cuda.synchronize()
    assert (qo[40:] == 7.0).all() and (ko[40:] == 7.0).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(M)
    torch.cuda.synchronize()
    check(qo.view(M, hq, D), q.reshape(M, hq, D), pos, freqs, D, L.LORA_ROPE_HALF, factor, 0)
    want_q, want_k = qo.clone(), ko.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(M)
    for _ in range(3):
        qo.zero_(), ko.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want_q) and torch.equal(ko, want_k)
        torch.ones(1000, device="cuda").sum()


def test_rows_past_2_31_elements():
    M, hq, D = 70000, 256, 128  # 2.3e9 elements
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough memory")
    log("rope past 2^31 elements")
    q = torch.empty(M, hq * D, dtype=torch.bfloat16, device="cuda").normal_()
    rows = torch.tensor([0, 1, M // 2, (1 << 31) // (hq * D), (1 << 31) // (hq * D) + 1, M - 1], device="cuda")
    before = q[rows]
    freqs, _ = L.lora_rope_freqs(D)
    pos = torch.arange(M, device="cuda", dtype=torch.int32)
    L.lora_rope(q, None, pos, freqs, M, hq, 0, D, D, hq * D, 0, L.LORA_ROPE_INTERLEAVED, 1.0, 0, q, hq * D, None, 0,
                L.LORA_BF16)
    torch.cuda.synchronize()
    check(q[rows].view(-1, hq, D), before.view(-1, hq, D), pos[rows], freqs, D, L.LORA_ROPE_INTERLEAVED, 1.0, 0)
