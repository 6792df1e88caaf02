"""The layer with its epilogue in 64 bits, and the bound its fp32 kernels stay within.

With S = |x| |W| + |scale| (|x| |A|) |B| element by element, the bound on z is
  * (k/8 + 64) 2^-24 S: MFMA chains over k = max(d_in, 64) products, the split sums and the
    expand's r_max products (each MFMA adds at least eight products per rounding);
  * 2^-16 |scale| (|x| |A|) |B|: the prefill epilogue carries scale t as two bf16 values, each
    off by half a step (2^-8) of what it holds.
The activations' slopes are at most 1.13 and their own error at most |z| 2^-20 (an exponent's
argument rounded at |z| of a few tens, exp2 and the reciprocal; Phi is off by 1.5e-7 / 2).  mul
multiplies both; y's rounding adds half a step: 2^-8 |y| in bf16, 2^-24 |y| in fp32 (and three
fp32 roundings of the terms before it).
"""

import math

import torch

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act64(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def layer64(x, W, A, B, scale, ranks, ids):
    """(z, bound of |z_gpu - z|) from float64 x[M, K], W[K, N] and the bf16 pool."""
    n, K, r = A.shape
    z, S = x @ W, x.abs() @ W.abs()
    D = torch.zeros_like(S)
    for i in sorted(set(ids.tolist())):
        if not 0 <= i < n:
            continue
        rows = (ids == i).nonzero()[:, 0]
        k = r if ranks is None else int(ranks[i])
        a, b, s = A[i, :, :k].double(), B[i, :k].double(), float(scale[i])
        z[rows] += s * ((x[rows] @ a) @ b)
        D[rows] += abs(s) * ((x[rows].abs() @ a.abs()) @ b.abs())
    c = (max(K, 64) / 8 + 64) * 2.0 ** -24
    return z, c * (S + D) + 2.0 ** -16 * D


def epilogue64(z, dz, act, bias, mul, residual, f32):
    """(y, bound) behind the epilogue."""
    if bias is not None:
        z = z + bias.double()
        dz = dz + 2.0 ** -24 * z.abs()
    y, dy = act64(z, act), 1.13 * dz
    if act != "none":
        dy = dy + 2.0 ** -20 * z.abs()
    if mul is not None:
        y, dy = y * mul.double(), dy * mul.double().abs() * 1.001
    if residual is not None:
        dy = dy + 2.0 ** -24 * y.abs()
        y = y + residual.double()
    step = 2.0 ** -24 if f32 else 2.0 ** -8
    return y, dy + (y.abs() + dy) * (step + 2 * 2.0 ** -24) + 1e-37


def assert_within(got, want, bound, what):
    assert torch.isfinite(got.float()).all(), f"{what}: non-finite"
    off = (got.double() - want).abs()
    bad = off > bound
    if bad.any():
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} elements off, first at {at}: "
                             f"{float(got[at])} for {float(want[at])}, bound {float(bound[at]):.3e}")
