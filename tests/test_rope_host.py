"""lora_rope and lora_rope_freqs on the host: what their checks reject, and the tables against their
formulas in 64 bits (CPU only)."""

import math

import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

FAKE = 1 << 20  # aligned, never dereferenced


def _rope(**over):
    args = dict(q=FAKE, k=FAKE, positions=FAKE, freqs=FAKE, M=4, q_heads=8, k_heads=2, head_dim=64, rot_dim=64,
                q_stride=512, k_stride=128, layout=L.LORA_ROPE_HALF, factor=1.0, inverse=0, q_out=2 * FAKE,
                q_out_stride=512, k_out=2 * FAKE, k_out_stride=128, dtype=L.LORA_BF16, stream=0)
    args.update(over)
    return L.lora_rope(**args)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), 2), (dict(M=L.LORA_MAX_ROWS + 1), 2), (dict(q_heads=0), 2), (dict(k_heads=-1), 2),
    (dict(q_heads=1025, q_stride=1 << 20, q_out_stride=1 << 20), 2),
    (dict(k_heads=1025, k_stride=1 << 20, k_out_stride=1 << 20), 2), (dict(head_dim=0), 2),
    (dict(head_dim=12, rot_dim=12), 2), (dict(head_dim=1032, q_stride=1 << 16, k_stride=1 << 16), 2),
    (dict(rot_dim=0), 2), (dict(rot_dim=7), 2), (dict(rot_dim=66), 2), (dict(q_stride=504), 2),
    (dict(q_stride=516), 2), (dict(k_stride=120), 2), (dict(q_out_stride=511), 2), (dict(k_out_stride=64), 2),
    (dict(q_stride=(1 << 28) + 8), 2), (dict(q_stride=-512), 2), (dict(q_out=FAKE, q_out_stride=520), 2),
    (dict(dtype=2), 6), (dict(layout=2), 9), (dict(layout=-1), 9), (dict(factor=0.0), 11),
    (dict(factor=float("nan")), 11), (dict(factor=float("inf")), 11), (dict(factor=-1.0), 11),
    (dict(inverse=2), 11), (dict(inverse=-1), 11), (dict(q=None), 1), (dict(q_out=None), 1), (dict(k=None), 1),
    (dict(k_out=None), 1), (dict(positions=None), 1), (dict(freqs=None), 1), (dict(q=FAKE + 8), 4),
    (dict(k=FAKE + 2), 4), (dict(q_out=FAKE + 8), 4), (dict(k_out=FAKE + 8), 4), (dict(positions=FAKE + 2), 4),
    (dict(freqs=FAKE + 4), 4),
])
def test_rope_rejects(over, code):
    with pytest.raises(L.LoraError) as e:
        _rope(**over)
    assert e.value.status == code


E = 2  # bytes of bf16


@pytest.mark.parametrize("over", [
    dict(),  # (k_out lies on q_out)
    dict(k_out=FAKE), dict(k_out=3 * FAKE, q_out=FAKE + 16), dict(q=FAKE, k=4 * FAKE, k_out=FAKE + 512 * E),
    dict(k_out=2 * FAKE + 3 * 512 * E + 16), dict(M=1, k_out=2 * FAKE + 1008),
    # a row of q, k and v: k_out reaches into q's part, q_out into the next row's
    dict(q_stride=768, k_stride=768, q_out_stride=768, k_out_stride=768, k=FAKE + 512 * E, q_out=FAKE,
         k_out=FAKE + 504 * E),
    dict(q_stride=768, k_stride=768, q_out_stride=768, k_out_stride=768, q=3 * FAKE + 512 * E, k=5 * FAKE,
         q_out=2 * FAKE + 272 * E, k_out=2 * FAKE + 768 * 4 * E - 32),
    dict(q_stride=640, q_out_stride=640, q=FAKE, q_out=FAKE + 640 * E, k_out=9 * FAKE, k=8 * FAKE),
])
def test_rope_rejects_outputs_over_each_other(over):
    with pytest.raises(L.LoraError) as e:
        _rope(**over)
    assert e.value.status == 2


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses of no memory must not reach a GPU")
@pytest.mark.parametrize("seed", range(4))
def test_rope_takes_rows_beside_each_other(seed):
    """Outputs given over rows against a plain count of bytes: what is refused overlaps, and every overlap that
    equal or gapless strides show is refused.  (A call that passes would launch; without a GPU it ends in
    another error.)"""
    import random

    rnd = random.Random(seed)
    seen = [0, 0]
    for _ in range(400):
        M, qw, kw = rnd.choice([1, 2, 5]), 16 * rnd.randint(1, 3), 16
        dense = rnd.random() < 0.5
        sq = qw if dense else qw + 16 * rnd.randint(0, 4)
        sk = sq if not dense and sq >= kw else kw + 8 * rnd.randint(0, 6)
        qo, ko = FAKE, FAKE + 16 * rnd.randint(-30, 60)
        a = {qo + 2 * (m * sq + j) for m in range(M) for j in range(qw)}
        b = {ko + 2 * (m * sk + j) for m in range(M) for j in range(kw)}
        hit = bool(a & b)
        seen[hit] += 1
        with pytest.raises(L.LoraError) as e:
            _rope(M=M, q_heads=qw // 16, k_heads=1, head_dim=16, rot_dim=16, q=FAKE << 8, k=FAKE << 9,
                  q_stride=sq, k_stride=sk, q_out=qo, q_out_stride=sq, k_out=ko, k_out_stride=sk)
        assert (e.value.status == 2) == hit, (M, qw, sq, sk, ko - qo)
    assert min(seen) > 40


def test_rope_empty_batch_is_noop():
    _rope(M=0, q=None, k=None, q_out=None, k_out=None, positions=None, freqs=None)
    _rope(M=0, k_heads=0, k=None, k_out=None, k_stride=0, k_out_stride=0)


BF = torch.bfloat16


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros(4, 512)), ("q", torch.zeros(3, 512, dtype=BF)), ("q", torch.zeros(4, 504, dtype=BF)),
    ("q", torch.zeros(512, 4, dtype=BF).t()), ("q", torch.zeros(4, 520, dtype=BF)[:, :512]),
    ("q", torch.zeros(4, 64, 8, dtype=BF).transpose(1, 2)), ("q", torch.zeros(2048, dtype=BF)),
    ("q", torch.zeros(4, 512, dtype=BF)),  # (on the CPU)
    ("k", torch.zeros(4, 128)), ("q_out", torch.zeros(4, 512)), ("k_out", torch.zeros(4, 64, dtype=BF)),
    ("positions", torch.zeros(4, dtype=torch.int64)), ("positions", torch.zeros(3, dtype=torch.int32)),
    ("freqs", torch.zeros(32)), ("freqs", torch.zeros(31, dtype=torch.float64)),
])
def test_binding_rejects_tensors(name, bad):
    with pytest.raises(ValueError, match=name):
        _rope(**{name: bad})


class _Stream:
    def __init__(self, device_index):
        self.device_index, self.cuda_stream = device_index, 0


def test_binding_rejects_a_stream_of_another_device(monkeypatch):
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    _rope(M=0, stream=_Stream(0))
    with pytest.raises(ValueError, match="stream"):
        _rope(M=0, stream=_Stream(1))


@pytest.mark.parametrize("rot", [2, 4, 52, 64, 128, 1024])
def test_tables(rot):
    plain = [10000.0 ** (-2 * i / rot) / (2 * math.pi) for i in range(rot // 2)]

    def close(got, want):
        f, factor = got
        assert f.dtype == torch.float64 and f.shape == (rot // 2,)
        # pow within an ulp or two, four more roundings
        assert (f - torch.tensor(want, dtype=torch.float64)).abs().max() <= 8 * 2.0 ** -53 * max(want)
        for a, b in zip(f.tolist(), want):
            assert abs(a - b) <= 16 * 2.0 ** -53 * abs(b)
        return factor

    assert close(L.lora_rope_freqs(rot, device="cpu"), plain) == 1.0
    assert close(L.lora_rope_freqs(rot, 10000.0, L.LORA_ROPE_LINEAR, 4.0, device="cpu"), [f / 4 for f in plain]) == 1.0
    ntk = 5e5 * 8.0 ** (rot / (rot - 2) if rot > 2 else 2.0)
    want = [ntk ** (-2 * i / rot) / (2 * math.pi) for i in range(rot // 2)]
    assert close(L.lora_rope_freqs(rot, 5e5, L.LORA_ROPE_NTK, 8.0, device="cpu"), want) == 1.0
    yarn = []
    for f in plain:
        g = min(max((4096.0 * f - 1.0) / 31.0, 0.0), 1.0)
        yarn.append(f / 8.0 * (1.0 - g) + f * g)
    factor = close(L.lora_rope_freqs(rot, 10000.0, L.LORA_ROPE_YARN, 8.0, 4096.0, device="cpu"), yarn)
    assert abs(factor - (0.1 * math.log(8.0) + 1.0)) <= 2.0 ** -23
    # the slowest pair of a long head is interpolated, the fastest keeps its pace
    if rot >= 64:
        assert yarn[0] == plain[0] and abs(yarn[-1] * 8 / plain[-1] - 1) < 1e-12


@pytest.mark.parametrize("args,code", [
    ((0,), 2), ((3,), 2), ((1026,), 2), ((64, 1.0), 11), ((64, float("nan")), 11), ((64, float("inf")), 11),
    ((64, 1e4, 4), 9), ((64, 1e4, -1), 9), ((64, 1e4, 1, 0.5), 11), ((64, 1e4, 2, float("inf")), 11),
    ((64, 1e4, 3, 8.0, 0.0), 11), ((64, 1e4, 3, 8.0, float("nan")), 11),
])
def test_tables_reject(args, code):
    with pytest.raises(L.LoraError) as e:
        L.lora_rope_freqs(*args, device="cpu")
    assert e.value.status == code
