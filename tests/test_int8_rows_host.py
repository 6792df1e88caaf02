"""lora_rmsnorm_int8 and lora_quant_int8 on the host: what their checks reject before anything is
enqueued (CPU only)."""

import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

FAKE = 1 << 20  # aligned, never dereferenced


def _norm(**over):
    args = dict(x=FAKE, residual=FAKE, weight=FAKE, eps=1e-5, M=4, d=64, sum=FAKE, y=FAKE, y8=FAKE,
                y_scale=FAKE, stream=0)
    args.update(over)
    return L.lora_rmsnorm_int8(**args)


def _quant(**over):
    args = dict(x=FAKE, M=4, d=64, y8=FAKE, y_scale=FAKE, stream=0)
    args.update(over)
    return L.lora_quant_int8(**args)


BOTH = [
    (dict(M=-1), 2), (dict(M=L.LORA_MAX_ROWS + 1), 2), (dict(d=0), 2), (dict(d=-8), 2), (dict(d=12), 2),
    (dict(d=(1 << 20) + 8), 2), (dict(x=None), 1), (dict(y8=None), 1), (dict(y_scale=None), 1),
    (dict(y8=None, y_scale=None), 1), (dict(x=FAKE + 8), 4), (dict(y8=FAKE + 8), 4),
    (dict(y_scale=FAKE + 2), 4),
]


@pytest.mark.parametrize("over,code", BOTH + [
    (dict(eps=0.0), 11), (dict(eps=float("nan")), 11), (dict(eps=float("inf")), 11),
    (dict(eps=1e-31), 11), (dict(residual=FAKE + 2), 4), (dict(weight=FAKE + 4), 4),
    (dict(sum=FAKE + 8), 4), (dict(y=FAKE + 8), 4),
])
def test_rmsnorm_int8_rejects(over, code):
    with pytest.raises(L.LoraError) as e:
        _norm(**over)
    assert e.value.status == code


@pytest.mark.parametrize("over,code", BOTH)
def test_quant_int8_rejects(over, code):
    with pytest.raises(L.LoraError) as e:
        _quant(**over)
    assert e.value.status == code


def test_empty_batch_is_noop():
    _norm(M=0, x=None, y=None, y8=None, y_scale=None)
    _quant(M=0, x=None, y8=None, y_scale=None)


@pytest.mark.parametrize("bad", [
    dict(x=torch.zeros(4, 64)),                                   # float32
    dict(x=torch.zeros(64, 4, dtype=torch.bfloat16).t()),         # not contiguous
    dict(x=torch.zeros(3, 64, dtype=torch.bfloat16)),             # too small
    dict(x=torch.zeros(4, 64, dtype=torch.bfloat16)),             # on the CPU
    dict(y8=torch.zeros(4, 64, dtype=torch.uint8)),               # E4M3 codes' type
    dict(y8=torch.zeros(4, 64, dtype=torch.float8_e4m3fn)),
    dict(y_scale=torch.zeros(4, dtype=torch.bfloat16)),
], ids=lambda b: next(iter(b)))
def test_binding_rejects_tensors(bad):
    for call in (_norm, _quant):
        with pytest.raises(ValueError, match=next(iter(bad))):
            call(**bad)


class _Stream:
    """What the binding reads of a torch stream."""

    def __init__(self, device_index):
        self.device_index, self.cuda_stream = device_index, 0


def test_binding_rejects_a_stream_of_another_device(monkeypatch):
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    for call in (_norm, _quant):
        call(M=0, stream=_Stream(0))
        with pytest.raises(ValueError, match="stream"):
            call(M=0, stream=_Stream(1))
