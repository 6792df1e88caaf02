"""lora_linear_fp8 on the host: what its checks reject before anything is enqueued (CPU only)."""

import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

FAKE = 1 << 20  # aligned, never dereferenced


def _fp8(epi=None, **over):
    args = dict(x8=FAKE, x_scale=FAKE, W8=FAKE, w_scale=FAKE, A=FAKE, B=FAKE, scale=FAKE, ranks=None,
                ids=FAKE, M=64, d_in=4096, d_out=4096, r_max=16, n_adapters=32, segs=None, epi=epi,
                y=FAKE, y_dtype=L.LORA_BF16, mode=L.LORA_MODE_AUTO, ws=FAKE,
                ws_bytes=L.lora_fp8_workspace_bytes(64, 4096, 4096, 16, 32), stream=0)
    args.update(over)
    return L.lora_linear_fp8(**args)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), 2), (dict(M=L.LORA_MAX_ROWS + 1), 2), (dict(d_in=4104), 2), (dict(d_in=0), 2),
    (dict(d_out=4100), 2), (dict(n_adapters=0), 2), (dict(r_max=0), 3), (dict(r_max=65), 3),
    (dict(y_dtype=5), 6), (dict(mode=L.LORA_MODE_DECODE), 9), (dict(mode=L.LORA_MODE_PREFILL), 9),
    (dict(mode=0x200), 9), (dict(x8=None), 1), (dict(x_scale=None), 1), (dict(W8=None), 1),
    (dict(w_scale=None), 1), (dict(ids=None), 1), (dict(scale=None), 1), (dict(y=None), 1),
    (dict(ws=None), 1), (dict(x8=FAKE + 8), 4), (dict(W8=FAKE + 8), 4), (dict(x_scale=FAKE + 2), 4),
    (dict(w_scale=FAKE + 2), 4), (dict(y=FAKE + 8), 4), (dict(ws=FAKE + 16), 4), (dict(ws_bytes=1024), 5),
    (dict(epi=L.lora_epilogue(7)), 11), (dict(epi=L.lora_epilogue(mul=FAKE + 8)), 4),
])
def test_linear_fp8_rejects(over, code):
    with pytest.raises(L.LoraError) as e:
        _fp8(**over)
    assert e.value.status == code


def test_linear_fp8_empty_batch_is_noop():
    _fp8(M=0, x8=None, y=None, ws=None)


def test_workspace_bytes():
    assert L.lora_fp8_workspace_bytes(0, 4096, 4096, 16, 32) == 0
    assert L.lora_fp8_workspace_bytes(64, 4104, 4096, 16, 32) == 0
    assert L.lora_fp8_workspace_bytes(64, 4096, 4096, 65, 32) == 0
    b = L.lora_fp8_workspace_bytes(64, 4096, 4096, 16, 32)
    assert b > 0 and b % 256 == 0
    assert L.lora_fp8_workspace_bytes(64, 4096, 4096, 64, 32) > b


@pytest.mark.parametrize("name,bad", [
    ("x8", torch.zeros(64, 4096, dtype=torch.bfloat16)), ("x_scale", torch.zeros(63)),
    ("W8", torch.zeros(4096, 4096, dtype=torch.int8)), ("w_scale", torch.zeros(4096, dtype=torch.float64)),
    ("y", torch.zeros(64, 4096)),
])
def test_binding_rejects_tensors(name, bad):
    with pytest.raises(ValueError, match=name):
        _fp8(**{name: bad})
