"""lora_linear_act on the host: what its checks reject before anything is enqueued (CPU only)."""

import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

FAKE = 1 << 20  # aligned, never dereferenced


def _act(epi=None, **over):
    args = dict(x=FAKE, W=FAKE, A=FAKE, B=FAKE, scale=FAKE, ranks=None, ids=FAKE, M=64, d_in=4096,
                d_out=4096, r_max=16, n_adapters=32, segs=None, epi=epi, y=FAKE, y_dtype=L.LORA_BF16,
                mode=L.LORA_MODE_DECODE, ws=FAKE,
                ws_bytes=L.lora_workspace_bytes(64, 4096, 4096, 16, 32), stream=0)
    args.update(over)
    return L.lora_linear_act(**args)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), 2), (dict(d_in=12), 2), (dict(n_adapters=0), 2), (dict(r_max=65), 3),
    (dict(y_dtype=5), 6), (dict(mode=7), 9), (dict(x=None), 1), (dict(ids=None), 1), (dict(y=None), 1),
    (dict(W=FAKE + 8), 4), (dict(ws=FAKE + 16), 4), (dict(ws_bytes=1024), 5),
    (dict(epi=L.lora_epilogue(-1)), 11), (dict(epi=L.lora_epilogue(5)), 11),
    (dict(epi=L.lora_epilogue(bias=FAKE + 8)), 4), (dict(epi=L.lora_epilogue(mul=FAKE + 4)), 4),
    (dict(epi=L.lora_epilogue(residual=FAKE + 2)), 4),
    (dict(epi=L.lora_epilogue_t(FAKE + 2, None, None, 0)), 4),
])
def test_linear_act_rejects(over, code):
    with pytest.raises(L.LoraError) as e:
        _act(**over)
    assert e.value.status == code


def test_linear_act_empty_batch_is_noop():
    _act(M=0, x=None, y=None, ws=None)
    _act(L.lora_epilogue(L.LORA_ACT_SILU), M=0, x=None, y=None, ws=None)
    with pytest.raises(L.LoraError):
        _act(L.lora_epilogue(9), M=0, x=None, y=None, ws=None)


@pytest.mark.parametrize("name,bad", [
    ("bias", torch.zeros(4096)), ("mul", torch.zeros(64, 4096)), ("residual", torch.zeros(64, 4096)),
    ("mul", torch.zeros(63, 4096, dtype=torch.bfloat16)),
    ("residual", torch.zeros(4096, 64, dtype=torch.bfloat16).t()),
])
def test_binding_rejects_epilogue_tensors(name, bad):
    with pytest.raises(ValueError, match=name):
        _act(L.lora_epilogue(**{name: bad}))


@pytest.mark.parametrize("name,bad", [
    ("x", torch.zeros(64, 4096)), ("ids", torch.zeros(64, dtype=torch.int64)),
    ("scale", torch.zeros(32, dtype=torch.bfloat16)), ("y", torch.zeros(64, 4096)),
    ("ws", torch.zeros(10, dtype=torch.uint8)),
])
def test_binding_rejects_tensors(name, bad):
    with pytest.raises(ValueError, match=name):
        _act(**{name: bad})
