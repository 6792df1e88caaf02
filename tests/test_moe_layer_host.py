"""lora_moe_layer on the host: what its checks reject before anything is enqueued (CPU only)."""

import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

FAKE = 1 << 20  # aligned, never dereferenced
SIZES = (16, 4, 8, 256, 400, 16, 5)  # M, top_k, experts, d, d_ff, r_max, adapters


def _weights(**over):
    w = {m + p: FAKE for p in "gud" for m in "WAB"}
    w.update(over)
    return L.lora_moe_weights(*(w[m + p] for p in "gud" for m in "WAB"))


def _layer(weights="own", **over):
    args = dict(x=FAKE, weights=_weights() if weights == "own" else weights, scale=FAKE, ranks=FAKE, ids=FAKE,
                topk_ids=FAKE, topk_w=FAKE, residual=FAKE, M=16, top_k=4, n_experts=8, d=256, d_ff=400, r_max=16,
                n_adapters=5, act=L.LORA_ACT_SILU, y=FAKE, y_dtype=L.LORA_BF16, mode=L.LORA_MODE_AUTO, ws=FAKE,
                ws_bytes=L.lora_moe_layer_workspace_bytes(*SIZES), stream=0)
    args.update(over)
    return L.lora_moe_layer(**args)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), 2), (dict(M=2049), 2), (dict(top_k=0), 2), (dict(top_k=65), 2), (dict(n_experts=0), 2),
    (dict(n_experts=4097), 2), (dict(d=120), 2), (dict(d=264), 2), (dict(d=0), 2), (dict(d_ff=112), 2),
    (dict(d_ff=408), 2), (dict(d=(1 << 20) + 16), 2), (dict(n_adapters=0), 2),
    (dict(n_adapters=L.LORA_MAX_ADAPTERS + 1), 2), (dict(r_max=0), 3), (dict(r_max=4), 3), (dict(r_max=12), 3),
    (dict(r_max=72), 3), (dict(act=5), 11), (dict(act=-1), 11), (dict(y_dtype=3), 6),
    (dict(mode=L.LORA_MODE_PREFILL), 9), (dict(mode=7), 9), (dict(x=None), 1), (dict(weights=None), 1),
    (dict(scale=None), 1), (dict(ids=None), 1), (dict(topk_ids=None), 1), (dict(y=None), 1), (dict(ws=None), 1),
    (dict(x=FAKE + 8), 4), (dict(y=FAKE + 8), 4), (dict(residual=FAKE + 8), 4), (dict(ws=FAKE + 16), 4),
    (dict(scale=FAKE + 2), 4), (dict(ids=FAKE + 2), 4), (dict(topk_ids=FAKE + 1), 4), (dict(topk_w=FAKE + 2), 4),
    (dict(ranks=FAKE + 2), 4), (dict(ws_bytes=1024), 5),
] + [(dict(weights=_weights(**{m + p: None})), 1) for p in "gud" for m in "WAB"]
  + [(dict(weights=_weights(**{m + p: FAKE + 8})), 4) for p in "gud" for m in "WAB"])
def test_moe_layer_rejects(over, code):
    with pytest.raises(L.LoraError) as e:
        _layer(**over)
    assert e.value.status == code


def test_empty_batch_is_noop():
    _layer(M=0, x=None, y=None, ws=None, topk_ids=None)
    _layer(weights=None, M=0)


def test_workspace_bytes():
    b = L.lora_moe_layer_workspace_bytes(*SIZES)
    assert b > 0 and b % 256 == 0 and L.moe_layer_workspace(*SIZES, device="cpu")[1] == b
    assert L.lora_moe_layer_workspace_bytes(0, *SIZES[1:]) == 0
    assert L.lora_moe_layer_workspace_bytes(16, 4, 8, 264, 400, 16, 5) == 0
    assert L.lora_moe_layer_workspace_bytes(2049, 4, 8, 256, 400, 16, 5) == 0
    assert L.lora_moe_layer_workspace_bytes(2048, 4, 8, 256, 400, 16, 5) > b
    # the largest batch at large sizes: more than 32 bits
    assert L.lora_moe_layer_workspace_bytes(128, 64, 64, 1 << 20, 1 << 20, 64, 16384) > 1 << 34


@pytest.mark.parametrize("name,bad", [
    ("x", torch.zeros(16, 256)), ("topk_ids", torch.zeros(16, 4, dtype=torch.int64)),
    ("topk_w", torch.zeros(16, 4, dtype=torch.bfloat16)), ("residual", torch.zeros(16, 256)),
    ("ids", torch.zeros(15, dtype=torch.int32)), ("y", torch.zeros(16, 256)), ("scale", torch.zeros(4)),
    ("ws", torch.zeros(10, dtype=torch.uint8)),
])
def test_binding_rejects_tensors(name, bad):
    with pytest.raises(ValueError, match=name):
        _layer(**{name: bad})


@pytest.mark.parametrize("at,name,shape", [
    ("Wg", "gate.W", (8, 256, 392)), ("Au", "up.A", (5, 8, 256, 8)), ("Bd", "down.B", (5, 8, 16, 248)),
])
def test_binding_rejects_weights(at, name, shape):
    for bad in (torch.zeros(shape, dtype=torch.bfloat16), torch.zeros(1 << 20)):
        with pytest.raises(ValueError, match=name):
            _layer(weights=_weights(**{at: bad}))


class _Stream:
    def __init__(self, device_index):
        self.device_index, self.cuda_stream = device_index, 0


def test_binding_rejects_a_stream_of_another_device(monkeypatch):
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    _layer(M=0, stream=_Stream(0))
    with pytest.raises(ValueError, match="stream"):
        _layer(M=0, stream=_Stream(1))
