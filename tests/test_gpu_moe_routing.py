"""How a workgroup of the expert-routed GEMM finds its expert, pairs and adapters: numbers of experts and adapters at
the ends of their range, batches on both sides of 64 pairs, fewer pairs than experts and more.  Every input is a small
integer, so that every sum is exact and the results have to be equal to 64-bit ones."""

import numpy as np
import pytest
import torch

from rank_adapter_gemm_sgmv_amd import lora as L

from .gpu_util import log

pytestmark = pytest.mark.gpu

# M, top_k, E, K, N, n, r
SHAPES = [
    (1, 1, 4096, 128, 128, 1, 8), (1, 4, 16, 512, 512, 3, 8), (2, 4, 33, 256, 136, 2, 16), (8, 8, 100, 128, 264, 8, 8),
    (13, 5, 66, 128, 128, 13, 24), (63, 1, 65, 128, 136, 500, 8), (64, 1, 4096, 128, 128, 2, 8),
    (16, 4, 65, 640, 640, 16, 8), (65, 1, 66, 128, 136, 9, 64), (66, 1, 2048, 128, 128, 3, 8),
    (64, 1, 1, 128, 136, 16384, 8), (200, 1, 1, 128, 128, 16384, 8), (48, 2, 2, 160, 128, 4097, 8), (90, 3, 7, 128, 400, 60, 24),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "x".join(map(str, c)))
def test_pairs_find_their_experts_and_adapters(shape):
    M, k, E, K, N, n, r = shape
    log(f"moe routing {shape}")
    rng = np.random.default_rng(SHAPES.index(shape))
    g = torch.Generator(device="cuda").manual_seed(SHAPES.index(shape))

    def signs(*s):
        return torch.randint(-1, 2, s, device="cuda", generator=g, dtype=torch.int8).bfloat16()

    def ends(limit, size):
        """Numbers below `limit`: its ends, next to powers of two, any."""
        edge = [v for b in range(15) for v in (2 ** b - 1, 2 ** b) if v < limit] + [limit - 1]
        return np.where(rng.random(size) < 0.5, rng.choice(edge, size), rng.integers(0, limit, size))

    topk, ids = ends(E, (M, k)), ends(n, M)
    topk[rng.random((M, k)) < 0.1] = -1
    topk[M // 2, 0], topk[-1, -1], ids[M // 3] = 0, E - 1, n - 1
    if M > 3:
        topk[1, 0], topk[2, 0], ids[1], ids[2] = E, -2 ** 31, -1, n
    topk_ids = torch.as_tensor(topk, dtype=torch.int32, device="cuda")
    ids = torch.as_tensor(ids, dtype=torch.int32, device="cuda")
    x, W, A, B = signs(M, K), signs(E, K, N), signs(n, E, K, r), signs(n, E, r, N)
    scale = 1.0 - 2.0 * torch.randint(0, 2, (n,), device="cuda", generator=g).float()
    y = torch.full((M, k, N), 7.0, device="cuda")
    nbytes = L.lora_moe_workspace_bytes(M, k, E, K, N, r, n)
    ws = torch.full((max(nbytes, 256),), 255, dtype=torch.uint8, device="cuda")
    L.lora_moe_linear(x, W, A, B, scale, None, ids, topk_ids, None, M, k, E, K, N, r, n, y, L.LORA_F32,
                      L.LORA_MODE_AUTO, ws, nbytes)
    torch.cuda.synchronize()
    want = torch.zeros(M, k, N, dtype=torch.float64, device="cuda")
    for m in range(M):
        i = int(ids[m])
        for j in range(k):
            e = int(topk_ids[m, j])
            if not 0 <= e < E:
                continue
            v = x[m].double()
            want[m, j] = v @ W[e].double()
            if 0 <= i < n:
                want[m, j] += scale[i].double() * ((v @ A[i, e].double()) @ B[i, e].double())
    assert 0 < want.abs().max() < 2 ** 24
    assert torch.equal(y.double(), want)
