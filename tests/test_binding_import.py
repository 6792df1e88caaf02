"""The binding on a torch without its private GPU names, as one built without GPU support: host-only
calls and refusals work (CPU only)."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from rank_adapter_gemm_sgmv_amd import lora as L

assert L.lora_max_tiles(100, 8) == 8 + 100 // L.LORA_TILE_ROWS
assert L.lora_workspace_bytes(64, 4096, 4096, 16, 32) > 0
try:
    L.lora_rmsnorm(torch.zeros(4, 64, dtype=torch.bfloat16), None, None, 1e-5, 4, 64, None, None, None, None,
                   stream=0)
except ValueError as e:
    assert "x" in str(e)
else:
    raise SystemExit("a CPU tensor was taken")
print("done")
"""


def test_import_without_private_names():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]
