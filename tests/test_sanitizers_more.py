"""The host code of the rows in 8-bit integers, the layer on them, the expert layer and the rotary
positions under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): the library's ABI, their kernels' host
parts and tests/sanitize/abi_more_driver.cpp are compiled with the sanitizers (for the host alone) and linked with
the library's other objects; the executable must exit 0 with no report."""

import os
import subprocess

from .test_sanitizers import HERE, _run

SANITIZED = ["api.cpp", "moe.hip", "moe_layer.hip", "norm.hip", "rope.hip", "abi_more_driver.cpp"]


def test_more_abi_host_under_asan_ubsan(tmp_path):
    from rank_adapter_gemm_sgmv_amd import build as B

    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
           "-Xarch_host", "-g"]
    hipcc = B.hipcc()
    built = [os.path.join(B.OBJ_DIR, os.path.splitext(s)[0] + ".o") for s in B.SOURCES if s not in SANITIZED]
    if not all(os.path.exists(o) for o in built):
        B.build()
    objs, procs = [], []
    for src in SANITIZED:
        path = os.path.join(HERE if src == "abi_more_driver.cpp" else B.CSRC, src)
        objs.append(str(tmp_path / (os.path.splitext(src)[0] + ".o")))
        procs.append(subprocess.Popen([hipcc, *B.COMMON_FLAGS, *san, "-c", path, "-o", objs[-1]],
                                      stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    for p in procs:
        out, _ = p.communicate(timeout=600)
        assert p.returncode == 0, out[-4000:]
    exe = str(tmp_path / "abi_more_driver")
    link = [hipcc, f"--offload-arch={B.ARCH}", *objs, *built, "-Xarch_host", "-fsanitize=address",
            "-Xarch_host", "-fsanitize=undefined", "-o", exe]
    res = subprocess.run(link, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "all calls returned the expected status" in _run(exe)
