"""tests/sanitize/abi_more_driver.cpp with the host code of every source of the library under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): its sweeps of workspace sizes go through the planners of the 8-bit layers in
decode_gemm.hip, gemm_fp8.hip and shrink.hip.  The present sources are compiled for the host alone, around an empty GPU
binary (the driver launches nothing)."""

import os
import subprocess

from .test_sanitizers import HERE, _run


def test_every_source_under_asan_ubsan(tmp_path):
    from rank_adapter_gemm_sgmv_amd import build as B

    hipcc = B.hipcc()
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
           "-Xarch_host", "-g"]
    empty, binary = tmp_path / "empty.hip", str(tmp_path / "empty.hipfb")
    empty.write_text("__global__ void nothing() {}\n")
    subprocess.run([hipcc, f"--offload-arch={B.ARCH}", "--offload-device-only", "-c", str(empty), "-o", binary],
                   check=True, capture_output=True)
    host = ["--offload-host-only", "-Xclang", "-fcuda-include-gpubinary", "-Xclang", binary]
    objs, procs = [], []
    for src in B.SOURCES + ["abi_more_driver.cpp"]:
        path = os.path.join(HERE if src == "abi_more_driver.cpp" else B.CSRC, src)
        objs.append(str(tmp_path / (os.path.splitext(src)[0] + ".o")))
        only = host if src.endswith(".hip") else []
        procs.append(subprocess.Popen([hipcc, *B.COMMON_FLAGS, *only, *san, "-c", path, "-o", objs[-1]],
                                      stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    for p in procs:
        out, _ = p.communicate(timeout=600)
        assert p.returncode == 0, out[-4000:]
    exe = str(tmp_path / "abi_more_driver")
    link = [hipcc, f"--offload-arch={B.ARCH}", *objs, "-Xarch_host", "-fsanitize=address",
            "-Xarch_host", "-fsanitize=undefined", "-o", exe]
    res = subprocess.run(link, capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "all calls returned the expected status" in _run(exe)
