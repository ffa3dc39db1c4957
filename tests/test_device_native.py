"""The library's device check on the host alone: csrc/iris_local.cpp linked with stand-ins of the HIP runtime
(tests/native/device_main.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.skipif(not os.path.exists(HIPCC) or shutil.which("g++") is None, reason="needs hipcc and g++")
def test_another_gpu_is_refused_at_every_call(tmp_path):
    objs = []
    for src in (os.path.join(ROOT, "gemm_collective_tile_amd", "csrc", "iris_local.cpp"),
                os.path.join(ROOT, "tests", "native", "device_main.cpp")):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        subprocess.run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-x", "hip",
                        "-I", os.path.join(ROOT, "include"), "-c", src, "-o", objs[-1]],
                       check=True, capture_output=True, timeout=600)
    exe = str(tmp_path / "device_main")
    subprocess.run(["g++", "-pthread", *objs, "-Wl,--unresolved-symbols=ignore-all", "-o", exe], check=True,
                   capture_output=True, timeout=600)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout[-2000:], r.stderr[-2000:])
