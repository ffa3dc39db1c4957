"""The block operators' entry points on the host alone: csrc/block_ops.cpp and csrc/fp8_ops.cpp
linked with stand-ins of the HIP runtime and of the kernels' launches
(tests/native/block_ops_main.cpp), called from several threads and with no memory left."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.skipif(not os.path.exists(HIPCC) or shutil.which("g++") is None, reason="needs hipcc and g++")
def test_calls_that_share_a_stream_share_its_workspaces_in_turn(tmp_path):
    objs = []
    csrc = os.path.join(ROOT, "gemm_collective_tile_amd", "csrc")
    for src in (os.path.join(csrc, "block_ops.cpp"), os.path.join(csrc, "fp8_ops.cpp"),
                os.path.join(ROOT, "tests", "native", "block_ops_main.cpp")):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        subprocess.run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17", "-fPIC", "-x", "hip",
                        "-I", os.path.join(ROOT, "include"), "-c", src, "-o", objs[-1]],
                       check=True, capture_output=True, timeout=600)
    exe = str(tmp_path / "block_ops_main")
    subprocess.run(["g++", "-pthread", *objs, "-o", exe], check=True, capture_output=True, timeout=600)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout[-2000:], r.stderr[-2000:])
