"""Order of shared-memory accesses in the compiled gated-activation kernels.

The transposed codes of a tile (`turn`, the first bytes of the shared memory, 16 KB
for each result that turns around at once) are read back by waves that did not
write them, and the next result reuses the memory. No wave may write into `turn`
between those reads and a barrier. What the compiler made of the source is read
from its assembly listing: the kernels are built here from their source, and no
GPU is needed.
"""
import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def hip_build():
    spec = importlib.util.spec_from_file_location("_iris_build", os.path.join(ROOT, "gemm_collective_tile_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


b = hip_build()


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("lds") / "fp8_quant.s")
    subprocess.run([b.HIPCC, *b.COMMON, "-x", "hip", "--cuda-device-only", "-S", os.path.join(b.CSRC, "fp8_quant.hip"),
                    "-o", out], check=True, capture_output=True, timeout=600)
    return open(out).read()


def written_before_a_barrier(body, turn):
    """Writes into the first `turn` bytes that follow a read of them with no barrier in between. Offsets are those
    of the instructions: a lane's own share of the address stays inside one array."""
    read, bad = False, []
    for line in body.splitlines():
        m = re.match(r"\s+(ds_read\w*|ds_write\w*|s_barrier)\b(.*)", line)
        if not m:
            continue
        op, rest = m.groups()
        off = re.search(r"offset:(\d+)", rest)
        inside = (int(off.group(1)) if off else 0) < turn
        if op == "s_barrier":
            read = False
        elif op == "ds_read_b128" and inside:
            read = True
        elif op.startswith("ds_write") and inside and read:
            bad.append(line.strip())
    return bad


def test_finds_a_write_that_no_barrier_orders():
    body = "\tds_read_b128 v[0:3], v9 offset:16384\n\tv_exp_f32 v1, v2\n\tds_write_b64 v7, v[4:5] offset:16384\n"
    assert written_before_a_barrier(body, 32768) == ["ds_write_b64 v7, v[4:5] offset:16384"]
    assert not written_before_a_barrier(body.replace("\tv_exp_f32 v1, v2", "\ts_barrier"), 32768)
    assert not written_before_a_barrier(body.replace("v[4:5] offset:16384", "v[4:5] offset:32768"), 32768)


@pytest.mark.skipif(not os.path.exists(b.HIPCC), reason="needs hipcc")
@pytest.mark.parametrize("kernel,results", [("fp8_swiglu_bwd_kernel", 2), ("fp8_swiglu_bwd_parts_kernel", 1)])
def test_a_turn_is_read_before_its_memory_is_written_again(listing, kernel, results):
    bodies = re.findall(rf"^(_ZN\S*{kernel}\S*):(.*?)s_endpgm", listing, re.S | re.M)
    assert len(bodies) == 4                                    # fp16 and bf16, whole and ragged
    for name, body in bodies:
        assert "ds_read_b128" in body and "s_barrier" in body
        assert not written_before_a_barrier(body, results * 128 * 128), name
