"""The hot loops of the output head's products (every tile of 256 x 256 and 128 x
128, both types), compiled for gfx950 here, keep every value in registers: no
scratch access and no wait for all loads in flight. Arithmetic on accumulators
straight behind the loop has made the compiler spill some of them inside it,
which took four times as long. The AMD assembly of our own build is read."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_gemm_epilogue_02_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


def loops(asm):
    """(function, lines) of each basic block of 32 matrix instructions and more."""
    function, block, out = None, [], []
    for line in asm.split("\n") + [".LBB0_0:"]:
        name = re.match(r"^(_Z\w+):", line)
        if name or re.match(r"^\.LBB\d+_\d+:", line):
            if sum("v_mfma" in x for x in block) >= 32:
                out.append((function, block))
            block = []
            function = name.group(1) if name else function
        elif not line.strip().startswith(";"):
            block.append(line)
    return out


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_main_loops_have_no_spills_or_drains(dtype, tmp_path):
    out = tmp_path / "k.s"
    cmd = [HIPCC, "-x", "hip", "-S", "--cuda-device-only", os.path.join(CSRC, f"kernels_head_{dtype}.hip"), "-o", str(out), "-O3",
           "-std=c++17", "--offload-arch=gfx950", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    found = loops(out.read_text())
    for kernel in ("head_stats", "head_grad", "head_dx", "head_dw"):
        assert sum(kernel in name for name, _ in found) == 2, kernel
    for name, lines in found:
        body = "\n".join(lines)
        assert "scratch_" not in body, f"{name}: scratch access in the loop"
        assert "vmcnt(0)" not in body, f"{name}: all loads waited for in the loop"
