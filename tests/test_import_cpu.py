"""The package where its Python extension does not load: the GEMMs are there, and
the block operators say what is missing when they are used."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys
class Missing:
    def find_spec(self, name, path=None, target=None):
        if name.endswith("._block"):
            raise ImportError("undefined symbol")
sys.meta_path.insert(0, Missing())
import dense_gemm_epilogue_02_amd as g
plan = g.Plan("bf16", la="row", lb="col", lc="row")
print(plan.describe(512, 512, 512, 256)["tile"], g.gemm_mx4_padded(3))
plan.close()
import torch
for call in (lambda: g.mx4_quantize(torch.ones(2, 32)), lambda: g.norm_residual(None, torch.ones(2, 32))):
    try:
        call()
    except ImportError as e:
        print("ImportError" if "not built or does not load" in str(e) and "undefined" in str(e.__cause__) else e)
"""


def test_gemms_without_the_extension():
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    lines = r.stdout.split("\n")
    assert lines[0].endswith(" 256") and lines[1:3] == ["ImportError"] * 2, r.stdout
