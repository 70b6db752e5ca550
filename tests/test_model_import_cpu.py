"""The package where the extension of the model operators does not load: the
GEMMs and the block's operators are there, and each model operator says what is
missing when it is used."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys
class Missing:
    def find_spec(self, name, path=None, target=None):
        if name.endswith("._model"):
            raise ImportError("undefined symbol")
sys.meta_path.insert(0, Missing())
import torch
import dense_gemm_epilogue_02_amd as g
try:
    g.mx4_quantize(torch.ones(2, 32))
except ImportError:
    print("no block")
except (TypeError, ValueError, RuntimeError):
    print("block")
x, w, t, k = torch.ones(2, 8), torch.ones(3, 8), torch.zeros(2, dtype=torch.int64), torch.zeros(2, 1, dtype=torch.int32)
order = g.ExpertOrder(torch.zeros(2, dtype=torch.int32), k)
for call in (lambda: g.linear_cross_entropy(x, w, t), lambda: g.linear_cross_entropy_backward(t, x, w, t, (t, t)),
             lambda: g.linear_distillation(x, w, k, k), lambda: g.linear_distillation_backward(t, x, w, (k,) * 5),
             lambda: g.expert_sort(k, 1), lambda: g.expert_gather(x, order), lambda: g.expert_combine(x, order),
             lambda: g.expert_combine_backward(x, x, order)):
    try:
        call()
    except ImportError as e:
        print("ImportError" if "_model" in str(e) and "does not load" in str(e) and "undefined" in str(e.__cause__) else e)
"""


def test_the_rest_without_the_extension():
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["block"] + ["ImportError"] * 8, r.stdout
