"""The binding of 8-bit rows where torch lacks the private function that it makes outputs with (no GPU needed)."""
import subprocess
import sys

from tests.conftest import ROOT

PROGRAM = """
import torch
del torch._C._dynamo.guards._empty_strided_cuda
import speculative_decoding_verification_45_gb300 as sv
from speculative_decoding_verification_45_gb300 import rows

asked = []
torch.empty_strided = lambda *a, **k: asked.append((a, k))
rows._new((3, 5, 32), torch.bfloat16, None)
rows._new((7, 16), torch.float8_e4m3fn, None)
assert asked == [(((3, 5, 32), (160, 32, 1)), dict(dtype=torch.bfloat16, device="cuda")),
                 (((7, 16), (16, 1)), dict(dtype=torch.float8_e4m3fn, device="cuda"))], asked
assert callable(sv.rows_quantise)
"""


def test_outputs_are_made_by_the_public_function():
    done = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr
