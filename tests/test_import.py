"""The package imports and names the current stream with nothing but torch's public functions."""
import subprocess
import sys
from pathlib import Path

ROOT = Path(__file__).resolve().parent.parent

WITHOUT = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import bit_matmul_amd as lq

class Stream:
    def __init__(self, device):
        self.cuda_stream = 4096 + device

assert lq.lq_version() > 0 and lq.lq_packed_size(16, 128, 2, 5) > 0
layer = lq.LQInt8Layer(64, 64, 64, 1, 0, 1 << 20, None, 1 << 20, None)
assert lq.lq_int8_gemm_plan(layer, 1)["workgroups"] >= 1
torch.cuda.current_device = lambda: 2
torch.cuda.current_stream = lambda device=None: Stream(device)
assert lq._stream(None) == 4098
assert lq._current_device() == 2
"""


def test_import_without_private_names():
    """A torch without the two private functions behind the short way to a stream's handle: the package
    imports, the queries work, and the public functions are asked for device and stream."""
    run = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr
