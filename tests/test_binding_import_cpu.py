"""The package on a torch without the raw stream call: it imports, host calls work, and the stream comes from the public
API."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import types
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
import int8_dequant_dot_amd as loom
assert loom.status_string(loom.OK)
assert loom.launch_config_lookup("copy_f32") >= 0
asked = []
torch.cuda.current_stream = lambda device: asked.append(device) or types.SimpleNamespace(cuda_stream=123)
torch.cuda.current_device = lambda: 1
assert loom._target(types.new_class("T", (torch.Tensor,), {}, lambda d: d.update(is_cuda=True))(), "x") == (1, 123)
assert asked == [1]
"""


def test_import_without_the_raw_stream_call():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
