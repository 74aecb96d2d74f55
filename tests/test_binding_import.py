"""The binding needs CUDA in torch for its calls, not to be imported: the sizes and
host checks work with a torch that has none."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
import nf4_base_lora_b200 as nf
assert nf.qlora_grouped_fwd_workspace_bytes(16, 2, 128, 128, 8) > 0
"""


def test_import_without_cuda_in_torch():
    subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, check=True, timeout=300)
