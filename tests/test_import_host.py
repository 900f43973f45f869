"""The package imports, and its host-side calls work, on a torch that was built without CUDA."""
import os
import subprocess
import sys

SCRIPT = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
import block_sparse_attention_nsa_gb300 as nsa
from block_sparse_attention_nsa_gb300 import build
build.build()
dims = nsa.make_dims(1, 64, 4, 2, 128, 64, 4, torch.bfloat16)
assert nsa.workspace_size(dims)
assert nsa.kv4_decode_workspace_size(8, 64, 2, 128, 3, 8) > 0
pool = nsa.kv4_pool(2, 64, 2, 128, device="cpu")
assert pool.shape == (2, 2, 64 * 144)
try:
    nsa.kv4_read(pool, torch.zeros(2, dtype=torch.int32), 128)
    raise SystemExit("a pool on the CPU was taken")
except ValueError:
    print("imported")
"""


def test_import_without_cuda_names():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", SCRIPT], cwd=root, capture_output=True, text=True,
                         timeout=600)
    assert "imported" in run.stdout, run.stderr[-2000:]
