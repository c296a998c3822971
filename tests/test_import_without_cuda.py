"""The package imports under a torch built without CUDA, whose C module lacks the
CUDA bindings: the allocator and the host helpers need none of them."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in [n for n in vars(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import numpy as np
import block_paged_kv_gb300 as pkv
a = pkv.BlockAllocator(4, 4, 4)
r = a.begin()
a.reserve(r, 9)
t = np.asarray(a.table(r), np.int32)[None]
print(pkv.slot_mapping_host(t, 4, np.zeros(9, np.int32), np.arange(9, dtype=np.int32), 4).tolist())
"""


def test_allocator_and_host_helpers_without_cuda():
    run = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr
    assert run.stdout.strip() == str(list(range(9)))
