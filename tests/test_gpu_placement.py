"""The XCD-local variants stay legal for a program that attends before its first
convolution: attention needs no device set-up and launches any number of
workgroups, after which a queue deals the next ones out from another XCD."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A process of its own, since the probe runs once in each.
PROGRAM = """
import sys
import torch
from _gpu_helpers import legal_configs
from tensor_compiler_tiling_amd import convtile as ct
from tensor_compiler_tiling_amd import workloads as wl
odd = int(sys.argv[1])
dev = torch.device("cuda:0")
cache = ct.KVCache(*(torch.randn(odd, 1, 16, 64, device=dev).bfloat16() for _ in range(2)))
lens = torch.full((odd,), 16, dtype=torch.int32, device=dev)
q = torch.randn(odd, 1, 64, device=dev).bfloat16()
streams = [torch.cuda.Stream() for _ in range(8)]
torch.cuda.synchronize()
for s in [None] + streams:
    y = ct.kv_attention(q, cache, lens, stream=s)  # a workgroup a sequence
torch.cuda.synchronize()
w = wl.CONV_WORKLOADS["resnet_final_c512_7x7_k3"]
names = {ct.variants()[c.variant]["name"] for c in legal_configs(w)}
print("legal:", sorted(n for n in names if n.startswith("f32skc7x_")), flush=True)
"""


@pytest.mark.parametrize("odd", [1, 3, 5])
def test_attention_before_the_first_convolution(odd):
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(odd)], capture_output=True, text=True, timeout=100, cwd=ROOT,
                       env=dict(os.environ, PYTHONPATH=os.pathsep.join((ROOT, os.path.join(ROOT, "tests")))))
    assert r.returncode == 0, r.stdout + r.stderr
    assert "f32skc7x_" in r.stdout, r.stdout
