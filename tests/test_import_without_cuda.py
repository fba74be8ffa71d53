"""A torch that was built without CUDA lacks some of its private functions: the package imports all the same, and its
host-only functions work."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_host_only_functions_work():
    code = """
import torch
for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, n):
        delattr(torch._C, n)
import top_moe_expert_gb300 as moe
print(moe.moe_align_capacity(3, 2, 4, 8), moe.moe_fp4_scale_cols(288, moe.MOE_FP4_NVFP4))
try:
    moe.moe_topk_softmax(torch.zeros((4, 16)), 2)
except ValueError as e:
    print(e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert " 32\n" in r.stdout and "must be a CUDA tensor" in r.stdout
