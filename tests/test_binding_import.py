"""The package on a torch without GPU support: it imports, and a call is refused as
one with CPU tensors is."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
for n in [n for n in dir(torch._C) if n.startswith("_cuda_get")]:
    delattr(torch._C, n)
import moe_expert_grouped_amd as mi
f8 = torch.float8_e4m3fn
a, s = torch.zeros(16, 128).to(f8), torch.zeros(16, 4)
x, i = torch.zeros(4, 16), torch.zeros(4, dtype=torch.int32)
for call in (lambda: mi.mm_fp8_block(a, a, s, s[:1]), lambda: mi.fp8_quantize(x),
             lambda: mi.add_rmsnorm_fp8(x, x[0]), lambda: mi.moe_combine_rows(x, i, x[:, :1].contiguous()),
             lambda: mi.moe_permute_rows_backward(x, i, 1)):
    try:
        call()
    except ValueError as e:
        assert "on the GPU" in str(e), e
    else:
        raise AssertionError("not refused")
print("refused")
"""


def test_import_and_refusals_without_gpu_support():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr[-800:]
