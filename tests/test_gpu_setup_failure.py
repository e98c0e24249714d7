"""A failed set-up of the cache-size and block kernels leaves the verify calls as they are (host-side fault, child process)."""
import os
import subprocess
import sys

import pytest

from parity_util import build_and_load, require_cuda

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

CHILD = """
import sys
sys.path[:0] = [{root!r}, {here!r}]
import torch
from parity_util import build_and_load, run_gpu
from speculative_decoding_tree_05_gb300 import ddtree, workloads as wl
L = build_and_load("testhooks")
L.ddtree_test_fail_cache_setup({fail})
w = wl.make_workload("tiny", prefix=(300,))
out, lse, st, _, _ = run_gpu(w, library=L)
assert st == 0 and bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
s = ddtree.BlockSelector(1, 1, 16, 320, 16, 5, library=L)
a = (torch.zeros(1, 1, 16, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 20, 576, dtype=torch.bfloat16, device="cuda"),
     torch.zeros(1, 20, device="cuda"), torch.tensor([320], dtype=torch.int32, device="cuda"))
try:
    s(*a)
    code = 0
except ddtree.DDTError as e:
    code = e.code
torch.cuda.synchronize()
print("code", code)
"""


@pytest.mark.parametrize("fail,code", [(0, 0), (1, -6)])
def test_verify_does_not_need_the_cache_kernels(fail, code):
    require_cuda()
    build_and_load("testhooks")
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=os.path.dirname(HERE), here=HERE, fail=fail)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split()[-2:] == ["code", str(code)]
