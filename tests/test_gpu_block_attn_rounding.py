"""How far block attention's bf16 output may be from fp64: its own rounding, and nothing else of that size.

Tolerance, from the arithmetic.  The result is rounded to bf16: half a step, 2^-8 of the value at most.  Each softmax
weight is two bf16 parts, so 2^-16 of it is lost at most, and 2^-20 covers its exponential, the row sum's and the
division.  A score carries at most 36 accumulation roundings of up to two units of 2^-24 of the sum of |q_i k_i|, one
more of its scaling and one against the running max, and moves a weight by that times e at most, the row sum as much.
The output is accumulated in two tensor-core steps per 16 keys, each up to two units of 2^-24 of the sum of
weight |v|; a merge of 32 splits at most adds 32 more.
"""
import pytest
import torch

from speculative_decoding_tree_05_gb300 import ddtree
from parity_util import require_cuda
from test_gpu_block_attn import SCALE, call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    require_cuda()
    from speculative_decoding_tree_05_gb300 import build
    build.build()


def errors_and_tolerances(d, out):
    batch, nodes = d["q"].shape[:2]
    block = d["block"]
    idx, parent = d["idx"].cpu().numpy(), d["parent"].cpu().numpy()
    for b in range(batch):
        n = int(d["lens"][b])
        nb = -(-n // block)
        for t in range(nodes):
            blocks = sorted({int(x) for x in idx[b, t] if 0 <= x < nb})
            pos = [p for x in blocks for p in range(x * block, min(n, (x + 1) * block))]
            up, u = [], t
            while u >= 0:
                up.append(u)
                u = parent[b, u]
            slots = torch.cat([d["slot"][b][torch.tensor(pos, dtype=torch.long, device="cuda")].long(),
                               d["tree"][b][torch.tensor(up, device="cuda")].long()])
            k, q = d["kv"][slots].double(), d["q"][b, t].double()
            s = SCALE * (q @ k.T)
            p = torch.softmax(s, -1)
            want, mass = p @ k[:, :512], p @ k[:, :512].abs()
            err_s = float((SCALE * (q.abs() @ k.abs().T) * 72 + 2 * s.abs()).max()) * 2.0 ** -24
            steps = 2 * ((n + nodes + 15) // 16 + 1) + 32     # of the longest union there can be
            rel = 2.0 ** -16 + 2.0 ** -20 + 2 * 2.718 * err_s + 2 * steps * 2.0 ** -24
            yield (b, t), (out[b, t].double() - want).abs(), 2.0 ** -8 * want.abs() + rel * mass + 1e-30


@pytest.mark.parametrize("lens,nodes,heads,block,topk", [
    ([1], 1, 1, 16, 1), ([65], 1, 16, 16, 5), ([3000, 70], 9, 16, 64, 12), ([2500], 33, 16, 64, 9), ([900], 3, 128, 32, 9),
    ([5000], 1, 16, 16, 100), ([2000], 6, 24, 128, 7), ([700], 65, 1, 16, 7), ([4000, 2000, 0, 1], 1, 64, 32, 40)])
@pytest.mark.parametrize("amp", [0.1, 1.0])
def test_only_the_result_is_rounded_to_bf16(lens, nodes, heads, block, topk, amp):
    d = make(lens, nodes, heads, block, topk, seed=3 * nodes + heads, amp=amp)
    out, lse, st = call(d)
    assert st == 0
    for at, err, tol in errors_and_tolerances(d, out):
        assert bool((err <= tol).all()), (at, float((err / tol).max()))
