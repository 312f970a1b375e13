"""Router losses at expert counts where a launch's shared memory crosses a limit, each in a process
of its own: a limit that an earlier, larger call has raised stays raised for that kernel.

Counts are integers: equal.  Probabilities and losses of 40 tokens carry at most 40 + 128 roundings
of 2^-24 relative (one token's exp, a sum over 32 lanes' 32 terms in short chains and a division
stay below 128), the z loss four times that (its square and the logarithm)."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys
import torch
import nvfp4_mixture_experts_softmax_gb300 as moe
router = sys.argv[1]
for E in map(int, sys.argv[2:]):
    g = torch.Generator(device="cuda").manual_seed(E)
    l = torch.randn(40, E, device="cuda", generator=g) * 2
    ids = torch.rand(40, E, device="cuda", generator=g).topk(8, -1).indices.int()
    o = moe.router_loss(l, ids, router=router)
    d = l.double()
    s = torch.softmax(d, -1) if router == "softmax" else torch.nn.functional.softplus(d, threshold=1e9).sqrt()
    P = (s / s.sum(-1, keepdim=True)).mean(0)
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E)
    want = E * (counts.double() / (40 * 8) * P).sum(), (torch.logsumexp(d, -1) ** 2).mean()
    tol = 168 * 2.0 ** -24
    assert torch.equal(o["counts"].long(), counts) and int(o["tokens"]) == 40, E
    assert bool(((o["probs"].double() - P).abs() <= tol * P).all()), E
    assert abs(float(o["losses"][0] - want[0])) <= tol * float(want[0]), E
    assert abs(float(o["losses"][1] - want[1])) <= 4 * tol * float(want[1]), E
print("agrees")
"""


# 17 (or 21, up to 512 experts) rows of the experts' sums beside the kernel's own bytes: 48 KB at 719
# experts; 720 to 722 are above it only with those bytes
@pytest.mark.parametrize("router", ["softmax", "sqrtsoftplus"])
@pytest.mark.parametrize("sizes", [(719, 720), (721,), (722,), (723, 724), (488, 512, 513), (585, 1023, 1024)])
def test_first_call_of_a_process(router, sizes):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", SCRIPT, router, *map(str, sizes)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "agrees" in r.stdout, r.stdout + r.stderr
