"""Logit processing at sizes whose tables and lists take just about 48 KB of a block's shared memory:
a launch of more has to ask for it, and what is static in the kernel counts too.

In a process of its own, ascending: one call that asks for more does so for all that follow.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir)
SWEEP = """
import sys
import torch
import rl_post_linear_gb300 as rlk

n, v0, v1, biases = (int(a) for a in sys.argv[1:])
g = torch.Generator(device="cuda").manual_seed(1)
wide = torch.randn(n, v1, device="cuda", generator=g)
t = torch.randint(0, v0, (n, 64), device="cuda", generator=g)
ids = torch.randint(0, v0, (n, biases), device="cuda", generator=g)
for v in range(v0, v1):
    x = wide[:, :v]
    want = x.scatter(1, t, x.gather(1, t) - 1.0)
    y = rlk.process_logits(x, t, presence=1.0, bias_ids=ids, bias_values=torch.zeros_like(ids).float())
    assert torch.equal(y, want), v
"""


@pytest.mark.parametrize("n,v0,v1,biases", [(256, 44897, 44993, 0), (16, 146849, 146913, 0),
                                            (33, 76780, 76850, 64)])
def test_about_48_kb(n, v0, v1, biases):
    run = subprocess.run([sys.executable, "-c", SWEEP, *map(str, (n, v0, v1, biases))], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
