"""Norms and sampling called from two host threads at a time, with sizes that need different amounts
of shared memory: neither call may change what the other one's launch is allowed."""
import threading

import pytest
import torch

import rl_post_linear_gb300 as rlk
from helpers import dev

pytestmark = pytest.mark.gpu


def at_once(*calls, times=3000):
    """Runs each call `times` times, one thread a call; the first error of any is raised."""
    errors = []

    def work(call):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(times):
                    call()
        except Exception as e:                                     # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("backward", [False, True])
def test_norms_of_different_widths(backward):
    calls, outs = [], []
    for h in (8208, 16376, 8208, 16376):
        x = torch.randn(1, h, generator=torch.Generator().manual_seed(h)).to(dev())
        w, rstd = torch.ones(h, device=dev()), torch.ones(1, device=dev())
        y, ws = torch.empty_like(x), torch.empty(256, dtype=torch.uint8, device=dev())

        def forward(x=x, w=w, y=y, rstd=rstd):
            rlk.rlk_rms_norm_fwd(x, w, None, 1e-6, y, None)

        def back(x=x, w=w, y=y, rstd=rstd, ws=ws):
            rlk.rlk_rms_norm_bwd(x, w, x, rstd, None, y, None, ws)

        calls.append(back if backward else forward)
        calls[-1]()
        torch.cuda.synchronize()
        outs.append((y, y.clone()))
    at_once(*calls, times=20000)
    assert all(torch.equal(y, want) for y, want in outs)


def test_sampling_of_different_vocabularies():
    calls, outs = [], []
    for v in (300000, 700000):
        z = 0.5 * torch.randn(1, v, generator=torch.Generator().manual_seed(v)).to(dev())
        u = torch.full((1,), 0.3, device=dev())
        out = (torch.empty(1, dtype=torch.int64, device=dev()), torch.empty(1, device=dev()),
               torch.empty(1, device=dev()))
        ws = torch.empty(rlk.rlk_sample_logits_workspace_bytes(1, v), dtype=torch.uint8, device=dev())

        def call(z=z, u=u, out=out, ws=ws):
            rlk.rlk_sample_logits(z, u, None, 1.0, 0, 0.9, 0.0, *out, ws)

        call()
        torch.cuda.synchronize()
        calls.append(call)
        outs.append([(t, t.clone()) for t in out])
    at_once(*calls)
    assert all(torch.equal(t, want) for out in outs for t, want in out)
