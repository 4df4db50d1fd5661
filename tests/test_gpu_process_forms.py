"""Logit processing in its forms of two launches: rows whose listed columns are changed by several
blocks, and calls behind the launches that wrote their tokens, lengths and settings."""
import pytest
import torch

import rl_post_linear_gb300 as rlk
from helpers import dev, same_bits
from test_gpu_process import DTYPES, check, gen, history, logits, pack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,v,length", [(128, 151936, 4200), (100, 170001, 9000), (140, 90001, 40000)])
def test_a_row_by_several_blocks(n, v, length, dtype):
    t, full, prompt = history(n, v, length, v, 0.02)
    t[:, 1::97] = v - 1 - (t[:, 1::97] % 1000)               # the last range too
    few = torch.arange(n, device=dev()) % 4 == 1             # rows that one block takes
    full = torch.where(few, full % 4000, full)
    prompt = torch.minimum(prompt, full)
    g = gen(length)
    ids = torch.randint(-1, v, (n, 5), generator=g).to(dev())
    vals = torch.randn(n, 5, generator=g).to(dev())
    if length > 16384:
        full[3], prompt[3] = length, 0                       # counts past 14 bits
    mask = torch.zeros(n, dtype=torch.uint8, device=dev())
    mask[[0, 1, 2, 3, 5, n // 2, n - 2, n - 1]] = 1
    allow = (torch.rand(n, v, generator=g) < 0.7).to(dev())
    for a in (None, allow):
        x = logits(n, v, 71, dtype, pad=3)
        want = check(x, t, full, prompt, 1.3, 0.2, 0.1, ids, vals, a, mask)
        same = x.clone()
        check(same, t, full, prompt, 1.3, 0.2, 0.1, ids, vals, a, mask, same)
        assert same_bits(same[mask != 0], want[mask != 0])
        assert same_bits(same[mask == 0], x[mask == 0])
        for i in (1, n - 1):                                 # as each row by itself
            one = rlk.process_logits(x[i:i + 1].clone(), t[i:i + 1], full[i:i + 1],
                                     prompt[i:i + 1], 1.3, 0.2, 0.1, ids[i:i + 1], vals[i:i + 1],
                                     None if a is None else pack(a[i:i + 1]))
            assert same_bits(one[0], want[i])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,v,length", [(128, 151936, 4200), (100, 170001, 9000)])
def test_a_row_that_cannot_be_by_several_blocks(n, v, length, in_place):
    x = logits(n, v, 72, torch.float32)
    t, full, _ = history(n, v, length, v + 1)
    full[:] = length
    full[5:9] = 50                                           # rows of few tokens
    bad = [3, 6, n - 2, n - 1]
    t[3, length - 1], t[6, 49] = v, 1 << 40                  # an id >= V, in a long row and a short
    full[n - 2], full[n - 1] = length + 1, -1
    out = x.clone() if in_place else None
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    y = rlk.process_logits(x if out is None else out, t, full, presence=1.0, out=out, error_word=err)
    assert int(err.item()) == rlk.RLK_DEVERR_TARGET_RANGE | rlk.RLK_DEVERR_SAMPLE_PARAM
    assert torch.isnan(y).any(1).nonzero()[:, 0].tolist() == bad
    assert bool(torch.isnan(y[bad]).all())
    for i in (0, 5):
        seen = t[i, :int(full[i])].unique()
        want = x[i].clone()
        want[seen] -= 1.0
        assert same_bits(y[i], want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,v", [(400, 60000), (200, 151936)])
def test_captured_behind_what_writes_its_tokens(n, v, in_place):
    # the second launch reads tokens, lengths and settings before it waits for the first
    length = 64
    x = logits(n, v, 73, torch.float32)
    t, full, prompt = (torch.zeros_like(a) for a in history(n, v, length, 74))
    rep = torch.ones(n, device=dev())
    src = [torch.zeros_like(a) for a in (t, full, prompt, rep)]
    y = torch.empty_like(x)

    def step():
        if in_place:
            y.copy_(x)
        for to, a in zip((t, full, prompt, rep), src):
            to.copy_(a)
        rlk.process_logits(y if in_place else x, t, full, prompt, rep, 0.1, 0.1, out=y)
        rlk.process_logits(y, t, full, prompt, rep, 0.1, 0.1, out=y)      # and on its own output

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(75, 80):
        x.copy_(logits(n, v, seed, torch.float32))
        for to, a in zip(src, (*history(n, v, length, seed + 30),
                               1.0 + torch.rand(n, generator=gen(seed)).to(dev()))):
            to.copy_(a)
        for a in (t, full, prompt):
            a.zero_()
        graph.replay()
        got = y.clone()
        torch.cuda.synchronize()
        want = rlk.process_logits(x.clone(), *src[:3], src[3], 0.1, 0.1)
        torch.cuda.synchronize()
        want = rlk.process_logits(want.clone(), *src[:3], src[3], 0.1, 0.1)
        assert same_bits(got, want)
