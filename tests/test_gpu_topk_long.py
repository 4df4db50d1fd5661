"""Top-K log-probs of vocabularies whose segments are long, so that the segments found are read again
some at a time.

The tolerances are those of the shorter ones: V = 2^22 in fp32 is 64 units a thread, so a row's sum
takes 31 + 5 + 64 + 13 additions at most, 2^-22 + 113 2^-24 < 2^-17 of it.
"""
import pytest
import torch

import rl_post_linear_gb300 as rlk
from helpers import dev
from test_gpu_topk import DTYPES, check, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("v,k", [(163840, 1024), (163841, 1024), (262144, 1000), (300001, 700),
                                 (327681, 1024), (524288, 512), ((1 << 20) + 77, 300),
                                 ((1 << 22) - 1, 65), (1 << 22, 100), (1 << 22, 1000)])
def test_values(v, k, dtype):
    check(normal(2, v, v % 1000 + k, dtype), k, 0.9)
    check(normal(2, v - 3, k, dtype, pad=3)[:, 1:], k)          # rows that start on no 16 bytes


@pytest.mark.parametrize("v", [262144, 1 << 20])
def test_banned_tokens_and_ties(v):
    x = normal(3, v, 1)
    x[0, torch.rand(v, device=dev(), generator=torch.Generator(dev()).manual_seed(2)) < 0.999] = -torch.inf
    x[1] = (x[1] * 4).round()                                   # hundreds of equals
    x[2, : v // 2] = -torch.inf
    for k in (100, 1024):
        check(x, k)


def time_of(n, v, k):
    x = normal(n, v, 3)
    rlk.topk_logp(x, k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rlk.topk_logp(x, k)
    best = float("inf")
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("v,k", [(163841, 1024), (262144, 1024), (524288, 512), (1 << 22, 100)])
def test_no_search_of_the_row_where_segments_get_longer(v, k):
    # such a search takes 30 to 100 times as long as the rows of its own length do
    assert time_of(4, v, k) < 8 * max(1.0, v / 163840) * time_of(4, 163840, 1024)
