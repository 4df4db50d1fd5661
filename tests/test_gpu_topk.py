"""Top-K log-probs against the definition: ids exactly (a stable sort), logp and lse in float64.

The fp32 sum of a row's weights: exponentials good to 2^-22 (their argument's roundings weigh
t 2^-t of 2^-23 each, less than that), at most 31 additions in a lane, 5 in a warp, 16 units a
thread and 13 in the block, 2^-24 each: 2^-22 + 65 2^-24 < 2^-17.8.  The logarithm and its product
with ln 2: 2^-22 and 2^-23 of at most 16.  Then z = (x - max)/T: two roundings, one of the sum.
"""
import math

import numpy as np
import pytest
import torch

import rl_post_linear_gb300 as rlk
from helpers import dev, same_bits

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]
ATOL, RTOL = 2.0 ** -17, 2.0 ** -22


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(n, v, seed, dtype=torch.float32, std=2.0, pad=0):
    return (std * torch.randn(n, v + pad, generator=gen(seed))).to(dtype).to(dev())[:, :v]


def check(x, k, t=1.0, mask=None):
    n, v = x.shape
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    ids, logp, lse = rlk.topk_logp(x, k, t, mask, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and ids.shape == (n, k)
    z = x.float().cpu().double().numpy()
    ids, logp, lse = ids.cpu().numpy(), logp.cpu().double().numpy(), lse.cpu().double().numpy()
    for i in range(n):
        if mask is not None and int(mask[i]) == 0:
            assert np.all(ids[i] == -1) and np.all(logp[i] == 0) and lse[i] == 0
            continue
        want = np.argsort(-z[i], kind="stable")[:k]
        want = want[z[i][want] > -np.inf]
        m = want.size
        assert np.array_equal(ids[i, :m], want), i
        assert np.all(ids[i, m:] == -1) and np.all(logp[i, m:] == -np.inf)
        top = z[i].max()
        l64 = top / t + math.log(np.exp((z[i] - top) / t).sum())
        assert abs(lse[i] - l64) <= ATOL + RTOL * (abs(l64) + abs(top) / t)
        lp = z[i][want] / t - l64
        assert np.all(np.abs(logp[i, :m] - lp) <= ATOL + RTOL * np.abs(lp))
    return ids


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("v", [1, 2, 7, 31, 33, 127, 255, 257, 1023, 1024, 1025, 2049, 5003, 16385,
                               32003, 65537])
def test_vocabulary_sizes(v, dtype):
    for k in (1, 2, 5, 20, 64, 257, 1024):
        check(normal(4, v, v + k, dtype), k, 0.7)


@pytest.mark.parametrize("v,dtype", [(151936, torch.float32), (129280, torch.bfloat16)])
@pytest.mark.parametrize("k", [1, 20, 64, 300, 1000, 1024])
def test_large_vocabularies(v, dtype, k):
    check(normal(5, v, k, dtype), k, 1.5)


@pytest.mark.parametrize("dtype", DTYPES)
def test_beyond_the_usual_vocabularies(dtype):
    for v, k in (((1 << 20) + 77, 50), (1 << 22, 1024), ((1 << 22) - 1, 3)):
        check(normal(2, v, 5, dtype), k)


@pytest.mark.parametrize("n", [1, 2, 37, 76, 77, 153, 304, 305, 700])
def test_row_counts_do_not_change_a_row(n):
    x = normal(n, 70001, 6, torch.bfloat16)
    ids, logp, lse = rlk.topk_logp(x, 33, 0.9)
    for i in sorted({0, n // 2, n - 1}):
        a, b, c = rlk.topk_logp(x[i:i + 1].clone(), 33, 0.9)
        assert torch.equal(a[0], ids[i]) and same_bits(b[0], logp[i]) and same_bits(c[0], lse[i])
    check(x[:3], 33, 0.9)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_strides(pad, dtype):
    check(normal(6, 9001, 7, dtype, pad=pad), 50)
    check(normal(6, 9002, 8, dtype, pad=pad)[:, 1:], 50)


@pytest.mark.parametrize("k", [1, 64, 1000, 1024])
@pytest.mark.parametrize("v", [1500, 40001, 151936])
@pytest.mark.parametrize("kind", ["constant", "ascending", "descending", "steps", "few", "zeros",
                                  "two", "lowest", "cluster", "tiny", "huge"])
def test_ties_and_orders(kind, v, k):
    i = torch.arange(v, dtype=torch.float64)
    g = gen(v)
    x = {
        "constant": torch.full((v,), 1.25),
        "ascending": i / v,
        "descending": -i / 64,
        "steps": (i % 7),
        "few": torch.where(i % 997 == 5, 1.0, -math.inf),
        "zeros": torch.where(torch.rand(v, generator=g) < 0.5, 0.0, -0.0),
        "two": torch.where(torch.rand(v, generator=g) < 0.01, 3.0, -3.0),
        "lowest": torch.where(torch.rand(v, generator=g) < 0.99, torch.finfo(torch.float32).min,
                              torch.randn(v, generator=g)),
        "cluster": torch.where((i >= 1024) & (i < 3200), 9.0 + torch.rand(v, generator=g), 0.0),
        "tiny": 1e-30 * torch.randn(v, generator=g),
        "huge": 1e30 * torch.randn(v, generator=g),
    }[kind]
    for dtype in DTYPES:
        row = x.to(torch.float32)
        if dtype == torch.bfloat16:
            row = row.clamp(min=torch.finfo(dtype).min).where(row > -math.inf, row).to(dtype)
        check(torch.stack((row, row.flip(0))).to(dev()), k, 1.0)


@pytest.mark.parametrize("banned", [0.5, 0.99, 0.9999])
def test_banned_tokens(banned):
    x = normal(6, 60000, 9)
    x[torch.rand(x.shape, generator=gen(10)).to(dev()) < banned] = -math.inf
    x[:, 59999] = 0.5
    check(x, 64)
    check(x, 1024)
    check(x.to(torch.bfloat16), 200)


def test_rows_without_an_answer_and_inactive_rows():
    x = normal(7, 3000, 11)
    x[1] = -math.inf
    x[2, 17] = math.nan
    x[3, 2999] = math.inf
    x[5] = math.nan
    mask = torch.tensor([1, 1, 1, 1, 1, 0, 1], dtype=torch.uint8, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    ids, logp, lse = rlk.topk_logp(x, 5, 1.0, mask, err)
    assert int(err.item()) == rlk.RLK_DEVERR_LOGITS
    for i in (1, 2, 3):
        assert bool((ids[i] == -1).all()) and bool(torch.isnan(logp[i]).all())
        assert bool(torch.isnan(lse[i]))
    assert bool((ids[5] == -1).all()) and bool((logp[5] == 0).all()) and lse[5] == 0
    check(x[[0, 4, 6]], 5)


@pytest.mark.parametrize("t", [1e-4, 0.05, 1.0, 30.0, 1e6])
def test_temperatures(t):
    check(normal(3, 20000, 12), 40, t)


def test_two_streams_and_a_captured_call():
    x, y = normal(3, 151936, 13), normal(300, 40000, 14, torch.bfloat16)
    want = [rlk.topk_logp(x, 20), rlk.topk_logp(y, 64)]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        p = [rlk.topk_logp(x, 20) for _ in range(8)]
    with torch.cuda.stream(b):
        q = [rlk.topk_logp(y, 64) for _ in range(8)]
    torch.cuda.synchronize()
    for got, ref in [(g, want[0]) for g in p] + [(g, want[1]) for g in q]:
        assert torch.equal(got[0], ref[0]) and same_bits(got[1], ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rlk.topk_logp(x, 20)
    x.copy_(normal(3, 151936, 15))
    graph.replay()
    ref = rlk.topk_logp(x, 20)
    assert torch.equal(out[0], ref[0]) and same_bits(out[1], ref[1]) and same_bits(out[2], ref[2])


@pytest.mark.parametrize("dtype", DTYPES)
def test_offsets_past_32_bits(dtype):
    v, apart = 5003, 1 << 30
    room = torch.empty(3 * apart + v, dtype=dtype, device=dev())
    x = room.as_strided((4, v), (apart, 1))
    x.copy_(torch.randn(4, v, generator=gen(61)))
    want = rlk.topk_logp(x.clone(), 20)
    for got, w in zip(rlk.topk_logp(x, 20), want):
        assert same_bits(got, w)
