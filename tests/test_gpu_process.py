"""Penalties, biases and masks on logits against the definition in float64, one row at a time.

A listed column goes through at most a division, a multiply-add, a subtraction, the sum of its B
biases and their addition, each rounded to fp32 (2^-24 of a value no larger than the sum of the
magnitudes that enter), then once to the output's type (2^-8 for bf16).  All others keep their
bits.
"""
import numpy as np
import pytest
import torch

import rl_post_linear_gb300 as rlk
from helpers import dev, same_bits

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def logits(n, v, seed, dtype, pad=0):
    x = 4.0 * torch.randn(n, v + pad, generator=gen(seed))
    return x.to(dtype).to(dev())[:, :v]


def pack(allow):
    """int32 words [N, ceil(V / 32)] of a boolean [N, V]; bits past V are 0."""
    n, v = allow.shape
    b = np.zeros((n, (v + 31) // 32 * 32), np.uint8)
    b[:, :v] = allow.cpu().numpy()
    return torch.from_numpy(np.packbits(b, axis=1, bitorder="little").view(np.int32).copy()).to(dev())


def at(value, i):
    return float(value[i]) if isinstance(value, torch.Tensor) else float(np.float32(value))


def check(x, tokens=None, lengths=None, prompt_lengths=None, repetition=1.0, frequency=0.0,
          presence=0.0, bias_ids=None, bias_values=None, allowed=None, mask=None, out=None):
    n, v = x.shape
    before = x.clone()
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    y = rlk.process_logits(x, tokens, lengths, prompt_lengths, repetition, frequency, presence,
                           bias_ids, bias_values, None if allowed is None else pack(allowed), mask,
                           out, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and y.dtype == x.dtype
    for i in range(n):
        if mask is not None and int(mask[i]) == 0:
            continue
        z = before[i].float().cpu().double().numpy()
        mag, ops = np.abs(z), np.zeros(v)
        if tokens is not None:
            row = tokens[i].cpu().numpy()
            end = row.size if lengths is None else int(lengths[i])
            first = 0 if prompt_lengths is None else int(prompt_lengths[i])
            seen = np.unique(row[:end][row[:end] >= 0])
            r, f, p = at(repetition, i), at(frequency, i), at(presence, i)
            z[seen] = np.where(z[seen] > 0, z[seen] / r, z[seen] * r)
            mag[seen] = np.abs(z[seen])
            drawn, c = np.unique(row[first:end][row[first:end] >= 0], return_counts=True)
            z[drawn] -= f * c + p
            mag[drawn] += np.abs(f * c) + abs(p)
            ops[seen] += 3
        if bias_ids is not None:
            ids, b = bias_ids[i].cpu().numpy(), bias_values[i].cpu().double().numpy()
            ids, b = ids[ids >= 0], b[ids >= 0]
            np.add.at(z, ids, b)
            np.add.at(mag, ids, np.abs(b))
            np.add.at(ops, ids, 2)
        if allowed is not None:
            z[~allowed[i].cpu().numpy()] = -np.inf
        got = y[i].float().cpu().double().numpy()
        plain = (ops == 0) & np.isfinite(z)
        assert same_bits(y[i][torch.from_numpy(plain)], before[i][torch.from_numpy(plain)])
        off = np.isinf(z)
        assert np.array_equal(got[off], z[off])
        on = (ops > 0) & ~off
        tol = ops * 2.0 ** -24 * mag
        if x.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (np.abs(z) + tol)
        assert np.all(np.abs(got - z)[on] <= tol[on])
    return y


def history(n, v, length, seed, holes=0.0):
    g = gen(seed)
    t = (v * torch.rand(n, length, generator=g) ** 3).long().clamp(max=v - 1)
    t[torch.rand(n, length, generator=g) < holes] = -1
    full = (torch.rand(n, generator=g) * (length + 1)).long().clamp(max=length)
    full[0] = length
    if n > 2:
        full[1], full[2] = 0, min(1, length)
    prompt = (full * torch.rand(n, generator=g)).long()
    prompt[-1] = full[-1]
    return t.to(dev()), full.to(dev()), prompt.to(dev())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("v", [1, 2, 7, 31, 32, 33, 255, 1000, 4097, 8191, 8192, 8193, 16400, 50021])
def test_vocabulary_sizes(v, dtype):
    n = 5
    t, full, prompt = history(n, v, 97, v, 0.1)
    g = gen(v + 1)
    ids = torch.randint(-1, v, (n, 9), generator=g).to(dev())
    vals = torch.randn(n, 9, generator=g).to(dev())
    allow = (torch.rand(n, v, generator=g) < 0.6).to(dev())
    x = logits(n, v, v + 2, dtype)
    check(x, t, full, prompt, 1.3, 0.4, -0.7)
    check(x, bias_ids=ids, bias_values=vals)
    check(x, allowed=allow)
    check(x, t, full, prompt, 0.8, -0.2, 0.5, ids, vals, allow)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad", [0, 1, 3, 8])
def test_strides_and_in_place(pad, dtype):
    n, v = 4, 9001
    t, full, prompt = history(n, v, 300, 3)
    allow = (torch.rand(n, v, generator=gen(4)) < 0.5).to(dev())
    x = logits(n, v, 5, dtype, pad)
    want = check(x, t, full, prompt, 1.2, 0.1, 0.3, allowed=allow)
    wide = torch.full((n, v + 5), 7.0, dtype=dtype, device=dev())
    got = check(x, t, full, prompt, 1.2, 0.1, 0.3, allowed=allow, out=wide[:, 2:v + 2])
    assert same_bits(got, want)
    assert bool((wide[:, :2] == 7.0).all()) and bool((wide[:, v + 2:] == 7.0).all())
    same = x.clone() if pad == 0 else x
    assert same_bits(check(same, t, full, prompt, 1.2, 0.1, 0.3, allowed=allow, out=same), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("length", [90, 4091, 4096, 9000])
def test_many_rows(length, dtype):
    # a copy and a launch for the listed columns: by hashing for short rows, in ranges for others
    n, v = 400, 70001
    t, full, prompt = history(n, v, length, length, 0.05)
    if length > 5000:
        full[7:390] %= 97
        prompt = torch.minimum(prompt, full)
    g = gen(length + 1)
    ids = torch.randint(-1, v, (n, 5), generator=g).to(dev())
    vals = torch.randn(n, 5, generator=g).to(dev())
    x = logits(n, v, 30, dtype)
    mask = (torch.arange(n) % 5 != 4).to(torch.uint8).to(dev())
    mask[10:380] = 0
    mask[100] = 1
    allow = (torch.rand(n, v, generator=g) < 0.5).to(dev())
    out = torch.full((n, v), 3.0, dtype=dtype, device=dev())
    want = check(x, t, full, prompt, 1.2, 0.3, -0.1, ids, vals, allow, mask, out)
    assert bool((want[mask == 0] == 3.0).all())
    same = x.clone()
    check(same, t, full, prompt, 1.2, 0.3, -0.1, ids, vals, allow, mask, same)
    assert same_bits(same[mask != 0], want[mask != 0]) and same_bits(same[mask == 0], x[mask == 0])
    # as each row by itself
    for i in (0, 1, 2, 3, 100, n - 1):
        if int(mask[i]):
            one = rlk.process_logits(x[i:i + 1].clone(), t[i:i + 1], full[i:i + 1],
                                     prompt[i:i + 1], 1.2, 0.3, -0.1, ids[i:i + 1],
                                     vals[i:i + 1], pack(allow[i:i + 1]))
            assert same_bits(one[0], want[i])
    again = rlk.process_logits(x, t, full, prompt, 1.2, 0.3, -0.1, ids, vals, None, mask)
    in_place = x.clone()
    rlk.process_logits(in_place, t, full, prompt, 1.2, 0.3, -0.1, ids, vals, None, mask, in_place)
    assert same_bits(in_place[mask != 0], again[mask != 0])


def test_a_row_that_cannot_be_among_many():
    n, v = 500, 60000
    x = logits(n, v, 31, torch.float32)
    t = torch.randint(0, v, (n, 50), generator=gen(32)).to(dev())
    full = torch.full((n,), 50, device=dev())
    t[3, 49], full[400] = v, 51
    for out in (None, x.clone()):
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        src = x if out is None else out
        y = rlk.process_logits(src, t, full, presence=1.0, out=out, error_word=err)
        assert int(err.item()) == rlk.RLK_DEVERR_TARGET_RANGE | rlk.RLK_DEVERR_SAMPLE_PARAM
        bad = torch.isnan(y).any(1)
        assert bad.nonzero()[:, 0].tolist() == [3, 400] and bool(torch.isnan(y[[3, 400]]).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_settings_of_each_row(dtype):
    n, v = 40, 3001
    t, full, prompt = history(n, v, 700, 6)
    g = gen(7)

    def pick(values):
        return torch.tensor(values)[torch.randint(len(values), (n,), generator=g)].to(dev())

    x = logits(n, v, 8, dtype)
    r, f, p = pick([1.0, 1.1, 2.0, 0.5]), pick([0.0, 0.3, -0.4]), pick([0.0, 1.0, -0.5])
    y = check(x, t, full, prompt, r, f, p)
    # a row's result is its own, whatever the batch
    for i in (0, 7, 39):
        one = check(x[i:i + 1].clone(), t[i:i + 1], full[i:i + 1], prompt[i:i + 1],
                    float(r[i]), float(f[i]), float(p[i]))
        assert same_bits(one[0], y[i])


def test_long_histories_and_repeats():
    v = 12000
    t = torch.zeros(3, 50000, dtype=torch.int64, device=dev())
    t[1] = 8191
    t[2] = torch.arange(50000, device=dev()) % v
    check(logits(3, v, 9, torch.float32), t, None, None, 1.1, 0.01, 0.2)
    check(logits(3, v, 10, torch.float32), t, None,
          torch.tensor([50000, 0, 25000], device=dev()), 1.1, 0.01, 0.2)


@pytest.mark.parametrize("b", [1, 2, 3, 64, 255, 256, 257, 300, 512, 513, 1025, 4096])
def test_numbers_of_biases(b):
    n, v = 3, 30011
    g = gen(b)
    ids = torch.randint(-1, v, (n, b), generator=g).to(dev())
    vals = torch.randn(n, b, generator=g).to(dev())
    t, full, prompt = history(n, v, 50, b + 1)
    for dtype in DTYPES:
        check(logits(n, v, b + 2, dtype), t, full, prompt, 1.1, 0.2, 0.1, ids, vals)


def test_many_biases_of_one_token():
    n, v = 2, 5000
    ids = torch.randint(0, 3, (n, 4096), generator=gen(11)).to(dev()) * 2000
    vals = torch.randn(n, 4096, generator=gen(12)).to(dev())
    x = logits(n, v, 13, torch.float32)
    a = check(x, bias_ids=ids, bias_values=vals)
    for _ in range(3):                                   # the sum's order is fixed
        assert same_bits(rlk.process_logits(x, bias_ids=ids, bias_values=vals), a)


def test_values_at_the_ends():
    x = torch.tensor([[0.0, -0.0, np.inf, -np.inf, np.nan, 3.0e38, -3.0e38, 1.0]], device=dev())
    t = torch.arange(8, device=dev())[None]
    y = rlk.process_logits(x, t, repetition=2.0)[0].cpu().numpy()
    assert y[0] == 0 and y[1] == 0 and y[2] == np.inf and y[3] == -np.inf and np.isnan(y[4])
    assert y[5] == np.float32(1.5e38) and y[6] == -np.inf and y[7] == 0.5
    none = torch.zeros(1, 1, dtype=torch.int32, device=dev())
    assert bool((rlk.process_logits(x, allowed=none) == -np.inf).all())
    lowest = torch.full((1, 8), torch.finfo(torch.float32).min, device=dev())
    assert same_bits(rlk.process_logits(lowest, t, frequency=0.0), lowest)
    ban = torch.full((1, 1), -np.inf, device=dev())
    y = rlk.process_logits(lowest, bias_ids=t[:, 3:4].clone(), bias_values=ban)
    assert y[0, 3] == -np.inf and bool((y[0, :3] > -np.inf).all())


def test_inactive_rows_are_left_as_they_are():
    n, v = 6, 2000
    x = logits(n, v, 14, torch.float32).clone()
    x[1], x[4] = np.nan, np.inf
    mask = torch.tensor([1, 0, 1, 1, 0, 1], dtype=torch.uint8, device=dev())
    t = torch.full((n, 3), 5, dtype=torch.int64, device=dev())
    t[1] = 1 << 40                                        # never looked at
    out = torch.full((n, v), 9.0, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    rlk.process_logits(x, t, presence=1.0, active_mask=mask, out=out, error_word=err)
    assert int(err.item()) == 0 and bool((out[1] == 9.0).all()) and bool((out[4] == 9.0).all())
    assert out[0, 5] == x[0, 5] - 1.0 and bool((out[0, 6:] == x[0, 6:]).all())


@pytest.mark.parametrize("kind", ["token", "bias", "length", "prompt", "negative", "repetition",
                                  "frequency", "presence"])
def test_rows_that_cannot_be(kind):
    n, v = 3, 20000
    x = logits(n, v, 15, torch.float32)
    t = torch.full((n, 4), 3, dtype=torch.int64, device=dev())
    full = torch.full((n,), 4, device=dev())
    prompt = torch.full((n,), 2, device=dev())
    ids, vals = t.clone(), torch.zeros(n, 4, device=dev())
    r, f, p = (torch.full((n,), w, device=dev()) for w in (1.0, 0.0, 0.0))
    flag = rlk.RLK_DEVERR_SAMPLE_PARAM
    if kind == "token":
        t[1, 3], flag = v, rlk.RLK_DEVERR_TARGET_RANGE
    elif kind == "bias":
        ids[1, 0], flag = 1 << 33, rlk.RLK_DEVERR_TARGET_RANGE
    elif kind == "length":
        full[1] = 5
    elif kind == "prompt":
        prompt[1] = 5
    elif kind == "negative":
        prompt[1] = -1
    elif kind == "repetition":
        r[1] = 0.0
    elif kind == "frequency":
        f[1] = np.nan
    else:
        p[1] = np.inf
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    y = rlk.process_logits(x, t, full, prompt, r, f, p, ids, vals, error_word=err)
    assert int(err.item()) == flag
    assert bool(torch.isnan(y[1]).all()) and same_bits(y[0], x[0]) and same_bits(y[2], x[2])


def test_no_tokens_yet():
    n, v = 3, 4000
    x = logits(n, v, 40, torch.float32)
    none = torch.empty(n, 0, dtype=torch.int64, device=dev())
    zero = torch.zeros(n, dtype=torch.int64, device=dev())
    assert same_bits(check(x, none, zero, zero, 1.5, 0.5, 0.5), x)
    assert same_bits(check(x, none, None, None, 1.5), x)
    one = zero.clone()
    one[1] = 1
    for out in (None, x.clone()):
        err = torch.zeros(1, dtype=torch.int32, device=dev())
        src = x if out is None else out
        y = rlk.process_logits(src, none, one, out=out, error_word=err)
        assert int(err.item()) == rlk.RLK_DEVERR_SAMPLE_PARAM
        assert bool(torch.isnan(y[1]).all()) and same_bits(y[0], x[0]) and same_bits(y[2], x[2])


@pytest.mark.parametrize("n", [8, 400])
def test_captured_with_the_draw(n):
    v = 30000
    x = logits(n, v, 16, torch.float32)
    t, full, prompt = history(n, v, 64, 17)
    u = torch.rand(n, generator=gen(18)).to(dev())
    y = torch.empty_like(x)
    ws = torch.empty(max(256, rlk.rlk_sample_logits_workspace_bytes(n, v)), dtype=torch.uint8,
                     device=dev())
    tok = torch.empty(n, dtype=torch.int64, device=dev())

    def step():
        rlk.rlk_process_logits(x, t, full, prompt, 1.2, 0.1, 0.1, None, None, None, None, y)
        rlk.rlk_sample_logits(y, u, None, 0.8, 0, 0.9, 0.0, tok, None, None, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (19, 20, 21):
        x.copy_(logits(n, v, seed, torch.float32))
        t.copy_(history(n, v, 64, seed + 30)[0])         # by the launch just before
        graph.replay()
        got = tok.clone()
        want = rlk.sample_logits(rlk.process_logits(x, t, full, prompt, 1.2, 0.1, 0.1), u, 0.8,
                                 top_p=0.9)[0]
        assert torch.equal(got, want)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_offsets_past_32_bits(dtype, many):
    # many: more than 152 ranges, so two launches, of rows that the mask leaves out but for four
    n, v = (200 if many else 4), 5003
    apart = (1 << 32) // n
    room = torch.empty((n - 1) * apart + v, dtype=dtype, device=dev())
    x = room.as_strided((n, v), (apart, 1))
    dense = logits(n, v, 62, dtype)
    x.copy_(dense)
    mask = torch.zeros(n, dtype=torch.uint8, device=dev())
    mask[[0, 1, n - 2, n - 1]] = 1
    t, full, prompt = history(n, v, 90, 63)
    want = rlk.process_logits(dense, t, full, prompt, 1.2, 0.1, 0.3, active_mask=mask)
    assert same_bits(rlk.process_logits(x, t, full, prompt, 1.2, 0.1, 0.3, active_mask=mask), want)
    rlk.process_logits(x, t, full, prompt, 1.2, 0.1, 0.3, active_mask=mask, out=x)
    assert same_bits(x[mask != 0], want[mask != 0]) and same_bits(x[mask == 0], dense[mask == 0])


def test_two_streams():
    calls = []
    for n, v, seed in ((300, 9001, 64), (40, 50021, 65)):
        x = logits(n, v, seed, torch.bfloat16)
        t, full, prompt = history(n, v, 200, seed)
        calls.append((x, t, full, prompt, 1.3, 0.2, 0.1))
    want = [rlk.process_logits(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(10):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(rlk.process_logits(*c))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert same_bits(y, want[i % 2])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,v,length", [(200, 8001, 90), (200, 8003, 700), (200, 40000, 20000),
                                        (170, 300001, 5000), (3, 60001, 50), (3, 60001, 3000),
                                        (160, 31, 40), (160, 33, 40)])
def test_listed_columns_few_and_many(n, v, length, dtype):
    # few and many rows, with few tokens for their columns (lists) and many (looks at each column),
    # counts past 14 bits, tables in parts; a copy, in place, and rows of other alignments
    t, full, prompt = history(n, v, length, v + length, 0.02)
    g = gen(length)
    ids = torch.randint(-1, v, (n, 3), generator=g).to(dev())
    vals = torch.randn(n, 3, generator=g).to(dev())
    if length > 16384:
        prompt[0], t[0, 1::2] = 0, 5                      # 5 is drawn often
        t[3] = 7
        full[3], prompt[3] = length, 1
    mask = torch.zeros(n, dtype=torch.uint8, device=dev())
    mask[[0, 1, 2, 3 % n, n // 2, n - 2, n - 1]] = 1
    allow = (torch.rand(n, v, generator=g) < 0.7).to(dev())
    for a in (None, allow):
        x = logits(n, v, 70, dtype, pad=3)
        want = check(x, t, full, prompt, 1.3, 0.2, 0.1, ids, vals, a, mask)
        same = x.clone()
        check(same, t, full, prompt, 1.3, 0.2, 0.1, ids, vals, a, mask, same)
        assert same_bits(same[mask != 0], want[mask != 0])
        assert same_bits(same[mask == 0], x[mask == 0])
