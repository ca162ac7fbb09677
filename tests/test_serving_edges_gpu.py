"""The serving operators where they could go wrong: many and empty sequences, tiles no
query of which sees a key, broadcast heads, long caches, graphs, streams that run at
once, repeated calls, and seeded random shapes.  Bounds as in test_serving_gpu.py."""
import math
import random

import pytest
import torch

import serving_plain as plain
from lut_attention_b200 import axr
from test_serving_gpu import (BF16, DEV, F16, F32, _cache, _check_evict, _check_prompt, _check_shared, _cu, _int32,
                              _prompt_inputs, _randn, _signs, _within)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _lib(axr_lib):
    return axr_lib


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 256), (F32, 64)])
@pytest.mark.parametrize("lens_q,lens_k", [([256], [100]), ([300, 130], [10, 131]), ([128, 129], [1, 128]),
                                           ([700], [401])])
def test_prompt_tiles_without_keys(dtype, d, lens_q, lens_k):
    """Fewer keys than queries: whole query tiles see none, their neighbours do."""
    cu_q, cu_k = _cu(lens_q), _cu(lens_k)
    q, K, V = _prompt_inputs(dtype, d, 2, 1, cu_q[-1], cu_k[-1], seed=d)
    out, lse = axr.axr_prompt_attention(q, K, V, _int32(cu_q), _int32(cu_k))
    _check_prompt(q, K, V, cu_q, cu_k, out, lse)
    first = lens_q[0] - lens_k[0]
    assert (out[:, :first] == 0).all() and (lse[:, :first] == -math.inf).all()


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64), (F16, 256)])
@pytest.mark.parametrize("batch", [31, 33, 90])
def test_prompt_many_sequences(dtype, d, batch):
    r = random.Random(batch)
    lens = [r.choice([0, 1, 5, 127, 128, 200, 300]) for _ in range(batch)]
    more = [n + r.choice([0, 0, 3, 140]) for n in lens]
    cu_q, cu_k = _cu(lens), _cu(more)
    q, K, V = _prompt_inputs(dtype, d, 1, 2, cu_q[-1], cu_k[-1], seed=batch)
    out, lse = axr.axr_prompt_attention(q, K, V, _int32(cu_q), _int32(cu_k))
    _check_prompt(q, K, V, cu_q, cu_k, out, lse)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (F16, 128)])
@pytest.mark.parametrize("group", [2, 3, 5, 6, 7, 8])
def test_prompt_even_and_odd_groups(dtype, d, group):
    """Even groups go two heads at a time, odd ones 256 queries at a time: sequences that
    end around 128 and 256, without keys, and with queries that see none."""
    lens_q, lens_k = [129, 1, 0, 257, 128, 300], [129, 600, 40, 257, 0, 45]
    cu_q, cu_k = _cu(lens_q), _cu(lens_k)
    q, K, V = _prompt_inputs(dtype, d, 2, group, cu_q[-1], cu_k[-1], seed=group)
    out, lse = axr.axr_prompt_attention(q, K, V, _int32(cu_q), _int32(cu_k))
    _check_prompt(q, K, V, cu_q, cu_k, out, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_broadcast_heads_and_no_keys(dtype):
    q, K, V = _prompt_inputs(dtype, 128, 3, 2, 140, 140, seed=2)
    K1, V1 = K[:1].expand(3, -1, -1), V[:1].expand(3, -1, -1)                # head stride 0
    out, lse = axr.axr_prompt_attention(q, K1, V1, _int32([0, 140]))
    _check_prompt(q, K1, V1, [0, 140], [0, 140], out, lse)
    none = K[:, :0]
    out, lse = axr.axr_prompt_attention(q, none, none, _int32([0, 140]), _int32([0, 0]))
    assert (out == 0).all() and (lse == -math.inf).all()
    assert axr.axr_prompt_attention(q[:, :0], K, V, _int32([0, 0]), _int32([0, 140]))[0].numel() == 0


def test_prompt_starts_out_of_order_stay_inside():
    """Starts that are wrong (decreasing, negative, past the end) give undefined rows but
    touch nothing outside: guard rows around out and lse keep their values."""
    q, K, V = _prompt_inputs(BF16, 128, 1, 2, 300, 300, seed=3, token_major=False)
    for cu in ([0, 500, 20, 300], [-7, 100, 1 << 30, 300], [300, 0, 0, 300]):
        wide = torch.full((2 * 300 + 64, 128), 9.0, dtype=BF16, device=DEV)
        out = wide[32:-32].view(2, 300, 128)
        guard = torch.full((2 * 300 + 64,), 9.0, device=DEV)
        axr.axr_prompt_attention(q, K, V, _int32(cu), out=out, lse=guard[32:-32].view(2, 300))
        torch.cuda.synchronize()
        assert (wide[:32] == 9).all() and (wide[-32:] == 9).all() and (guard[:32] == 9).all() and (guard[-32:] == 9).all()
        assert axr.axr_device_status() == 0


def test_prompt_and_shared_on_two_streams_at_once():
    q, K, V = _prompt_inputs(BF16, 128, 4, 4, 1500, 1500, seed=5)
    cu = _int32([0, 700, 1500])
    pre, own = _cache(4, 9000, 128, 4, BF16, seed=1), _cache(16, 300, 128, 4, BF16, seed=2)
    qs, lens, signs = _randn((64, 128), 3, BF16), _int32([300, 0, 7, 129]), _signs(128)
    want = axr.axr_prompt_attention(q, K, V, cu)[0], axr.axr_attention_shared(qs, *pre, *own, lens, 4, 4, signs)[0]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append((i, axr.axr_prompt_attention(q, K, V, cu)[0] if i == 0
                            else axr.axr_attention_shared(qs, *pre, *own, lens, 4, 4, signs)[0]))
    torch.cuda.synchronize()
    for i, x in got:
        assert torch.equal(x, want[0] if i == 0 else want[1])
    assert axr.axr_device_status() == 0


def test_prompt_repeats_bit_for_bit():
    for dtype, d in ((BF16, 128), (F16, 64), (F16, 256)):
        q, K, V = _prompt_inputs(dtype, d, 2, 3, 2300, 2300, seed=5)
        cu = _int32([0, 900, 901, 2300])
        ref, rl = axr.axr_prompt_attention(q, K, V, cu)
        for _ in range(10):
            out, lse = axr.axr_prompt_attention(q, K, V, cu)
            assert torch.equal(out, ref) and torch.equal(lse, rl)
    assert axr.axr_device_status() == 0


@pytest.mark.parametrize("vdtype", [BF16, F32])
def test_shared_many_sequences(vdtype):
    """More sequences than the kernel keeps in shared memory, one query each."""
    batch, d, b = 300, 64, 2
    r = random.Random(1)
    lens = [r.choice([0, 0, 1, 40, 129]) for _ in range(batch)]
    pre, own = _cache(1, 200, d, b, vdtype, seed=1), _cache(batch, 130, d, b, vdtype, seed=2)
    q = _randn((batch, d), 3, F16)
    out, lse = axr.axr_attention_shared(q, *pre, *own, _int32(lens), 1, b, _signs(d))
    _check_shared(q, pre, own, lens, 1, b, _signs(d), out, lse)


@pytest.mark.parametrize("vdtype,d", [(BF16, 128), (F16, 64), (F32, 32)])
def test_shared_without_any_keys(vdtype, d):
    pre, own = _cache(2, 0, d, 4, vdtype, seed=1), _cache(6, 5, d, 4, vdtype, seed=2)
    q = _randn((6, d), 3, F32)
    out, lse = axr.axr_attention_shared(q, *pre, *own, _int32([0, 5, 0]), 1, 4, _signs(d))
    _check_shared(q, pre, own, [0, 5, 0], 1, 4, _signs(d), out, lse)
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all()
    empty = [t[:, :0].contiguous() for t in own]
    out, lse = axr.axr_attention_shared(q, *pre, *empty, _int32([0, 0, 0]), 1, 4, _signs(d))
    assert (out == 0).all() and (lse == -math.inf).all() and axr.axr_device_status() == 0


def test_shared_zero_and_extreme_queries_and_norms():
    d, b = 128, 4
    pre, own = _cache(1, 400, d, b, BF16, seed=1), _cache(3, 50, d, b, BF16, seed=2)
    pre[1][0, ::3] = 0.0
    q = _randn((6, d), 3, F32)
    q[0] = 0.0
    q[2] *= 1e-30
    q[3] *= 50.0
    q[4, 1:] = 0.0
    out, lse = axr.axr_attention_shared(q, *pre, *own, _int32([50, 0, 17]), 2, b, _signs(d))
    _check_shared(q, pre, own, [50, 0, 17], 2, b, _signs(d), out, lse)


def test_shared_weights_and_evict_past_32_bit_offsets():
    """A head of 2^24 + 5 rows: its values pass 2^32 bytes and 2^31 elements.  All norms
    but those of the last rows are 0, so the other keys score 0 with values of 0."""
    n, tail, group, d, b = (1 << 24) + 5, 300, 4, 128, 4
    idx = torch.zeros((1, n, d * b // 8), dtype=torch.uint8, device=DEV)
    norms = torch.zeros((1, n), device=DEV)
    V = torch.zeros((1, n, d), dtype=BF16, device=DEV)
    last = _cache(1, tail, d, b, BF16, seed=9)
    for whole, part in zip((idx, norms, V), last):
        whole[:, n - tail:] = part
    norms[:, n - tail:] += 30.0
    small = [t[:, n - tail:] for t in (idx, norms, V)]
    q, signs = _randn((group, d), 10, BF16), _signs(d)
    empty = [t[:, :0].contiguous() for t in small]

    # a: the long head as the prefix; b: as a sequence's own cache
    cent = torch.from_numpy(axr.axr_make_codebook(d, b)[0]).to(DEV)
    want, lse_t, tol, tol_lse = plain.shared(q, [t.contiguous() for t in small], empty, [0], group, b, signs, cent, 2.0 ** -8,
                                       3 * 2.0 ** -22)
    lse = torch.logaddexp(lse_t, torch.full_like(lse_t, math.log(n - tail)))     # n - tail keys of score 0
    shrink = torch.exp(lse_t - lse)[:, None]
    A = last[2].double().abs().amax(1)                                           # |V| bound of the weighted sums
    # a CTA of at least 100 adds up at most n / 100 weights, rounding 2^-24 each, and 1000 more in the merge
    sums = (n / 100 + 1000) * 2.0 ** -24
    for pre, own, length in (((idx, norms, V), empty, 0), (empty, (idx, norms, V), n)):
        out, got = axr.axr_attention_shared(q, *pre, *own, _int32([length]), group, b, signs)
        _within(out, want * shrink, (tol + 2 * sums * A) * shrink, "out")
        _within(got, lse, tol_lse + sums + 2.0 ** -20, "lse")

    # the weights of a step that looks at the head's ends, then the choice by them
    scores = torch.full((group, n), -30.0, device=DEV)
    scores[:, :50] = 3.0
    scores[:, n - tail:n - 200] = 2.0
    w = torch.zeros((1, n), device=DEV)
    axr.axr_accumulate_weights(scores, w, group)
    total = 50 * math.exp(3.0) + 100 * math.exp(2.0) + (n - 150) * math.exp(-30.0)
    # a thread adds up n / 4096 weights, exponents up to 33 round by 33 2^-23: below 2^-11
    for part, x in ((w[0, :50], 3.0), (w[0, n - tail:n - 200], 2.0)):
        assert ((part.double() * total / (group * math.exp(x)) - 1).abs() <= 2.0 ** -11).all()
    got = axr.axr_evict(idx, norms, V, w, _int32([n]), 250, 100)
    rows = list(range(50)) + list(range(n - tail, n - 200)) + list(range(n - 100, n))
    assert got[4][0].tolist() == rows
    at = torch.tensor(rows, device=DEV)
    assert torch.equal(got[0][0], idx[0, at]) and torch.equal(got[1][0], norms[0, at]) and torch.equal(got[2][0], V[0, at])
    assert axr.axr_device_status() == 0


@pytest.mark.parametrize("n,keep", [(8191, 100), (8193, 4000), (250001, 1000), (250001, 200000)])
def test_evict_long_caches(n, keep):
    cache = _cache(1, n, 32, 1, F16, seed=4)
    w = torch.round(_randn((1, n), 5).abs() * 256) / 256
    got = axr.axr_evict(*cache, w, _int32([n]), keep, 50)
    _check_evict(cache, w, [n], keep, 50, got)


def test_weights_and_evict_in_a_graph():
    heads, group, n, keep = 3, 4, 3000, 500
    cache = _cache(heads, n, 64, 4, BF16, seed=4)
    scores, sums = _randn((heads * group, n), 1), torch.zeros((heads, n), device=DEV)
    lens = _int32([n, 2000, 400])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = axr.axr_evict(*cache, sums, lens, keep, 20)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            axr.axr_accumulate_weights(scores, sums, group, lengths=lens)
            axr.axr_evict(*cache, sums, lens, keep, 20, out=out)
    torch.cuda.synchronize()
    for seed, ms in ((7, [n, 2000, 400]), (8, [10, 2999, 0])):
        lens.copy_(_int32(ms))
        scores.copy_(_randn(scores.shape, seed))
        sums.zero_()
        g.replay()
        torch.cuda.synchronize()
        want, tol = plain.weights(scores, torch.zeros_like(sums), group, ms)
        _within(sums, want, tol, "weights")
        _check_evict(cache, sums, ms, keep, 20, out)


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    r = random.Random(1000 + seed)
    dtype, d = r.choice([(BF16, 128), (F16, 64), (F16, 128), (BF16, 256), (F32, 64), (BF16, 64)])
    heads, group, batch = r.randint(1, 4), r.randint(1, 8), r.randint(1, 9)
    lens = [r.choice([0, 1, r.randint(2, 130), r.randint(100, 900)]) for _ in range(batch)]
    more = [max(0, n + r.choice([0, 0, r.randint(-60, 300)])) for n in lens]
    cu_q, cu_k = _cu(lens, r.randint(0, 3)), _cu(more, r.randint(0, 3))
    q, K, V = _prompt_inputs(dtype, d, heads, group, cu_q[-1] + r.randint(0, 9), cu_k[-1] + r.randint(0, 9) + 1,
                             seed=seed, token_major=r.random() < 0.5)
    out, lse = axr.axr_prompt_attention(q, K, V, _int32(cu_q), _int32(cu_k))
    _check_prompt(q, K, V, cu_q, cu_k, out, lse)
    d, b, n = r.choice([64, 128]), r.randint(1, 4), r.choice([0, 1, r.randint(2, 300), r.randint(300, 5000)])
    own_lens = [r.choice([0, 1, r.randint(0, 300)]) for _ in range(batch)]
    pre, own = _cache(heads, n, d, b, dtype, seed), _cache(batch * heads, max(own_lens) + r.randint(0, 5), d, b, dtype, seed + 1)
    qs = _randn((batch * heads * group, d), seed, r.choice([F32, F16, BF16]))
    out, lse = axr.axr_attention_shared(qs, *pre, *own, _int32(own_lens), group, b, _signs(d))
    _check_shared(qs, pre, own, own_lens, group, b, _signs(d), out, lse)
