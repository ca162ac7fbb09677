"""The serving operators on the GPU against plain 64-bit forms: prompt attention,
decode over a shared prefix, accumulated weights, eviction, and a run of them
together.  Bounds are derived in serving_plain.py."""
import math

import pytest
import torch

import serving_plain as plain
from lut_attention_b200 import axr, workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _lib(axr_lib):
    return axr_lib


def _randn(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device=DEV)).to(dtype)


def _cu(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _within(got, want, tol, what):
    got = got.double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= tol))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst " \
                          f"{float(((got - want).abs() / tol.clamp(min=1e-300))[bad].max()):.3g} times the bound"


# ---- prompt attention ----------------------------------------------------------

def _prompt_inputs(dtype, d, heads, group, nq, nk, seed, token_major=True):
    q, K, V = (_randn((n, h, d) if token_major else (h, n, d), seed + i, dtype, s)
               for i, (n, h, s) in enumerate(((nq, heads * group, 1.0), (nk, heads, 1.5), (nk, heads, 1.0))))
    return [t.transpose(0, 1) for t in (q, K, V)] if token_major else [q, K, V]


def _u_weights(dtype):
    """Weights are rounded to 16-bit types where the tensor cores take them."""
    return 0.0 if dtype == F32 else plain.U[dtype]


def _check_prompt(q, K, V, cu_q, cu_k, got, got_lse):
    want, lse, tol, tol_lse = plain.prompt(q, K, V, cu_q, cu_k, _u_weights(q.dtype))
    rows = torch.zeros(q.shape[1], dtype=torch.bool, device=DEV)
    for a, z in zip(cu_q, cu_q[1:]):
        rows[a:z] = True
    _within(got[:, rows], want[:, rows], tol[:, rows], "out")
    _within(got_lse[:, rows], lse[:, rows], tol_lse[:, rows], "lse")
    assert axr.axr_device_status() == 0


LENS = [([1], [1]), ([5, 1, 0, 70], [5, 1, 0, 70]), ([63, 64, 65], [63, 64, 65]),
        ([127, 128, 129, 1], [127, 128, 129, 1]), ([255, 256, 257], [255, 256, 257]),
        ([1, 40, 200], [300, 128, 513]), ([130, 9, 3], [7, 0, 2]), ([385, 0, 640], [1025, 12, 640])]


@pytest.mark.parametrize("lens_q,lens_k", LENS)
@pytest.mark.parametrize("dtype,d,heads,group", [(BF16, 128, 2, 4), (F16, 64, 3, 1), (F32, 64, 1, 2), (F16, 256, 1, 3),
                                                 (BF16, 64, 1, 8)])
def test_prompt_lengths(dtype, d, heads, group, lens_q, lens_k):
    cu_q, cu_k = _cu(lens_q), _cu(lens_k)
    q, K, V = _prompt_inputs(dtype, d, heads, group, cu_q[-1], cu_k[-1], seed=d + group)
    out, lse = axr.axr_prompt_attention(q, K, V, _int32(cu_q), _int32(cu_k))
    _check_prompt(q, K, V, cu_q, cu_k, out, lse)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("d", [32, 64, 128, 256, 512])
def test_prompt_types_and_widths(dtype, d):
    cu = _cu([190, 33])
    q, K, V = _prompt_inputs(dtype, d, 2, 2, cu[-1], cu[-1], seed=d, token_major=False)
    out, lse = axr.axr_prompt_attention(q, K, V, _int32(cu))
    _check_prompt(q, K, V, cu, cu, out, lse)


def test_prompt_long_and_grouped():
    cu = _cu([2500, 1300])
    q, K, V = _prompt_inputs(BF16, 128, 2, 5, cu[-1], cu[-1], seed=5)
    out, lse = axr.axr_prompt_attention(q, K, V, _int32(cu))
    _check_prompt(q, K, V, cu, cu, out, lse)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64), (F16, 256), (F32, 64), (BF16, 32)])
def test_prompt_leaves_other_rows_and_ignores_their_values(dtype, d):
    """Rows before the first and behind the last sequence: outputs as they were, and
    NaN in them (or in a neighbour's keys and values) reaches no other sequence."""
    cu_q, cu_k = [3, 40, 40, 170], [9, 60, 60, 200]
    q, K, V = _prompt_inputs(dtype, d, 2, 2, 180, 230, seed=11)
    dirty = [t.clone() for t in (q, K, V)]
    dirty[0][:, 170:] = math.nan
    dirty[0][:, :3] = math.nan
    for t in dirty[1:]:
        t[:, :9] = math.nan
        t[:, 200:] = math.inf
    out = torch.full_like(q, 7.0)
    lse = torch.full((4, 180), 5.0, device=DEV)
    axr.axr_prompt_attention(*dirty, _int32(cu_q), _int32(cu_k), out=out, lse=lse)
    _check_prompt(q, K, V, cu_q, cu_k, out, lse)
    for part in (slice(0, 3), slice(170, 180)):
        assert (out[:, part] == 7.0).all() and (lse[:, part] == 5.0).all()
    dirty[1][:, 60:] = math.nan               # the second sequence's keys and values
    dirty[2][:, 60:] = math.nan
    out2, lse2 = axr.axr_prompt_attention(*dirty, _int32(cu_q), _int32(cu_k))
    assert torch.equal(out2[:, 3:40], out[:, 3:40]) and torch.equal(lse2[:, 3:40], lse[:, 3:40])


def test_prompt_extreme_scores():
    """Scores of hundreds: one key takes all the weight; equal scores share it."""
    q, K, V = _prompt_inputs(BF16, 128, 1, 2, 300, 300, seed=13)
    K = (K * 60).contiguous()
    out, lse = axr.axr_prompt_attention(q, K, V, _int32([0, 300]))
    _check_prompt(q, K, V, [0, 300], [0, 300], out, lse)
    K.zero_()
    out, lse = axr.axr_prompt_attention(q, K, V, _int32([0, 300]))
    _check_prompt(q, K, V, [0, 300], [0, 300], out, lse)


def test_prompt_offsets_past_32_bits():
    """Head strides of 2^31 elements (4 GB): the second head lies past 32-bit offsets."""
    d, n, step = 64, 70, 1 << 31
    big = torch.empty(step + n * d, dtype=BF16, device=DEV)
    q = torch.as_strided(big, (2, n, d), (step, d, 1))
    q.copy_(_randn((2, n, d), 3, BF16))
    K = _randn((2, n, d), 4, BF16)
    V = _randn((2, n, d), 5, BF16)
    for args in ((q, K, V), (q, q, q)):
        out, lse = axr.axr_prompt_attention(*args, _int32([0, n]), out=torch.empty((2, n, d), dtype=BF16, device=DEV))
        _check_prompt(*args, [0, n], [0, n], out, lse)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_prompt_in_a_graph_with_new_lengths(dtype, d):
    q, K, V = _prompt_inputs(dtype, d, 2, 2, 400, 400, seed=17)
    cu = _int32([0, 100, 400])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        axr.axr_prompt_attention(q, K, V, cu)
        out, lse = torch.empty_like(q), torch.empty((4, 400), device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            axr.axr_prompt_attention(q, K, V, cu, out=out, lse=lse)
    torch.cuda.synchronize()
    for lens in ([0, 100, 400], [0, 333, 400], [0, 0, 400]):
        cu.copy_(_int32(lens))
        out.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        _check_prompt(q, K, V, lens, lens, out, lse)


# ---- decode over a shared prefix -------------------------------------------------

def _cache(heads, n, d, b, vdtype, seed):
    idx, norms = workloads.make_random_packed(heads, n, d, b, seed=seed, device=DEV)
    return idx, norms.clamp(max=4.0), _randn((heads, n, d), seed + 7, vdtype)


def _signs(d):
    return workloads.make_signs(workloads.GQA_DECODE_128K.with_(d=d)).to(DEV)


def _u_cent(vdtype, d):
    """For 16-bit values queries and centroids are pairs of fp16 parts: 2^-22 each, and
    the product of the two low parts, left out, another 2^-22."""
    return 0.0 if vdtype == F32 else 3 * 2.0 ** -22


def _check_shared(q, pre, own, lengths, group, b, signs, out, lse):
    d = q.shape[1]
    cent = torch.from_numpy(axr.axr_make_codebook(d, b)[0]).to(DEV)
    want, wl, tol, tol_lse = plain.shared(q, pre, own, lengths, group, b, signs, cent, _u_weights(pre[2].dtype),
                                          _u_cent(pre[2].dtype, d))
    _within(out, want, tol, "out")
    _within(lse, wl, tol_lse, "lse")
    assert axr.axr_device_status() == 0


SHARED = [
    # heads, group, prefix keys, own lengths
    (2, 4, 300, [5, 0, 40]), (1, 1, 1, [1]), (2, 8, 127, [128, 129, 0, 127]), (3, 3, 0, [7, 0, 200]),
    (2, 4, 1000, [0, 0]), (1, 4, 128, [0] * 33), (2, 2, 1537, [3] * 70), (1, 8, 700, list(range(0, 300, 17))),
    (1, 5, 4000, [1000, 1]),
]


@pytest.mark.parametrize("heads,group,n,lengths", SHARED)
@pytest.mark.parametrize("vdtype,d,b", [(BF16, 128, 4), (F16, 128, 3), (BF16, 64, 2), (F32, 64, 4), (F16, 64, 1)])
def test_shared_shapes(vdtype, d, b, heads, group, n, lengths):
    batch = len(lengths)
    pre = _cache(heads, n, d, b, vdtype, seed=n + d)
    own = _cache(batch * heads, max(lengths) + 3, d, b, vdtype, seed=n + 1)
    q = _randn((batch * heads * group, d), 3 * n + d, BF16 if vdtype == BF16 else F16)
    out, lse = axr.axr_attention_shared(q, *pre, *own, _int32(lengths), group, b, _signs(d))
    assert out.dtype == vdtype
    _check_shared(q, pre, own, lengths, group, b, _signs(d), out, lse)


@pytest.mark.parametrize("d,b,vdtype,qdtype", [(32, 3, BF16, F32), (256, 2, F16, F16), (512, 4, F32, BF16),
                                               (128, 1, BF16, F32), (256, 3, BF16, BF16), (128, 2, F32, F16)])
def test_shared_widths_and_types(d, b, vdtype, qdtype):
    heads, group, lengths = 2, 3, [0, 140, 12]
    pre, own = _cache(heads, 333, d, b, vdtype, seed=d), _cache(6, 150, d, b, vdtype, seed=d + 1)
    q = _randn((18, d), d, qdtype)
    out, lse = axr.axr_attention_shared(q, *pre, *own, _int32(lengths), group, b, _signs(d))
    _check_shared(q, pre, own, lengths, group, b, _signs(d), out, lse)


def test_shared_long_prefix():
    heads, group, lengths, d, b = 2, 4, [700, 0, 33, 1], 128, 4
    pre, own = _cache(heads, 70001, d, b, BF16, seed=1), _cache(8, 704, d, b, BF16, seed=2)
    q = _randn((32, d), 3, BF16)
    out, lse = axr.axr_attention_shared(q, *pre, *own, _int32(lengths), group, b, _signs(d))
    _check_shared(q, pre, own, lengths, group, b, _signs(d), out, lse)


def test_shared_prefix_alone_is_the_decode_attention():
    """One sequence without own keys: what axr_attention gives, up to its fp32 output."""
    heads, group, d, b = 3, 4, 128, 4
    pre = _cache(heads, 3000, d, b, BF16, seed=5)
    q = _randn((heads * group, d), 6, BF16)
    empty = (pre[0][:, :0], pre[1][:, :0], pre[2][:, :0])
    out, _ = axr.axr_attention_shared(q, *pre, *[t.contiguous() for t in empty], _int32([0]), group, b, _signs(d))
    want, _ = axr.axr_attention(q, *pre, group, b, _signs(d))
    # the two differ by the roundings of the weights and of out (u each)
    p_abs = pre[2].float().abs().amax(1).repeat_interleave(group, 0)
    assert ((out.float() - want).abs() <= 4 * plain.U[BF16] * p_abs).all()


@pytest.mark.parametrize("vdtype,d", [(BF16, 128), (F16, 64), (F32, 64)])
def test_shared_ignores_rows_past_the_lengths(vdtype, d):
    """Unused rows of the own caches may hold anything, NaN and infinities too; lengths
    outside [0, capacity] are clamped."""
    heads, group, b, lengths = 2, 2, 4, [5, 130, 0]
    pre, own = _cache(heads, 200, d, b, vdtype, seed=1), _cache(6, 140, d, b, vdtype, seed=2)
    q = _randn((12, d), 3, F16)
    ref, ref_lse = axr.axr_attention_shared(q, *pre, *own, _int32(lengths), group, b, _signs(d))
    for s, m in enumerate(lengths):
        for h in range(heads):
            own[0][s * heads + h, m:] = 255
            own[1][s * heads + h, m:] = math.nan
            own[2][s * heads + h, m:] = math.inf if h else math.nan
    out, lse = axr.axr_attention_shared(q, *pre, *own, _int32(lengths), group, b, _signs(d))
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    own = _cache(6, 140, d, b, vdtype, seed=2)
    ref, _ = axr.axr_attention_shared(q, *pre, *own, _int32([140, 0, 3]), group, b, _signs(d))
    out, _ = axr.axr_attention_shared(q, *pre, *own, _int32([1 << 30, -5, 3]), group, b, _signs(d))
    assert torch.equal(out, ref)
    assert axr.axr_device_status() == 0


def test_shared_workspace_stream_and_graph():
    """A used workspace on a side stream, and a replayed graph whose lengths and keys change."""
    heads, group, d, b, lengths = 2, 4, 128, 4, [100, 0, 259]
    pre, own = _cache(heads, 900, d, b, BF16, seed=1), _cache(6, 260, d, b, BF16, seed=2)
    q = _randn((24, d), 3, BF16)
    lens = _int32(lengths)
    ref, _ = axr.axr_attention_shared(q, *pre, *own, lens, group, b, _signs(d))
    need = axr.axr_attention_shared_workspace_bytes(3, heads, group, d)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(ref), torch.empty(24, device=DEV)
    side, signs = torch.cuda.Stream(), _signs(d)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        axr.axr_attention_shared(q, *pre, *own, lens, group, b, signs, workspace=ws, out=out, lse=lse, stream=side)
        side.synchronize()
        assert torch.equal(out, ref)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            axr.axr_attention_shared(q, *pre, *own, lens, group, b, signs, workspace=ws, out=out, lse=lse)
    for new in ([100, 0, 259], [0, 0, 0], [260, 1, 2]):
        lens.copy_(_int32(new))
        own[2].copy_(_randn(own[2].shape, sum(new) + 9, BF16))
        g.replay()
        torch.cuda.synchronize()
        _check_shared(q, pre, own, new, group, b, signs, out, lse)


def test_shared_repeats_bit_for_bit():
    heads, group, d, b, lengths = 8, 4, 128, 4, [100, 700, 259, 31]
    pre, own = _cache(heads, 5000, d, b, BF16, seed=1), _cache(32, 700, d, b, BF16, seed=2)
    q = _randn((128, d), 3, BF16)
    ref, rl = axr.axr_attention_shared(q, *pre, *own, _int32(lengths), group, b, _signs(d))
    for _ in range(5):
        out, lse = axr.axr_attention_shared(q, *pre, *own, _int32(lengths), group, b, _signs(d))
        assert torch.equal(out, ref) and torch.equal(lse, rl)


# ---- accumulated weights ---------------------------------------------------------

@pytest.mark.parametrize("heads,group,n,capacity", [(1, 1, 1, 1), (3, 4, 7, 9), (2, 8, 1000, 1000), (5, 3, 4097, 5000),
                                                    (1, 2, 100003, 100003), (40, 4, 513, 600)])
@pytest.mark.parametrize("ragged", [False, True])
def test_weights(heads, group, n, capacity, ragged):
    scores = _randn((heads * group, n), n + group, scale=3.0)
    start = torch.rand((heads, capacity), device=DEV)
    lens = [(h * 7919) % (n + 1) for h in range(heads)] if ragged else [n] * heads
    want, tol = plain.weights(scores, start, group, lens)
    got = axr.axr_accumulate_weights(scores, start.clone(), group, lengths=_int32(lens) if ragged else None)
    _within(got, want, tol, "weights")
    for h, m in enumerate(lens):
        assert torch.equal(got[h, m:], start[h, m:])


def test_weights_masked_scores():
    """-inf scores weigh nothing, rows of them add nothing, the lowest finite value is
    a score like others, and a NaN stays in its own head."""
    scores = _randn((8, 300), 3)
    scores[0, :250] = -math.inf
    scores[1] = -math.inf
    scores[2, 5:] = torch.finfo(F32).min
    scores[3] = torch.finfo(F32).min
    start = torch.zeros((2, 300), device=DEV)
    want, tol = plain.weights(scores, start, 4, [300, 300])
    got = axr.axr_accumulate_weights(scores, start.clone(), 4)
    _within(got, want, tol, "weights")
    scores[1, 7] = math.nan
    bad = axr.axr_accumulate_weights(scores, start.clone(), 4)
    assert bad[0].isnan().all() and torch.equal(bad[1], got[1])


# ---- eviction --------------------------------------------------------------------

def _check_evict(cache, weights, lens, keep, recent, got):
    idx, norms, V, w, kept, new = got
    for h, m in enumerate(lens):
        m = min(max(m, 0), weights.shape[1])
        stay = plain.evict(weights[h, :m].tolist(), m, keep, recent)
        n = len(stay)
        assert kept[h, :n].tolist() == stay and (kept[h, n:] == -1).all() and int(new[h]) == n, (h, m)
        for src, to in zip((*cache, weights), (idx, norms, V, w)):
            assert torch.equal(to[h, :n].view(torch.uint8), src[h, stay].contiguous().view(torch.uint8))


@pytest.mark.parametrize("heads,n,keep,recent", [(1, 1, 1, 0), (2, 5, 3, 1), (3, 700, 256, 64), (2, 700, 64, 64),
                                                 (2, 700, 699, 0), (4, 9000, 1024, 100), (1, 40000, 37000, 5),
                                                 (2, 33, 100, 50), (9, 4097, 1, 0), (9, 4097, 1, 1)])
@pytest.mark.parametrize("d,b,vdtype", [(128, 4, BF16), (64, 3, F32), (8, 1, F16)])
def test_evict(heads, n, keep, recent, d, b, vdtype):
    cache = _cache(heads, n, d, b, vdtype, seed=n)
    weights = torch.round(_randn((heads, n), n + 1).abs() * 64) / 64        # many equal
    lens = [n if h % 2 == 0 else (n * 2) // 3 for h in range(heads)]
    got = axr.axr_evict(*cache, weights, _int32(lens), keep, recent)
    _check_evict(cache, weights, lens, keep, recent, got)


@pytest.mark.parametrize("what", ["equal", "signed", "special", "descending"])
def test_evict_orders(what):
    heads, n, keep, recent, d, b = 2, 3001, 700, 30, 64, 2
    cache = _cache(heads, n, d, b, BF16, seed=4)
    w = _randn((heads, n), 9)
    if what == "equal":
        w.fill_(0.25)
    if what == "special":
        w[0, ::3], w[0, 1::5], w[0, 2::7], w[0, 3::11] = math.nan, math.inf, -math.inf, -0.0
        w[1] = 0.0
        w[1, ::2] = -0.0                                       # equal to 0
    if what == "descending":
        w = torch.arange(n, 0, -1, device=DEV).float().repeat(heads, 1) * 1e-42      # subnormal
    lens = [n, n - 1]
    got = axr.axr_evict(*cache, w, _int32(lens), keep, recent)
    _check_evict(cache, w, lens, keep, recent, got)


def test_evict_into_a_larger_cache_leaves_the_rest():
    heads, n, keep, recent, d, b = 3, 500, 200, 20, 128, 4
    cache = _cache(heads, n, d, b, BF16, seed=4)
    w = torch.rand((heads, n), device=DEV)
    out = (torch.full((heads, 260, 64), 77, dtype=torch.uint8, device=DEV), torch.full((heads, 260), 7.0, device=DEV),
           torch.full((heads, 260, d), 7.0, dtype=BF16, device=DEV), torch.full((heads, 260), 7.0, device=DEV),
           torch.empty((heads, keep), dtype=torch.int32, device=DEV), torch.empty(heads, dtype=torch.int32, device=DEV))
    lens = [500, 150, -3]
    axr.axr_evict(*cache, w, _int32([500, 150, -3]), keep, recent, out=out)
    _check_evict(cache, w, lens, keep, recent, out)
    for h, m in enumerate([200, 150, 0]):
        assert all((t[h, m:] == (77 if t.dtype == torch.uint8 else 7.0)).all() for t in out[:4])


# ---- together --------------------------------------------------------------------

def test_serving_run():
    """A prompt is attended to and its keys written; three sequences then decode on it as
    a shared prefix, each appending its key, and one head's cache is shrunk by the weights
    that its steps gathered, and scored on."""
    heads, group, d, b, n, batch, steps = 2, 4, 128, 4, 700, 3, 5
    signs = _signs(d)
    q, K, V = _prompt_inputs(BF16, d, heads, group, n, n, seed=23, token_major=False)
    out, lse = axr.axr_prompt_attention(q, K, V, _int32([0, n]))
    _check_prompt(q, K, V, [0, n], [0, n], out, lse)
    idx, norms = axr.axr_quantize_keys(K, b, signs)
    cap = 16
    own = (torch.zeros((batch * heads, cap, d * b // 8), dtype=torch.uint8, device=DEV),
           torch.zeros((batch * heads, cap), device=DEV), torch.zeros((batch * heads, cap, d), dtype=BF16, device=DEV))
    for step in range(steps):
        k_new, v_new = _randn((batch * heads, d), 50 + step, BF16), _randn((batch * heads, d), 90 + step, BF16)
        qs = _randn((batch * heads * group, d), 70 + step, BF16)
        axr.axr_append_scores(k_new, qs, own[0], own[1], step, group, b, signs)
        own[2][:, step] = v_new
        lens = [step + 1] * batch
        got, lse = axr.axr_attention_shared(qs, idx, norms, V, *own, _int32(lens), group, b, signs)
        _check_shared(qs, (idx, norms, V), own, lens, group, b, signs, got, lse)
    # the prompt's own cache, shrunk by what a few queries weighed
    sums = torch.zeros((heads, n), device=DEV)
    want = sums.double()
    for step in range(3):
        qs = _randn((heads * group, d), 200 + step, BF16)
        scores = axr.axr_scores(qs, idx, norms, group, b, signs)
        w, tol = plain.weights(scores, sums, group, [n] * heads)
        axr.axr_accumulate_weights(scores, sums, group)
        _within(sums, w, tol, "weights")
    kept = axr.axr_evict(idx, norms, V, sums, _int32([n] * heads), 256, 32)
    _check_evict((idx, norms, V), sums, [n] * heads, 256, 32, kept)
    qs = _randn((heads * group, d), 300, BF16)
    short = axr.axr_scores(qs, kept[0], kept[1], group, b, signs)
    full = axr.axr_scores(qs, idx, norms, group, b, signs)
    rows = kept[4].long().repeat_interleave(group, 0)
    scale = qs.double().norm(dim=1)[:, None] * kept[1].double().repeat_interleave(group, 0) / math.sqrt(d)
    assert ((short - full.gather(1, rows)).abs() <= 1e-4 * scale).all()
    att, _ = axr.axr_attention(qs, *kept[:3], group, b, signs)
    assert att.isfinite().all() and axr.axr_device_status() == 0
    del want
