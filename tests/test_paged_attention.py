"""xpress_paged_attention against the definition in 64 bits.

Tolerances, per output element, with A = sum_j softmax_j |v_j| and R the row's
largest scale * sum_d |q_d k_d|:

* the output is rounded once: half a step of its type, relative;
* a score is an fp32 sum of D exact products, scaled: its error is at most
  (D + 4) 2^-24 R, and moves every weight by as much, relatively; so do the
  exponential (4 * 2^-24, plus the rounding of its argument, 2^-24 times the
  distance in base 2 of the scores, at most 3 R) and the weight's own rounding
  (two 16-bit parts: 2^-16);
* the sums over the keys run 32 at a time: (L / 32 + 40) 2^-24.

A weight's relative error e moves the output by at most 2 e A."""
import math

import numpy as np
import pytest
import torch

import serving_ref as ref
from gpu_util import say
from vocab_wide_add_amd import native


def call(q, kc, vc, table, lens, max_len, window=0, scale=None, k_scale=None, v_scale=None, lse=True,
         stream=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    l_out = torch.full(q.shape[:3], 7.0, device="cuda") if lse else None
    native.xpress_paged_attention(q, kc, vc, table, lens, out, max_len, lse=l_out, scale=scale,
                                  window=window, k_scale=k_scale, v_scale=v_scale, stream=stream)
    return out, l_out


def up(x):
    if x is None:
        return None
    return torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)


def verify(q, kc, vc, table, lens, max_len, window=0, scale=None, k_scale=None, v_scale=None):
    D = q.shape[-1]
    real = 1.0 / math.sqrt(D) if scale is None else scale
    want, want_lse, A, R = ref.attention64(q, kc, vc, table, lens, max_len, float(np.float32(real)),
                                           window, k_scale, v_scale)
    out, lse = call(up(q), up(kc), up(vc), up(table), up(lens), max_len, window, scale, up(k_scale),
                    up(v_scale))
    torch.cuda.synchronize()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    u = 2.0 ** -24
    sums = (max_len / 32 + 40) * u
    e = (D + 4) * u * R + 4 * u + 3 * R * u + sums
    tol = ref.half_step(q.dtype) * np.abs(want) + 2 * (e + 2.0 ** -16)[..., None] * A
    if q.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    bad = ~(np.abs(out - want) <= tol * (1 + 2.0 ** -8))
    assert not bad.any(), (int(bad.sum()), bad.size, float(np.nanmax(np.abs(out - want))))
    empty = np.isinf(want_lse)
    assert np.array_equal(np.isneginf(lse), empty)
    assert (out[empty] == 0).all()
    off = np.abs(lse - want_lse)[~empty]
    assert (off <= (2 * e + u * np.abs(np.where(empty, 0, want_lse)) * 4)[~empty]).all(), off.max()
    return out, lse


def made(seed, lens, Q, Hq, Hk, D, page, dtype="bf16", cache=None, layout="head", sigma=1.5,
         fill=float("nan")):
    rng = np.random.default_rng([seed, 9])
    cache = cache or dtype
    kc, vc, table = ref.paged_pool(rng, lens, Hk, D, page, cache, layout, fill=fill)
    q = torch.from_numpy((rng.standard_normal((len(lens), Q, Hq, D)) * sigma).astype(np.float32))
    scales = {}
    if cache == "e4m3":
        scales = dict(k_scale=torch.from_numpy(rng.uniform(0.04, 0.08, Hk).astype(np.float32)),
                      v_scale=torch.from_numpy(rng.uniform(0.04, 0.08, Hk).astype(np.float32)))
    return (q.to(ref.TYPES[dtype]), kc, vc, table, torch.tensor(lens, dtype=torch.int32)), scales


CASES = [
    # lens, Q, Hq, Hk, D, page, layout, window
    ([1], 1, 1, 1, 64, 16, "head", 0),
    ([0, 1, 2, 31, 32, 33, 64, 65], 1, 8, 2, 128, 16, "head", 0),
    ([127, 128, 129, 255, 0, 300], 1, 4, 4, 64, 32, "token", 0),
    ([700, 5, 1300], 1, 16, 1, 128, 24, "token", 0),
    ([513, 90], 2, 6, 3, 80, 7, "head", 0),
    ([40, 16, 3, 0, 200], 16, 8, 2, 128, 16, "head", 0),      # fewer tokens than queries
    ([260], 16, 8, 1, 64, 16, "token", 0),                     # 128 rows of one head
    ([333, 31], 5, 35, 5, 96, 64, "head", 0),
    ([290, 17], 1, 8, 8, 256, 16, "head", 0),
    ([150], 3, 4, 2, 192, 1, "head", 0),
    ([600, 40, 9], 1, 8, 2, 128, 16, "head", 33),
    ([600, 40, 9, 130], 7, 10, 2, 64, 16, "token", 100),
    ([500, 64], 4, 4, 1, 8, 8, "head", 1),
    ([77], 33, 3, 1, 40, 16, "head", 20),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"),
                                         ("fp16", "e4m3")])
def test_against_64_bits(case, dtype, cache):
    lens, Q, Hq, Hk, D, page, layout, window = CASES[case]
    if cache == "e4m3" and D % 16:
        pytest.skip("8-bit caches take head sizes in sixteens")
    say("attention %d %s %s" % (case, dtype, cache))
    # places that hold no token are NaN
    args, scales = made(case, lens, Q, Hq, Hk, D, page, dtype, cache, layout)
    verify(*args, max(1, max(lens)), window, **scales)


@pytest.mark.gpu
@pytest.mark.parametrize("Q,heads", [(1, (4, 1)), (16, (8, 2))])
def test_long_context_is_split_and_joined(Q, heads):
    lens = [20011, 4097]
    args, _ = made(40, lens, Q, *heads, 128, 64)
    q, kc, vc, table, lens_t = args
    plan = native.xpress_paged_attention_plan(2, Q, *heads, 128, 20011)
    assert plan["splits"] > 1 and plan["launches"] == 2
    # the reference is slow per query: look at the first and last one only
    some = q[:, [0, Q - 1]] if Q > 1 else q
    out, lse = call(up(q), up(kc), up(vc), up(table), up(lens_t), 20011)
    torch.cuda.synchronize()
    for i, at in enumerate([0, Q - 1] if Q > 1 else [0]):
        want, want_lse, A, R = ref.attention64(some[:, i:i + 1], kc, vc, table,
                                               [x - (Q - 1 - at) for x in lens], 20011,
                                               float(np.float32(1 / math.sqrt(128))))
        e = 132 * 2.0 ** -24 * R + 4 * 2.0 ** -24 + 3 * R * 2.0 ** -24 + (20011 / 32 + 40) * 2.0 ** -24
        tol = 2.0 ** -8 * np.abs(want) + 2 * (e + 2.0 ** -16)[..., None] * A
        assert (np.abs(out[:, at:at + 1].double().cpu().numpy() - want) <= tol * (1 + 2.0 ** -8)).all()
        assert (np.abs(lse[:, at:at + 1].double().cpu().numpy() - want_lse) <= 2 * e +
                2.0 ** -22 * np.abs(want_lse)).all()


@pytest.mark.gpu
def test_scores_far_apart_and_all_alike():
    """Scores of +-hundreds (weights underflow, the maximum comes late) and keys
    that are all the same (flat weights)."""
    args, _ = made(50, [900, 300], 2, 4, 2, 64, 16, sigma=60.0)
    verify(*args, 900)
    q, kc, vc, table, lens = args
    verify(q, torch.zeros_like(kc), vc, table, lens, 900)
    # ascending scores: every tile raises the maximum
    up_k = torch.arange(kc.shape[0] * 16).view(-1, 1, 16, 1).expand_as(kc).to(torch.bfloat16) / 64
    verify(q.abs() / 60, up_k.contiguous(), vc, table, lens, 900)
    args, _ = made(51, [900, 300], 1, 4, 2, 64, 16, "fp16", sigma=40.0)
    verify(*args, 900)
    q, kc, vc, table, lens = args
    verify(q, torch.zeros_like(kc), vc, table, lens, 900)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3")])
def test_missing_pages_take_no_part(dtype, cache):
    args, scales = made(60, [200, 70, 48], 2, 4, 2, 64, 16, dtype, cache)
    q, kc, vc, table, lens = args
    table = table.clone()
    table[0, 3], table[0, 7], table[0, 12] = -1, kc.shape[0], 2 ** 31 - 1
    table[1, :] = -5                       # nothing left of sequence 1
    table[2, 2] = -2 ** 31                 # its newest page
    out, lse = verify(q, kc, vc, table, lens, 200, **scales)
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()


@pytest.mark.gpu
def test_lengths_are_clamped():
    args, _ = made(61, [64, 64, 64], 1, 4, 2, 64, 16)
    q, kc, vc, table, _ = args
    table = table[:, :4].contiguous()
    lens = torch.tensor([1000000, -3, 50], dtype=torch.int32)
    verify(q, kc, vc, table, lens, 64)
    verify(q, kc, vc, table, lens, 37)     # a bound below the lengths is the length


@pytest.mark.gpu
def test_nan_and_inf_only_where_they_are_seen():
    args, _ = made(62, [100, 100], 2, 4, 2, 64, 16)
    q, kc, vc, table, lens = args
    kc, vc = kc.clone(), vc.clone()
    p, o = int(table[0, 99 // 16]), 99 % 16
    kc[p, :, o], vc[p, :, o] = float("nan"), float("inf")    # seen by the last query of sequence 0 only
    out, lse = call(up(q), up(kc), up(vc), up(table), up(lens), 100)
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1]).all()
    assert torch.isfinite(out[0, 0]).all() and torch.isfinite(out[1]).all()
    # a finite score against an infinite value gives that infinity
    kc[p, :, o] = 0.0
    out, lse = call(up(q), up(kc), up(vc), up(table), up(lens), 100)
    torch.cuda.synchronize()
    assert torch.isposinf(out[0, 1]).all() and torch.isfinite(lse).all()
    # a key at -inf score has no weight
    kc[p, :, o] = float("-inf")
    vc[p, :, o] = 1.0
    verify(q.abs() + 0.5, kc, vc, table, lens, 100)


@pytest.mark.gpu
@pytest.mark.parametrize("off,pad", [(0, 0), (1, 3), (8, 8)])
def test_strided_queries_and_outputs(off, pad):
    """q and out as slices of larger rows, aligned or not; nothing beside out is written."""
    args, _ = made(63, [150, 33], 3, 6, 2, 64, 16)
    q, kc, vc, table, lens = args
    want, _ = call(up(q), up(kc), up(vc), up(table), up(lens), 150)
    wide = torch.zeros(2, 3, 9, 64 + pad, dtype=torch.bfloat16, device="cuda")
    wide[:, :, 1:7, off:off + 64] = q.cuda()
    big = torch.full((2, 9, 3, 64 + pad), 5.0, dtype=torch.bfloat16, device="cuda")
    out = big[:, 2:8, :, off:off + 64].transpose(1, 2)
    native.xpress_paged_attention(wide[:, :, 1:7, off:off + 64], up(kc), up(vc), up(table), up(lens),
                                  out, 150)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    big[:, 2:8, :, off:off + 64] = 5.0
    assert (big == 5.0).all()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements with the sequence on its last pages."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GiB of GPU memory")
    Hk, D, page = 2, 128, 16
    pages = (2 ** 32) // (Hk * page * D) + 64
    args, _ = made(64, [300], 1, 4, Hk, D, page)
    q, kc, vc, table, lens = args
    big = [torch.zeros(pages, Hk, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    shift = pages - kc.shape[0]
    for b, x in zip(big, (kc, vc)):
        b[shift:] = x.cuda()
    t2 = torch.where(table >= 0, table + shift, table)
    want, want_lse = call(up(q), up(kc), up(vc), up(table), up(lens), 300)
    got, lse = call(up(q), big[0], big[1], up(t2), up(lens), 300)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(lse, want_lse)


@pytest.mark.gpu
def test_results_do_not_change_from_run_to_run():
    args, _ = made(65, [3000, 1500, 20], 4, 8, 2, 128, 16)
    q, kc, vc, table, lens = [up(x) for x in args]
    want, want_lse = call(q, kc, vc, table, lens, 3000)
    for _ in range(5):
        got, lse = call(q, kc, vc, table, lens, 3000)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(lse, want_lse)


@pytest.mark.gpu
def test_capture_needs_the_workspace_reserved():
    args, _ = made(66, [9000, 7000], 1, 4, 1, 128, 16)
    q, kc, vc, table, lens = [up(x) for x in args]
    want, want_lse = call(q, kc, vc, table, lens, 9000)
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    native.xpress_paged_attention_reserve(2, 1, 4, 1, 128, 9000, stream=s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        native.xpress_paged_attention(q, kc, vc, table, lens, out, 9000, lse=lse)
    for _ in range(3):
        out.zero_(), lse.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        call(q, kc, vc, table, lens, 9000)
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_two_streams_at_once():
    sets = []
    for i in range(2):
        args, _ = made(70 + i, [5000 + i, 800], 2, 8, 2, 128, 16)
        args = [up(x) for x in args]
        sets.append((args, call(*args, 5000 + i)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(4):
        got = [call(*a, 5000 + i, stream=s) for i, ((a, _), s) in enumerate(zip(sets, streams))]
    torch.cuda.synchronize()
    for (_, want), have in zip(sets, got):
        assert torch.equal(want[0], have[0]) and torch.equal(want[1], have[1])


@pytest.mark.gpu
def test_append_then_attend_gives_the_same_as_a_fresh_cache():
    """Tokens appended one call at a time, then attended to, against a cache built whole."""
    rng = np.random.default_rng(80)
    Hq, Hk, D, page, L = 4, 2, 64, 16, 45
    rows = torch.from_numpy(rng.standard_normal((L, Hq + 2 * Hk, D)).astype(np.float32)).to(torch.bfloat16)
    rows = rows.cuda()
    angle = np.arange(L)[:, None] * 10000.0 ** (-np.arange(D // 2) / (D // 2))
    cs = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    caches = [[torch.zeros(4, Hk, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
              for _ in range(2)]
    q1, q2 = (torch.zeros(L, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:]
    native.xpress_kv_append(q, k, v, q1, *caches[0], table, pos, cs)
    outs = []
    for t in range(L):
        native.xpress_kv_append(q[t:t + 1], k[t:t + 1], v[t:t + 1], q2[t:t + 1], *caches[1], table,
                                pos[t:t + 1], cs)
        lens = torch.tensor([t + 1], dtype=torch.int32, device="cuda")
        outs.append(call(q2[t:t + 1][None], *caches[1], table, lens, 48)[0])
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    whole, _ = call(q1[None], *caches[0], table, lens, 48)
    torch.cuda.synchronize()
    for a, b in zip(caches[0], caches[1]):
        assert torch.equal(a, b)
    assert torch.equal(q1, q2)
    # one query at a time or all together: the sums run in another order
    one = torch.cat(outs, 1).double().cpu().numpy()
    want, _, A, R = ref.attention64(q1[None].cpu(), caches[0][0].cpu(), caches[0][1].cpu(), table.cpu(),
                                    [L], 48, float(np.float32(1 / 8)))
    e = 71 * 2.0 ** -24 * R + 46 * 2.0 ** -24 + 2.0 ** -16
    for got in (one, whole.double().cpu().numpy()):
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2 * e[..., None] * A * 1.01).all()


def near64(out, lse, q, kc, vc, table, lens, max_len, at, n, window=0, k_scale=None, v_scale=None):
    """Query `at` of sequence n of a call against 64 bits, with the tolerances above."""
    Q, D = q.shape[1], q.shape[-1]
    want, want_lse, A, R = ref.attention64(
        q[n:n + 1, at:at + 1], kc, vc, table[n:n + 1], [int(lens[n]) - (Q - 1 - at)], max_len,
        float(np.float32(1 / math.sqrt(D))), window, k_scale, v_scale)
    u = 2.0 ** -24
    e = (D + 4) * u * R + 4 * u + 3 * R * u + (int(lens[n]) / 32 + 40) * u
    tol = ref.half_step(q.dtype) * np.abs(want) + 2 * (e + 2.0 ** -16)[..., None] * A
    if q.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    got, got_lse = out[n:n + 1, at:at + 1].double().cpu().numpy(), lse[n:n + 1, at:at + 1].double().cpu().numpy()
    assert (np.abs(got - want) <= tol * (1 + 2.0 ** -8)).all(), np.abs(got - want).max()
    empty = np.isinf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty) and (got[empty] == 0).all()
    off = np.abs(np.where(empty, 0, got_lse) - np.where(empty, 0, want_lse))
    assert (off <= 2 * e + 4 * u * np.abs(np.where(empty, 0, want_lse))).all(), off.max()


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 3001])
def test_a_prompt_in_one_part(window):
    """Hundreds of queries over several thousand keys: one part, several tables of places."""
    say("attention prompt %d" % window)
    Hq, Hk, D, Q, L = 256, 8, 64, 512, 5000
    assert native.xpress_paged_attention_plan(1, Q, Hq, Hk, D, L, window)["splits"] == 1
    args, _ = made(90, [L], Q, Hq, Hk, D, 16)
    q, kc, vc, table, lens = args
    table = table.clone()
    table[0, 100], table[0, 200] = -1, kc.shape[0]            # pages that are not there, in later tables
    out, lse = call(up(q), up(kc), up(vc), up(table), up(lens), L, window)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    for at in (0, 1, 255, Q - 1):
        near64(out, lse, q, kc, vc, table, lens, L, at, 0, window)


@pytest.mark.gpu
def test_a_prompt_with_values_that_some_do_not_see():
    """A NaN value that only the last queries see: the others' sums are taken again, table by table."""
    Hq, Hk, D, Q, L = 256, 8, 64, 512, 5000
    args, _ = made(91, [L], Q, Hq, Hk, D, 16)
    q, kc, vc, table, lens = args
    vc = vc.clone()
    vc[int(table[0, (L - 3) // 16]), :, (L - 3) % 16] = float("nan")
    out, lse = call(up(q), up(kc), up(vc), up(table), up(lens), L)
    torch.cuda.synchronize()
    assert torch.isnan(out[0, Q - 3:]).all() and torch.isfinite(out[0, :Q - 3]).all()
    for at in (0, 300, Q - 4):
        near64(out, lse, q, kc, vc, table, lens, L, at, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("N,Q,Hq,Hk,D,dtype,cache", [
    (4000, 1, 8, 8, 64, "bf16", "bf16"), (4000, 1, 8, 8, 128, "fp16", "fp16"), (1000, 2, 32, 2, 64, "fp16", "e4m3"),
    (1000, 8, 8, 1, 128, "bf16", "bf16"), (4000, 1, 4, 2, 256, "bf16", "e4m3"), (1000, 3, 14, 2, 80, "bf16", "e4m3")])
def test_many_rows_under_a_high_bound(N, Q, Hq, Hk, D, dtype, cache):
    """Parts longer than a table of places, as the workspace's limit asks for."""
    say("attention bound %d %d %d %d %d %s %s" % (N, Q, Hq, Hk, D, dtype, cache))
    bound, page = 2 ** 20, 256
    plan = native.xpress_paged_attention_plan(N, Q, Hq, Hk, D, bound)
    assert plan["chunk"] > 2048 and plan["splits"] > 1
    rng = np.random.default_rng([92, D])
    lens = rng.integers(0, 60, N)
    far = [0, N // 2, N - 1]
    lens[far] = 20011, 4097, 9000
    args, scales = made(92, [600], 1, Hq, Hk, D, page, dtype, cache, fill=0.0)
    _, kc, vc, _, _ = args
    q = torch.from_numpy((rng.standard_normal((N, Q, Hq, D)) * 1.5).astype(np.float32)).to(ref.TYPES[dtype])
    # every sequence on pages of the one small pool, in an order of its own
    table = torch.full((N, bound // page), -1, dtype=torch.int32)
    for n in range(N):
        need = -(-int(lens[n]) // page)
        table[n, :need] = torch.from_numpy(rng.integers(0, kc.shape[0], need).astype(np.int32))
    table[0, 30] = -1
    lens_t = torch.from_numpy(lens.astype(np.int32))
    try:
        out, lse = call(up(q), up(kc), up(vc), up(table), up(lens_t), bound, **{k: up(v) for k, v in scales.items()})
        torch.cuda.synchronize()
        assert native.xpress_workspace_bytes() <= 3 << 30       # with what earlier calls left
    finally:
        native.xpress_release()
    assert torch.isfinite(out).all()
    for n in far + [1, 2, 3, 4]:
        for at in {0, Q - 1}:
            near64(out, lse, q, kc, vc, table, lens, bound, at, n, **scales)


@pytest.mark.gpu
def test_more_owners_than_a_grid_has_threads_for():
    """2^24 workgroups of 256 threads are 2^32."""
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GiB of GPU memory")
    say("attention owners past a grid")
    N, D, page = 2 ** 24 + 1000, 8, 16
    g = torch.Generator(device="cuda").manual_seed(93)
    kc, vc = (torch.randn(64, 1, page, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(N, 1, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randint(0, 64, (N, 1), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.randint(0, page + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
    out, lse = call(q, kc, vc, table, lens, page)
    torch.cuda.synchronize()
    for part in (slice(0, 3000), slice(2 ** 22 - 2000, 2 ** 22 + 2000), slice(N - 3000, N)):
        got, l_got = call(q[part], kc, vc, table[part], lens[part], page)
        torch.cuda.synchronize()
        assert torch.equal(got, out[part]) and torch.equal(l_got, lse[part])


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_strides_of_single_places_do_not_matter(cache):
    """One key-value head, one page, pages of one token: their strides address nothing (torch's
    channels-last form gives a single head the stride 1)."""
    for Hk, page, length in ((1, 16, 90), (2, 128, 90), (2, 1, 90)):
        args, scales = made(94, [length], 2, 4, Hk, 64, page, "bf16", cache)
        q, kc, vc, table, lens = args
        if Hk == 2 and page == 128:      # the sequence's one page alone
            at = int(table[0, 0])
            kc, vc, table = kc[at:at + 1].clone(), vc[at:at + 1].clone(), torch.zeros_like(table[:, :1])
        scales = {k: up(v) for k, v in scales.items()}
        want = call(up(q), up(kc), up(vc), up(table), up(lens), length, **scales)
        odd = [up(x) for x in (kc, vc)]
        odd = [x.as_strided(x.shape, [s if n > 1 else 3 for n, s in zip(x.shape[:3], x.stride()[:3])] + [1])
               for x in odd]
        got = call(up(q), *odd, up(table), up(lens), length, **scales)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_a_single_head_in_the_channels_last_form():
    args, _ = made(95, [90, 33], 2, 4, 1, 64, 16, fill=0.0)
    q, kc, vc, table, lens = [up(x) for x in args]
    want = call(q, kc, vc, table, lens, 90)
    last = [x.to(memory_format=torch.channels_last) for x in (kc, vc)]
    assert last[0].stride(1) == 1
    got = call(q, *last, table, lens, 90)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
