"""xpress_tree_attention and xpress_sink_attention against the definition in 64 bits.

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

import drafts_ref as ref
import serving_ref
from gpu_util import say
from vocab_wide_add_amd import native


def up(x):
    if x is None:
        return None
    return torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)


def call(q, kc, vc, table, lens, max_len, window, sinks, tree, scale=None, k_scale=None, v_scale=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    more = dict(lse=lse, scale=scale, k_scale=up(k_scale), v_scale=up(v_scale))
    args = [up(q), up(kc), up(vc), up(table), up(lens)]
    if tree is None:
        native.xpress_sink_attention(*args, out, max_len, window, sinks, **more)
    else:
        native.xpress_tree_attention(*args, up(tree), out, max_len, window=window, sinks=sinks, **more)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def verify(q, kc, vc, table, lens, max_len, window=0, sinks=0, sees=None, scale=None, k_scale=None, v_scale=None,
           tree=None):
    D = q.shape[-1]
    real = 1.0 / math.sqrt(D) if scale is None else scale
    want, want_lse, A, R = ref.attention64(q, kc, vc, table, lens, max_len, float(np.float32(real)), window,
                                           sinks, sees, k_scale, v_scale)
    if sees is not None and tree is None:
        tree = ref.words_of(sees)
    out, lse = call(q, kc, vc, table, lens, max_len, window, sinks, tree, scale, k_scale, v_scale)
    u = 2.0 ** -24
    e = (D + 4) * u * R + 4 * u + 3 * R * u + (max_len / 32 + 40) * u
    tol = serving_ref.half_step(q.dtype) * np.abs(want) + 2 * (e + 2.0 ** -16)[..., None] * A
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


def made(seed, lens, Q, Hq, Hk, D, page, dtype="bf16", cache=None, layout="head", sigma=1.5):
    """Inputs whose places without a token are NaN, and random trees."""
    rng = np.random.default_rng([seed, 19])
    cache = cache or dtype
    kc, vc, table = serving_ref.paged_pool(rng, lens, Hk, D, page, cache, layout, fill=float("nan"))
    q = torch.from_numpy((rng.standard_normal((len(lens), Q, Hq, D)) * sigma).astype(np.float32))
    scales = {}
    if cache == "e4m3":
        scales = dict(k_scale=torch.from_numpy(rng.uniform(0.04, 0.08, Hk).astype(np.float32)),
                      v_scale=torch.from_numpy(rng.uniform(0.04, 0.08, Hk).astype(np.float32)))
    args = (q.to(serving_ref.TYPES[dtype]), kc, vc, table, torch.tensor(lens, dtype=torch.int32))
    return args, scales, ref.random_trees(rng, len(lens), Q)[1], rng


def without(kc, vc, table, lens, Q, window, sinks, late):
    """Pages that no query sees given back: -1 in the table, and NaN throughout."""
    table, kc, vc = table.clone(), kc.clone(), vc.clone()
    page = kc.shape[2]
    for n, length in enumerate(lens.tolist()):
        for s in range(-(-length // page)):
            if s * page >= sinks and (s + 1) * page <= length - Q - window + late:
                kc[table[n, s]], vc[table[n, s]] = float("nan"), float("nan")
                table[n, s] = -1
    return kc, vc, table


CASES = [
    # lens, Q, Hq, Hk, D, page, layout, window, sinks
    ([1], 1, 1, 1, 64, 16, "head", 0, 0),
    ([0, 1, 2, 31, 32, 33, 64, 65], 1, 8, 2, 128, 16, "head", 0, 0),
    ([127, 128, 129, 255, 0, 300], 2, 4, 4, 64, 32, "token", 40, 3),
    ([700, 5, 1300], 8, 16, 4, 128, 24, "token", 0, 0),
    ([513, 90], 2, 6, 3, 80, 7, "head", 100, 7),
    ([40, 16, 3, 0, 200], 16, 8, 2, 128, 16, "head", 0, 0),      # fewer tokens than nodes
    ([260, 64], 33, 8, 1, 64, 16, "token", 0, 0),                 # 264 rows of one head, two words
    ([333, 31], 5, 35, 5, 96, 64, "head", 64, 64),
    ([290, 17], 1, 8, 8, 256, 16, "head", 20, 1),
    ([150, 700], 70, 2, 1, 32, 16, "head", 0, 0),                 # three words
    ([600, 40, 9], 1, 8, 2, 128, 16, "head", 33, 4),
    ([600, 40, 9, 130], 7, 10, 2, 64, 16, "token", 100, 33),
    ([500, 64], 4, 4, 1, 8, 8, "head", 1, 2),
    ([77, 400], 33, 3, 1, 40, 16, "head", 20, 500),               # more sinks than what the window leaves
    ([2600], 3, 4, 2, 64, 16, "head", 1000, 130),
    # more than 64 rows a key-value head
    ([100, 64, 65, 1, 0], 9, 16, 2, 128, 16, "token", 0, 0),      # 72 rows
    ([1500, 40], 20, 4, 1, 256, 16, "head", 0, 0),
    ([333, 20], 33, 9, 3, 192, 1, "head", 50, 7),
    ([200] * 9 + [35, 0, 700], 17, 8, 2, 64, 7, "token", 60, 20), # more parts than XCDs
    ([65, 63], 129, 2, 1, 96, 32, "head", 0, 0),                  # more nodes than tokens, five words
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("form", ["tree", "sinks"])
def test_against_64_bits(case, dtype, cache, form):
    lens, Q, Hq, Hk, D, page, layout, window, sinks = CASES[case]
    if cache == "e4m3" and D % 16:
        pytest.skip("8-bit caches take head sizes in sixteens")
    say("%s %d %s %s" % (form, case, dtype, cache))
    (q, kc, vc, table, lens_t), scales, sees, _ = made(case, lens, Q, Hq, Hk, D, page, dtype, cache, layout)
    if window:
        kc, vc, table = without(kc, vc, table, lens_t, Q, window, sinks, 0 if form == "tree" else 1)
    verify(q, kc, vc, table, lens_t, max(1, max(lens)), window, sinks, sees if form == "tree" else None, **scales)


@pytest.mark.gpu
@pytest.mark.parametrize("Q", [5, 40, 65])
def test_any_mask_and_nodes_that_see_nothing(Q):
    """Masks that are no trees: bits drawn, rows of none, and with no token before the
    tree nothing at all is left to them."""
    (q, kc, vc, table, lens), _, _, rng = made(70 + Q, [Q, Q + 100, Q - 2], Q, 4, 2, 64, 16)
    sees = rng.random((3, Q, Q)) < 0.3
    sees[:, 1] = False
    sees[0, 3] = False
    out, lse = verify(q, kc, vc, table, lens, Q + 100, sees=sees)
    assert (out[0, [1, 3]] == 0).all() and np.isneginf(lse[0, [1, 3]]).all()
    verify(q, kc, vc, table, lens, Q + 100, 20, 3, sees=sees)
    # a window of one leaves a node that sees no node the place before the tree's
    verify(q, kc, vc, table, lens, Q + 100, 1, 0, sees=sees)


@pytest.mark.gpu
def test_bits_past_the_tree_are_not_looked_at():
    (q, kc, vc, table, lens), _, sees, _ = made(80, [200, 50], 37, 4, 2, 64, 16)
    tree = ref.words_of(sees)
    tree[..., 1] |= -32          # nodes 37 to 63
    verify(q, kc, vc, table, lens, 200, 30, 2, sees=sees, tree=tree)


@pytest.mark.gpu
def test_one_tree_for_all_and_strided_words():
    (q, kc, vc, table, lens), _, sees, _ = made(81, [200, 50, 31], 34, 4, 2, 64, 16)
    one = ref.words_of(sees[0])
    sees = np.broadcast_to(sees[0], sees.shape)
    wide = torch.full((34, 7), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:4] = one.cuda()
    tree = wide[:, 2:4].expand(3, 34, 2)
    want = call(q, kc, vc, table, lens, 200, 0, 0, ref.words_of(sees))
    out, lse = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(q.shape[:3], device="cuda")
    native.xpress_tree_attention(up(q), up(kc), up(vc), up(table), up(lens), tree, out, 200, lse=lse)
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want[0])
    assert np.array_equal(lse.double().cpu().numpy(), want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("Q,window,sinks", [(1, 0, 0), (6, 0, 0), (20, 50, 0), (20, 50, 5)])
def test_a_chain_is_the_dense_form(Q, window, sinks):
    """A tree without branches sees what the dense form sees; its window is of the places
    before the tree, so that only Q <= window is the same."""
    (q, kc, vc, table, lens), _, _, _ = made(82, [900, 77, 20], Q, 8, 2, 128, 16)
    sees = np.broadcast_to(np.tril(np.ones((Q, Q), bool)), (3, Q, Q))
    tree = call(q, kc, vc, table, lens, 900, window, sinks, ref.words_of(sees))
    flat = call(q, kc, vc, table, lens, 900, window, sinks, None)
    for x, y in zip(tree, flat):
        assert np.allclose(x, y, rtol=2.0 ** -7, atol=2.0 ** -14)   # two roundings of results near each other
    verify(q, kc, vc, table, lens, 900, window, sinks)


@pytest.mark.gpu
def test_no_sinks_is_the_windowed_form_bit_for_bit():
    (q, kc, vc, table, lens), _, _, _ = made(83, [900, 77, 20], 3, 8, 2, 128, 16)
    for window in (0, 1, 40, 5000):
        got = call(q, kc, vc, table, lens, 900, window, 0, None)
        out, lse = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(q.shape[:3], device="cuda")
        native.xpress_paged_attention(up(q), up(kc), up(vc), up(table), up(lens), out, 900, lse=lse, window=window)
        torch.cuda.synchronize()
        assert np.array_equal(got[0], out.double().cpu().numpy())
        assert np.array_equal(got[1], lse.double().cpu().numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 1500])
def test_not_finite_values_reach_only_the_nodes_that_see_them(window):
    """Two siblings: what one of them put into the cache is NaN or infinite and must not
    reach the other, nor a place behind the window anything."""
    (q, kc, vc, table, lens), _, _, _ = made(84, [2000, 600], 3, 4, 2, 64, 16)
    kc, vc = kc.clone(), vc.clone()
    sees = np.zeros((2, 3, 3), bool)
    sees[:, 0, 0] = sees[:, 1, [0, 1]] = sees[:, 2, [0, 2]] = True
    for n, length in enumerate((2000, 600)):
        at = length - 2               # node 1
        kc[table[n, at // 16], :, at % 16] = float("nan")
        vc[table[n, at // 16], :, at % 16] = float("inf")
    if window:
        kc[table[0, 10], :, 3], vc[table[0, 10], :, 3] = float("nan"), float("nan")     # place 163, past the sinks
    out, lse = call(q, kc, vc, table, lens, 2000, window, 100, ref.words_of(sees))
    assert np.isnan(out[:, 1]).all() and np.isnan(lse[:, 1]).all()
    assert np.isfinite(out[:, [0, 2]]).all() and np.isfinite(lse[:, [0, 2]]).all()
    clean_k, clean_v = torch.nan_to_num(kc, nan=0.0), torch.nan_to_num(vc, nan=0.0, posinf=0.0)
    want, _ = call(q, clean_k, clean_v, table, lens, 2000, window, 100, ref.words_of(sees))
    # the careful form adds its products in another order: two roundings apart at most
    assert np.allclose(out[:, [0, 2]], want[:, [0, 2]], rtol=2.0 ** -7, atol=2.0 ** -12)


@pytest.mark.gpu
def test_long_contexts_in_parts():
    """Splits with a join, whose first part holds the sinks; lengths under and over."""
    say("long window")
    (q, kc, vc, table, lens), _, sees, _ = made(85, [9000, 40, 4000], 2, 4, 1, 64, 64)
    kc, vc, table = without(kc, vc, table, lens, 2, 3000, 70, 0)
    verify(q, kc, vc, table, lens, 9000, 3000, 70)
    verify(q, kc, vc, table, lens, 9000, 3000, 70, sees=sees)
    (q, kc, vc, table, lens), _, sees, _ = made(86, [9000, 70], 20, 4, 1, 64, 64)
    verify(q, kc, vc, table, lens, 9000, sees=sees)
    say("a bound far above the lengths")
    wide = torch.full((2, 4000), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    verify(q, kc, vc, wide, lens, 200000, sees=sees)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cache,page", [("bf16", "bf16", 64), ("fp16", "e4m3", 5), ("bf16", "bf16", 1)])
def test_long_contexts_under_many_rows(dtype, cache, page):
    """More stages than the ring of places has, in one part and in several."""
    say("many rows %s %s %d" % (dtype, cache, page))
    (q, kc, vc, table, lens), scales, sees, _ = made(88, [4500, 70, 1300, 600], 18, 8, 2, 64, page, dtype, cache)
    verify(q, kc, vc, table, lens, 4500, sees=sees, **scales)
    kc, vc, table = without(kc, vc, table, lens, 18, 2000, 70, 0)
    verify(q, kc, vc, table, lens, 4500, 2000, 70, sees=sees, **scales)
    verify(q[:1, -1:].expand(1, 18, 8, 64).contiguous(), kc, vc, table[:1], lens[:1], 4500, 900, 33, **scales)


@pytest.mark.gpu
@pytest.mark.parametrize("Q,dtype,cache", [(1, "bf16", "bf16"), (4, "fp16", "e4m3"), (9, "bf16", "bf16")])
def test_parts_by_size_and_of_many_lengths(Q, dtype, cache):
    """More workgroups than the chip holds, of parts between none and all of their keys: every
    part is taken once, whatever its rank."""
    lens = [(37 * i * i) % 2600 for i in range(38)] + [0, 2600]
    (q, kc, vc, table, lens), scales, sees, _ = made(93, lens, Q, 16, 8, 64, 16, dtype, cache)
    verify(q, kc, vc, table, lens, 2600, sees=sees, **scales)
    verify(q, kc, vc, table, lens, 2600, **scales)


@pytest.mark.gpu
def test_more_sequences_than_are_ranked():
    say("300 sequences")
    rng = np.random.default_rng(4)
    (q, kc, vc, table, lens), _, sees, _ = made(89, rng.integers(0, 40, 300).tolist(), 33, 2, 1, 32, 16)
    verify(q, kc, vc, table, lens, 40, sees=sees)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("Q", [3, 40])
def test_other_scales(scale, Q):
    (q, kc, vc, table, lens), _, sees, _ = made(90, [300, 50], Q, 4, 2, 64, 16)
    verify(q, kc, vc, table, lens, 300, sees=sees, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Q", [3, 40])
def test_a_scale_of_zero_keeps_queries_that_are_not_finite(Q, dtype):
    (q, kc, vc, table, lens), _, sees, _ = made(90, [300, 50], Q, 4, 2, 64, 16, dtype, dtype)
    q = q.clone()
    q[0, 1, 2, 5], q[1, 2, 0, 60], q[1, 0, 1, 0] = float("nan"), float("inf"), float("-inf")
    out, lse = call(q, kc, vc, table, lens, 300, 0, 0, ref.words_of(sees), 0.0)
    hit = np.zeros(q.shape[:3], bool)
    hit[0, 1, 2] = hit[1, 2, 0] = hit[1, 0, 1] = True
    assert np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
    assert np.isfinite(out[~hit]).all() and np.isfinite(lse[~hit]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_not_finite_values_under_many_rows(cache):
    """As above with 40 nodes: 80 rows a head, four words of them in two waves and more."""
    (q, kc, vc, table, lens), scales, sees, _ = made(91, [700, 90], 40, 4, 2, 64, 16, "bf16", cache)
    kc, vc = kc.clone(), vc.clone()
    sees = sees.copy()
    sees[:, :, 7] = False
    sees[:, 7, 7] = sees[:, 30, 7] = True
    for n, length in enumerate((700, 90)):
        at = length - 40 + 7
        kc[table[n, at // 16], :, at % 16] = 1.0
        vc[table[n, at // 16], :, at % 16] = float("nan")
    out, lse = call(q, kc, vc, table, lens, 700, 0, 0, ref.words_of(sees), **scales)
    hit = [7, 30]
    rest = [i for i in range(40) if i not in hit]
    assert np.isnan(out[:, hit]).all() and np.isfinite(out[:, rest]).all() and np.isfinite(lse).all()
    clean = torch.nan_to_num(vc.float(), nan=0.0).to(vc.dtype)
    kc2 = torch.nan_to_num(kc.float(), nan=0.0).to(kc.dtype)
    want, _ = call(q, kc2, clean, table, lens, 700, 0, 0, ref.words_of(sees), **scales)
    # the careful form adds its products in another order: two roundings apart at most
    assert np.allclose(out[:, rest], want[:, rest], rtol=2.0 ** -7, atol=2.0 ** -12)


@pytest.mark.gpu
@pytest.mark.parametrize("Q", [6, 40])
def test_missing_pages_take_no_part(Q):
    (q, kc, vc, table, lens), _, sees, _ = made(92, [400, 70 + Q, 48 + Q], Q, 4, 2, 64, 16)
    table = table.clone()
    table[0, 3], table[0, 7], table[0, 12] = -1, kc.shape[0], 2 ** 31 - 1
    table[1, :] = -5
    table[2, 2] = -2 ** 31
    out, lse = verify(q, kc, vc, table, lens, 400, sees=sees)
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()
    verify(q, kc, vc, table, lens, 400, 37, 20)


@pytest.mark.gpu
def test_captured_and_replayed():
    (q, kc, vc, table, lens), _, sees, _ = made(87, [3000, 500], 12, 8, 2, 128, 16)
    want = call(q, kc, vc, table, lens, 3000, 0, 0, ref.words_of(sees))
    args = [up(q), up(kc), up(vc), up(table), up(lens)]
    tree, out = up(ref.words_of(sees)), torch.zeros(q.shape, dtype=q.dtype, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    native.xpress_sparse_attention_reserve(2, 12, 8, 2, 128, 3000, tree=True, stream=stream)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        native.xpress_tree_attention(*args, tree, out, 3000)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), want[0])
        # other work on the default stream's workspace in between
        call(q, kc, vc, table, lens, 3000, 100, 5, None)
    # without its workspace a capture is refused and nothing is queued
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out.add_(0)
        with pytest.raises(native.XpressError) as e:
            native.xpress_tree_attention(*args, tree, out, 3000)
    assert e.value.status == native.XPRESS_ECAPTURE


def _cpu(**change):
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    d = dict(q=torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), k=k, v=k.clone(),
             table=torch.zeros(2, 2, dtype=torch.int32), lens=torch.zeros(2, dtype=torch.int32),
             out=torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), tree=torch.zeros(2, 3, 1, dtype=torch.int32))
    d.update(change)
    return d


def test_tensors_on_the_cpu_are_refused():
    d = _cpu()
    with pytest.raises(ValueError, match="GPU"):
        native.xpress_tree_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], d["tree"], d["out"], 32)
    with pytest.raises(ValueError, match="GPU"):
        native.xpress_sink_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], d["out"], 32, 8, 4)


@pytest.mark.gpu
def test_trees_of_other_shapes_and_types_are_refused():
    d = {k: v.cuda() for k, v in _cpu().items()}

    def go(**change):
        x = dict(d, **change)
        native.xpress_tree_attention(x["q"], x["k"], x["v"], x["table"], x["lens"], x["tree"], x["out"], 32,
                                     sinks=x.get("sinks", 0), window=x.get("window", 0))
    go()
    for bad in (d["tree"].long(), d["tree"][:, :2], torch.zeros(2, 3, 2, dtype=torch.int32, device="cuda"),
                d["tree"].cpu()):
        with pytest.raises(ValueError, match="tree"):
            go(tree=bad)
    for bad in (dict(sinks=-1), dict(window=-1), dict(sinks=2 ** 31)):
        with pytest.raises(native.XpressError):
            go(**bad)
    # out on the tree's words
    words = torch.zeros(2 * 3 * 4 * 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(native.XpressError):
        go(out=words.view(2, 3, 4, 64), tree=words.view(torch.int32)[:6].view(2, 3, 1))
