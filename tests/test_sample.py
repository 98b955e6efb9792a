"""xpress_sample_to_blk against the definition in 64 bits: the ids have to be equal, the
probability is rounded once to fp32 (2^-24, and 2^-40 for the 64-bit sums before it)."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from gpu_util import say
from vocab_wide_add_amd import native

OPEN = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)


def settings(rows, rng, **given):
    out = {}
    for name, default in OPEN.items():
        v = given.get(name, default)
        out[name] = np.broadcast_to(np.asarray(v, np.int32 if name == "top_k" else np.float32), rows).copy()
    u = given.get("u")
    out["u"] = rng.random(rows, np.float32) if u is None else np.broadcast_to(np.float32(u), rows).copy()
    return out


def draw(base, bias, N, B, V, s, prob=True):
    blk = torch.full((N, B), -5, dtype=torch.int64, device="cuda")
    p = torch.full((N * (B - 1),), 7.0, device="cuda") if prob else None
    dev = {k: torch.from_numpy(v).cuda() for k, v in s.items()}
    native.xpress_sample_to_blk(base, bias, blk, dev["temperature"], dev["top_k"], dev["top_p"],
                                dev["min_p"], dev["u"], N, B, V, base.stride(0),
                                bias.stride(0) if bias is not None else 0, prob=p)
    torch.cuda.synchronize()
    assert (blk[:, 0] == -5).all()
    return blk[:, 1:].reshape(-1).cpu().numpy(), p.cpu().numpy() if prob else None


def verify(base, bias, N, B, V, s):
    """base, bias: CPU bf16 tensors [rows, stride]."""
    z = base[:, :V].double()
    if bias is not None:
        z = (base[:, :V].float() + bias[:, :V].float()).to(torch.bfloat16).double()
    ids, probs = ref.sample64(z.numpy(), s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"])
    got, p = draw(base.cuda(), bias.cuda() if bias is not None else None, N, B, V, s)
    assert np.array_equal(got, ids), (got, ids, s)
    assert (np.abs(p - probs) <= probs * (2.0 ** -24 + 2.0 ** -40)).all(), (p, probs)
    return ids, probs


def normal(rng, rows, stride, sigma=4.0):
    return torch.from_numpy((rng.standard_normal((rows, stride)) * sigma).astype(np.float32)).to(torch.bfloat16)


FILTERS = {
    "open": {},
    "cold": dict(temperature=0.05),
    "hot": dict(temperature=50.0),
    "greedy": dict(temperature=0.0),
    "k1": dict(top_k=1),
    "k50": dict(top_k=50, temperature=2.0),
    "p": dict(top_p=0.9),
    "p_small": dict(top_p=1e-6),
    "min_p": dict(min_p=0.02),
    "k_p_min": dict(top_k=40, top_p=0.95, min_p=0.001, temperature=1.7),
    "k_over": dict(top_k=10 ** 9),
}


@pytest.mark.gpu
@pytest.mark.parametrize("filters", sorted(FILTERS))
@pytest.mark.parametrize("N,B,V,pad,with_bias", [
    (1, 2, 1, 0, False), (2, 4, 7, 1, True), (3, 5, 1000, 0, True), (2, 16, 1003, 0, False),
    (1, 9, 8192, 64, True), (1, 4, 32000, 0, False), (2, 3, 40961, 7, True), (1, 3, 152064, 0, True),
    (1, 2, 200001, 0, False)])
def test_against_64_bits(filters, N, B, V, pad, with_bias):
    say("sample %s %d %d %d %d %s" % (filters, N, B, V, pad, with_bias))
    rng = np.random.default_rng([V, sorted(FILTERS).index(filters)])
    rows = N * (B - 1)
    base, bias = normal(rng, rows, V + pad), normal(rng, rows, V + pad, 0.5) if with_bias else None
    verify(base, bias, N, B, V, settings(rows, rng, **FILTERS[filters]))


@pytest.mark.gpu
def test_rows_have_settings_of_their_own():
    rng = np.random.default_rng(11)
    rows, V = 60, 5000
    s = settings(rows, rng)
    s["temperature"] = rng.choice([0.0, 0.3, 1.0, 4.0, -1.0, np.nan], rows).astype(np.float32)
    s["top_k"] = rng.choice([-3, 0, 1, 2, 17, 600], rows).astype(np.int32)
    s["top_p"] = rng.choice([0.0, -1.0, 0.5, 0.99, 1.0, 2.0, np.nan], rows).astype(np.float32)
    s["min_p"] = rng.choice([0.0, 0.1, 1.0, 2.0, -1.0, np.nan], rows).astype(np.float32)
    verify(normal(rng, rows, V), normal(rng, rows, V, 0.5), 15, 5, V, s)


@pytest.mark.gpu
@pytest.mark.parametrize("u", [0.0, 1.0, 1 - 2.0 ** -24, -1.0, 2.0, float("nan"), 0.5])
def test_ends_of_the_uniform_number(u):
    rng = np.random.default_rng(12)
    base = normal(rng, 3, 500)
    for f in ("open", "k50", "p", "min_p"):
        verify(base, None, 1, 4, 500, settings(3, rng, u=u, **FILTERS[f]))


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1000, 70000, 152064])
def test_ties(V):
    """Integer logits: thousands of equal values, picked by id; all equal; two values."""
    rng = np.random.default_rng([13, V])
    ints = torch.from_numpy(rng.integers(-8, 9, (4, V)).astype(np.float32)).to(torch.bfloat16)
    for f in ("open", "k50", "p", "k_p_min", "hot"):
        verify(ints, None, 2, 3, V, settings(4, rng, **FILTERS[f]))
    for value in (0.0, 3.5, -2.0):
        flat = torch.full((4, V), value, dtype=torch.bfloat16)
        for f in ("open", "k50", "p", "greedy", "min_p"):
            verify(flat, None, 2, 3, V, settings(4, rng, **FILTERS[f]))
    two = torch.where(torch.from_numpy(rng.random((4, V)) < 0.02), 1.0, -1.0).to(torch.bfloat16)
    for f in ("open", "k50", "p", "greedy"):
        verify(two, None, 2, 3, V, settings(4, rng, **FILTERS[f]))


@pytest.mark.gpu
def test_both_zeros_are_one_value():
    rng = np.random.default_rng(14)
    base = torch.from_numpy(np.where(rng.random((6, 900)) < 0.5, 0.0, -0.0).astype(np.float32)).to(torch.bfloat16)
    base[:3, 5::7] = -1.0
    base[3:, 5::7] = 2.0
    for f in ("open", "k50", "p", "greedy"):
        verify(base, None, 2, 4, 900, settings(6, rng, **FILTERS[f]))


@pytest.mark.gpu
@pytest.mark.parametrize("V", [300, 152064])
def test_masked_logits(V):
    """-inf, the type's lowest value, NaN of both signs and +inf among the logits."""
    rng = np.random.default_rng([15, V])
    low = torch.finfo(torch.bfloat16).min
    nan = torch.tensor(float("nan"), dtype=torch.bfloat16)
    rows = []
    for mask in (float("-inf"), low, nan, -nan):
        x = normal(rng, 1, V)[0]
        keep = torch.from_numpy(rng.random(V) < 0.05)
        keep[V // 2] = True
        rows.append(torch.where(keep, x, torch.as_tensor(mask, dtype=torch.bfloat16)))
    one = torch.full((V,), float("-inf"), dtype=torch.bfloat16)
    one[V - 1] = -3.0
    rows.append(one)
    rows.append(torch.full((V,), low, dtype=torch.bfloat16))            # all alike
    mixed = torch.full((V,), low, dtype=torch.bfloat16)
    mixed[::3] = float("-inf")
    rows.append(mixed)
    huge = normal(rng, 1, V)[0]
    huge[::11] = float("inf")
    rows.append(huge)
    steep = torch.from_numpy(rng.choice([low, low / 2, low / 256], V).astype(np.float32)).to(torch.bfloat16)
    rows.append(steep)
    base = torch.stack(rows)
    for f in ("open", "k50", "p", "greedy", "min_p", "hot"):
        verify(base, None, 3, 4, V, settings(9, rng, **FILTERS[f]))
    verify(base[-1:], None, 1, 2, V, settings(1, rng, temperature=1e38))
    verify(base[:2], None, 1, 3, V, settings(2, rng, temperature=float("inf"), top_k=20))


@pytest.mark.gpu
def test_rows_with_nothing_to_draw():
    rng = np.random.default_rng(16)
    base = torch.full((3, 1000), float("-inf"), dtype=torch.bfloat16)
    base[1] = float("nan")
    base[2, ::2] = float("nan")
    for f in ("open", "greedy", "p"):
        ids, probs = verify(base, None, 1, 4, 1000, settings(3, rng, **FILTERS[f]))
        assert (ids == 0).all() and (probs == 0).all()


@pytest.mark.gpu
def test_extreme_temperatures():
    rng = np.random.default_rng(17)
    base = normal(rng, 4, 3001)
    for t in (1e-45, 1e-30, 1e-3, 1e5, 1e27, 1e30, 3e38, float("inf")):
        verify(base, None, 1, 5, 3001, settings(4, rng, temperature=t))
    tiny = (normal(rng, 4, 3001).float() * 1e-38).to(torch.bfloat16)       # subnormal logits
    for t in (1e-38, 1.0):
        verify(tiny, None, 1, 5, 3001, settings(4, rng, temperature=t))


@pytest.mark.gpu
def test_frequencies_follow_the_softmax():
    """A grid of u over one row reproduces the probabilities to the grid's step."""
    rng = np.random.default_rng(18)
    V, rows = 40, 4096
    x = normal(rng, 1, V, 1.5)
    s = settings(rows, rng)
    s["u"] = ((np.arange(rows) + 0.5) / rows).astype(np.float32)
    ids, _ = draw(x.expand(rows, V).contiguous().cuda(), None, rows, 2, V, s)
    p = np.exp(x[0].double().numpy())
    p /= p.sum()
    assert (np.abs(np.bincount(ids, minlength=V) / rows - p) <= 1.01 / rows).all()


@pytest.mark.gpu
def test_greedy_is_the_argmax_readout():
    rng = np.random.default_rng(19)
    N, B, V = 4, 8, 32000
    base, bias = normal(rng, N * (B - 1), V).cuda(), normal(rng, N * (B - 1), V, 1.0).cuda()
    blk = torch.zeros(N, B, dtype=torch.int64, device="cuda")
    native.xpress_add_argmax_to_blk(base, bias, blk, N, B, V, V, V)
    ids, p = draw(base, bias, N, B, V, settings(N * (B - 1), rng, temperature=0.0))
    assert np.array_equal(ids, blk[:, 1:].reshape(-1).cpu().numpy()) and (p == 1).all()


@pytest.mark.gpu
def test_misaligned_rows_draw_the_same():
    rng = np.random.default_rng(20)
    N, B, V = 2, 4, 5001
    base, bias = normal(rng, 6, V).cuda(), normal(rng, 6, V, 0.5).cuda()
    s = settings(6, rng, **FILTERS["p"])
    want = draw(base, bias, N, B, V, s)
    for off, stride in ((1, V + 2), (8, 5008)):
        wide = [torch.full((6 * stride + 16,), 100.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        views = [w[off:off + 6 * stride].view(6, stride) for w in wide]
        for v, x in zip(views, (base, bias)):
            v[:, :V] = x
        got = draw(views[0], views[1], N, B, V, s)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.gpu
def test_without_probabilities_and_in_a_graph():
    rng = np.random.default_rng(21)
    N, B, V = 2, 4, 20000
    base = normal(rng, 6, V).cuda()
    s = settings(6, rng, **FILTERS["k_p_min"])
    want, _ = draw(base, None, N, B, V, s, prob=False)
    dev = {k: torch.from_numpy(v).cuda() for k, v in s.items()}
    blk = torch.zeros(N, B, dtype=torch.int64, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        native.xpress_sample_to_blk(base, None, blk, dev["temperature"], dev["top_k"], dev["top_p"],
                                    dev["min_p"], dev["u"], N, B, V, V)
    for _ in range(3):
        blk.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(blk[:, 1:].reshape(-1).cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("filters", ["open", "greedy", "k_p_min", "hot", "cold"])
@pytest.mark.parametrize("rows,V", [(33, 152064), (32, 98304), (31, 98303), (2, 1000003), (1, 3000001)])
def test_either_side_of_the_split_into_parts(filters, rows, V):
    """With a bias, up to 32 rows of 98304 to 2 million logits go in parts, others do not."""
    say("sample sides %s %d %d" % (filters, rows, V))
    rng = np.random.default_rng([rows, V])
    base, bias = normal(rng, rows, V), normal(rng, rows, V, 0.5)
    s = settings(rows, rng, **FILTERS[filters])
    verify(base, bias, rows, 2, V, s)
    verify(base, None, rows, 2, V, s)


@pytest.mark.gpu
def test_whole_rows_and_parts_draw_the_same():
    """The same rows among more than 32, and alone; also where the workspace is not to be had."""
    rng = np.random.default_rng(22)
    rows, V = 40, 100000
    base, bias = normal(rng, rows, V), normal(rng, rows, V, 0.5).cuda()
    base[3, ::2] = float("-inf")
    base[4, ::3] = torch.finfo(torch.bfloat16).min
    base[5] = (base[5].float() * 4).round().to(torch.bfloat16)        # ties
    base[6, 7] = float("inf")
    s = settings(rows, rng)
    s["temperature"] = rng.choice([0.0, 0.5, 1.0, 3.0, 20.0, 100.0], rows).astype(np.float32)
    s["top_p"] = rng.choice([0.5, 0.9, 1.0], rows).astype(np.float32)
    s["min_p"] = rng.choice([0.0, 0.01], rows).astype(np.float32)
    s["top_k"] = rng.choice([0, 5, 700], rows).astype(np.int32)
    bias[5] = 0
    dev = base.cuda()
    ids, p = draw(dev, bias, rows, 2, V, s)
    few = {k: v[:20].copy() for k, v in s.items()}
    native.xpress_release()
    got, q = draw(dev[:20], bias[:20], 20, 2, V, few)
    assert np.array_equal(got, ids[:20]) and np.array_equal(q, p[:20])
    native.xpress_release()
    native.xpress_set_workspace_limit(1 << 10)
    try:
        got, q = draw(dev[:20], bias[:20], 20, 2, V, few)
    finally:
        native.xpress_set_workspace_limit(0)
    assert np.array_equal(got, ids[:20]) and np.array_equal(q, p[:20])


@pytest.mark.gpu
@pytest.mark.parametrize("reserve", [False, True])
def test_parts_in_a_graph(reserve):
    rng = np.random.default_rng(23)
    N, B, V = 1, 4, 100000
    base, bias = normal(rng, 3, V).cuda(), normal(rng, 3, V, 0.5).cuda()
    s = settings(3, rng, **FILTERS["p"])
    want, _ = draw(base, bias, N, B, V, s)
    dev = {k: torch.from_numpy(v).cuda() for k, v in s.items()}
    blk = torch.zeros(N, B, dtype=torch.int64, device="cuda")
    stream = torch.cuda.Stream()
    if reserve:
        native.xpress_sample_reserve(N, B, V, stream=stream)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        native.xpress_sample_to_blk(base, bias, blk, dev["temperature"], dev["top_k"], dev["top_p"],
                                    dev["min_p"], dev["u"], N, B, V, V, V)
    for _ in range(3):
        blk.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(blk[:, 1:].reshape(-1).cpu().numpy(), want)
        draw(base, bias, N, B, V, s)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [3000, 152064])
def test_rows_past_32_bits(V):
    """Rows 2^31 elements apart."""
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GiB of GPU memory")
    rng = np.random.default_rng([24, V])
    stride = 2 ** 31 + 8
    rows = normal(rng, 3, V)
    base = torch.empty(2 * stride + V, dtype=torch.bfloat16, device="cuda")
    for r in range(3):
        base[r * stride:r * stride + V] = rows[r].cuda()
    s = settings(3, rng, **FILTERS["p"])
    want = draw(rows.cuda(), None, 1, 4, V, s)
    got = draw(base.as_strided((3, V), (stride, 1)), None, 1, 4, V, s)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.gpu
def test_two_streams_at_once():
    """Rows in parts on two streams, each with a workspace of its own."""
    rng = np.random.default_rng(25)
    V = 120000
    bias = normal(rng, 6, V, 0.5).cuda()
    sets = []
    for i in range(2):
        base = normal(rng, 6, V)
        s = settings(6, rng, **FILTERS["k_p_min"])
        sets.append((base.cuda(), {k: torch.from_numpy(v).cuda() for k, v in s.items()},
                     draw(base.cuda(), bias, 2, 4, V, s)[0]))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        out = [torch.zeros(2, 4, dtype=torch.int64, device="cuda") for _ in sets]
        torch.cuda.synchronize()
        for (base, d, _), blk, stream in zip(sets, out, streams):
            native.xpress_sample_to_blk(base, bias, blk, d["temperature"], d["top_k"], d["top_p"], d["min_p"],
                                        d["u"], 2, 4, V, V, V, stream=stream)
        torch.cuda.synchronize()
        for (_, _, want), blk in zip(sets, out):
            assert np.array_equal(blk[:, 1:].reshape(-1).cpu().numpy(), want)


@pytest.mark.gpu
def test_every_wave_agrees_on_the_segment_of_the_draw():
    """Rows counted again over all values (a tiny logit, a high temperature, one of 2^16) whose
    searches end in the window that the bins hold already, so that no barrier but the searches' own
    stands between the last one's answer and its use."""
    rng = np.random.default_rng(26)
    rows, V = 96, 4099
    base = normal(rng, rows, V)
    base[0::3, 3] = 2.0 ** -40
    base[1::3, 5] = -2.0 ** 17
    s = settings(rows, rng)
    s["temperature"] = np.where(np.arange(rows) % 3 == 0, 1.0, 50.0).astype(np.float32)
    s["top_k"] = rng.choice([0, 9, 1000], rows).astype(np.int32)
    s["top_p"] = rng.choice([0.3, 0.95, 1.0], rows).astype(np.float32)
    s["min_p"] = rng.choice([0.0, 0.05], rows).astype(np.float32)
    want = verify(base, None, 32, 4, V, s)[0]
    for _ in range(8):
        assert np.array_equal(draw(base.cuda(), None, 32, 4, V, s)[0], want)


@pytest.mark.gpu
def test_errors_of_others_are_not_cleared():
    """A HIP error that the caller has pending is reported by the launch, whether the rows would
    have gone in parts or not; an allocation that failed in the library leaves none behind."""
    import ctypes
    rng = np.random.default_rng(27)
    V = 100000
    base, bias = normal(rng, 1, V).cuda(), normal(rng, 1, V, 0.5).cuda()
    s = settings(1, rng)
    lib = native.load()
    lib.hipMalloc.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_size_t]
    none = ctypes.c_void_p()
    native.xpress_release()
    native.xpress_set_workspace_limit(1 << 10)
    try:
        want = draw(base, bias, 1, 2, V, s)
        dev = {k: torch.from_numpy(v).cuda() for k, v in s.items()}
        blk = torch.zeros(1, 2, dtype=torch.int64, device="cuda")
        for b in (bias, None):
            assert lib.hipMalloc(ctypes.byref(none), 1 << 60) != 0
            assert lib.hipPeekAtLastError() != 0
            with pytest.raises(native.XpressError) as e:
                native.xpress_sample_to_blk(base, b, blk, dev["temperature"], dev["top_k"], dev["top_p"],
                                            dev["min_p"], dev["u"], 1, 2, V, V, V)
            assert e.value.status == native.XPRESS_EHIP
            assert lib.hipPeekAtLastError() == 0
        got = draw(base, bias, 1, 2, V, s)
    finally:
        native.xpress_set_workspace_limit(0)
    assert np.array_equal(got[0], want[0])
    with pytest.raises(native.XpressError) as e:
        native.xpress_latent_reserve(1 << 22, 16, 64, 8192)      # 1 TB
    assert e.value.status == native.XPRESS_ENOMEM
    assert lib.hipPeekAtLastError() == 0
    assert np.array_equal(draw(base, bias, 1, 2, V, s)[0], want[0])


@pytest.mark.gpu
def test_more_rows_than_a_grid_has_threads_for():
    """2^23 rows of 512 threads are 2^32."""
    if torch.cuda.mem_get_info()[0] < 4 << 30:
        pytest.skip("needs 4 GiB of GPU memory")
    say("sample rows past a grid")
    rng = np.random.default_rng(28)
    rows, V = 2 ** 23 + 1000, 3
    base = normal(rng, rows, V).cuda()
    s = settings(rows, rng)
    s["top_k"] = rng.choice([0, 1, 2], rows).astype(np.int32)
    ids, probs = draw(base, None, rows, 2, V, s)
    for part in (slice(0, 5000), slice(2 ** 21 - 2000, 2 ** 21 + 2000), slice(rows - 5000, rows)):
        few = {k: v[part].copy() for k, v in s.items()}
        got, p = draw(base[part], None, len(few["u"]), 2, V, few)
        assert np.array_equal(got, ids[part]) and np.array_equal(p, probs[part])
