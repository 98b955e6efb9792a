"""xpress_beam_select against the definition in 64 bits, and xpress_beam_reorder.

Rows and ids are equal where the definition's neighbours in the order lie further apart
than the scores' error; inputs are drawn so, or tie exactly.  A score is a sum in 64
bits with the log of a sum S of terms 2^x, each off by at most 2 steps of its fp32 value
(2^-22, the hardware's exponential), and a rest of (z - m)^2 2^-35 at most, under the
weight exp(z - m) at most 2^-34; a thread sums up to 256 of them in fp32 (256 * 2^-24
at most, relatively).  So |log S| is off by at most 2^-22 + 2^-16 + 2^-34 < 2^-15.9,
and the result is rounded once (2^-24)."""
import numpy as np
import pytest
import torch

import drafts_ref as ref
from gpu_util import say
from vocab_wide_add_amd import native

OFF = 2.0 ** -15.9


def summed(base, bias):
    """float64 logits of bf16 tensors."""
    if bias is None:
        return base.double().numpy()
    return (base.double() + bias.double()).float().to(torch.bfloat16).double().numpy()


def call(base, bias, scores, N, beams, V, K, stride=None, off=0, stream=None):
    stride = stride or V
    rows = N * beams

    def up(x):
        if x is None:
            return None
        flat = torch.full((off + rows * stride,), float("nan"), dtype=torch.bfloat16, device="cuda")
        flat[off:].view(rows, stride)[:, :V] = x.cuda()
        return flat[off:].view(rows, stride)
    best = torch.full((N, K), 7.0, device="cuda")
    out_rows = torch.full((N, K), 7, dtype=torch.int32, device="cuda")
    ids = torch.full((N, K), 7, dtype=torch.int64, device="cuda")
    native.xpress_beam_select(up(base), up(bias), scores.cuda(), best, out_rows, ids, N, beams, V, K, stride, stride,
                              stream=stream)
    torch.cuda.synchronize()
    return best.double().cpu().numpy(), out_rows.cpu().numpy(), ids.cpu().numpy()


def verify(base, bias, scores, N, beams, K, **kw):
    V = base.shape[1]
    best, rows, ids = call(base, bias, scores, N, beams, V, K, **kw)
    want = ref.beams(summed(base, bias), scores.double().numpy(), N, beams, K)
    assert np.array_equal(rows, want[1]), (rows, want[1])
    assert np.array_equal(ids, want[2])
    there = want[1] >= 0
    assert np.isneginf(best[~there]).all()
    assert (np.abs(best - want[0])[there] <= OFF + 2.0 ** -24 * np.abs(want[0][there])).all()
    return best, rows, ids


def drawn(seed, rows, V, bias, sigma=4.0):
    g = torch.Generator().manual_seed(seed)
    base = (torch.randn(rows, V, generator=g) * sigma).to(torch.bfloat16)
    b = (torch.randn(rows, V, generator=g) * 0.5).to(torch.bfloat16) if bias else None
    return base, b, -torch.rand(rows, generator=g) * 10


def settled(base, bias, scores, N, beams, K):
    """Scores moved so that no two neighbours of different rows lie closer than 1e-3."""
    z = summed(base, bias)
    scores = scores.clone()
    for _ in range(50):
        best, rows, _ = ref.beams(z, scores.double().numpy(), N, beams, K + 1)
        close = (np.abs(np.diff(best)) < 1e-3) & (np.diff(rows) != 0)
        if not close.any():
            return scores
        scores[torch.from_numpy(np.unique(rows[:, 1:][close]))] -= 0.0131
    raise AssertionError("no such scores")


CASES = [
    # N, beams, V, K, bias, stride, off
    (1, 1, 1, 1, False, None, 0), (1, 1, 5, 8, False, None, 0), (2, 3, 7, 4, True, None, 0),
    (3, 4, 1000, 8, False, None, 0), (2, 8, 4099, 16, True, 4104, 0), (1, 4, 50000, 8, False, None, 0),
    (5, 2, 32000, 2, True, 32011, 0), (1, 1, 152064, 128, True, None, 0), (2, 5, 9000, 5, False, None, 1),
    (1, 16, 20000, 32, False, None, 8), (4, 1, 300, 128, True, None, 0), (1, 2, 140001, 7, True, 140008, 0),
    (70, 8, 600, 8, False, None, 0), (1, 300, 64, 100, False, None, 0), (2, 2, 131073, 3, False, None, 0),
    (40, 16, 4500, 3, True, None, 0), (1, 600, 40, 8, False, None, 0), (1, 1100, 3, 20, True, None, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_64_bits(case):
    N, beams, V, K, bias, stride, off = CASES[case]
    say("beams %d" % case)
    base, b, scores = drawn(case, N * beams, V, bias)
    scores = settled(base, b, scores, N, beams, K)
    verify(base, b, scores, N, beams, K, stride=stride, off=off)


@pytest.mark.gpu
@pytest.mark.parametrize("V,K", [(9000, 5), (50000, 64), (300, 128)])
def test_ties_go_to_the_lower_row_then_the_lower_id(V, K):
    """Equal rows and few distinct values: whole runs of equal logits."""
    g = torch.Generator().manual_seed(V)
    one = torch.randint(0, 4, (1, V), generator=g).to(torch.bfloat16)
    verify(one.expand(6, V), None, torch.zeros(6), 2, 3, K)
    verify(torch.full((6, V), -2.5, dtype=torch.bfloat16), None, torch.zeros(6), 2, 3, K)
    # more equal candidates, and more lists, than are ranked by counting
    verify(one.expand(300, V), None, torch.zeros(300), 1, 300, K)
    verify(one.expand(600, V), None, torch.zeros(600), 1, 600, K)
    # -0 equals +0
    zero = torch.zeros(2, V, dtype=torch.bfloat16)
    zero[:, ::2] = -0.0
    verify(zero, None, torch.zeros(2), 1, 2, K)
    # the largest ones all in one place of the order of the work
    at = torch.arange(V)
    verify(torch.where(at % 4096 < 8, 5.0 + at / 8192, -at / 1000.0)[None].to(torch.bfloat16), None,
           torch.zeros(1), 1, 1, K)
    verify((at / 64.0)[None].to(torch.bfloat16), None, torch.zeros(1), 1, 1, K)
    verify((-at / 64.0)[None].to(torch.bfloat16), None, torch.zeros(1), 1, 1, K)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [40, 5000, 70000])
def test_masked_logits_and_candidates_that_run_out(V):
    low = float(torch.finfo(torch.bfloat16).min)
    base, _, _ = drawn(V, 8, V, False)
    base[0] = float("-inf")
    base[1] = float("nan")
    base[2, 3:] = float("-inf")
    base[3, 5:] = low                       # the type's lowest value is a logit like others
    base[4, 1:] = float("nan")
    base[5, ::2] = float("-inf")
    base[6, 7], base[6, 9] = float("inf"), float("inf")
    base[7] = low
    scores = settled(base, None, -torch.arange(8) * 0.7, 1, 8, 12)
    verify(base, None, scores, 1, 8, 12)
    verify(base[:3], None, scores[:3], 1, 3, 12)          # three candidates in all
    verify(base[:2], None, scores[:2], 2, 1, 5)           # none
    verify(base[6:], None, scores[6:], 2, 1, 9)
    best, rows, ids = verify(base[6:7], None, torch.zeros(1), 1, 1, 4)
    assert ids[0].tolist() == [7, 9, -1, -1] and np.allclose(best[0, :2], -np.log(2.0))


@pytest.mark.gpu
@pytest.mark.parametrize("at", [0.0, 100.0, -100.0, 8000.0, -8190.0, 8192.0, -9000.0, 1e6, -1e6, 3e38, -3e38])
def test_logits_of_any_size(at):
    """Rows around one value: steps of its type decide how many logits count."""
    g = torch.Generator().manual_seed(3)
    base = (at + torch.randn(3, 6000, generator=g) * 3).to(torch.bfloat16)
    scores = torch.tensor([0.0, -0.3, -0.71])
    best, rows, ids = call(base, None, scores, 3, 1, 6000, 6)
    want = ref.beams(base.double().numpy(), scores.double().numpy(), 3, 1, 6)
    assert np.array_equal(ids, want[2]) and np.array_equal(rows, want[1])
    assert (np.abs(best - want[0]) <= OFF + 2.0 ** -24 * np.abs(want[0])).all()
    # one that towers above the others, some of them far below
    base[:, 77] = base.float().abs().max() * 1.5 if at else 1e30
    base[1, 100:200] = -3e38
    verify(base, None, scores, 3, 1, 1)


@pytest.mark.gpu
def test_beams_that_are_not_in_use():
    base, bias, scores = drawn(11, 6, 3000, True)
    scores = settled(base, bias, scores, 2, 3, 6)
    for bad in (float("-inf"), float("nan"), float("inf")):
        s = scores.clone()
        s[1] = s[3] = s[4] = s[5] = bad
        best, rows, ids = verify(base, bias, s, 2, 3, 6)
        assert (rows[1] == -1).all() and not (rows == 1).any()


@pytest.mark.gpu
def test_a_row_gives_the_same_whatever_stands_beside_it():
    """Equal rows have equal scores to the bit, at any place."""
    base, bias, _ = drawn(12, 1, 20011, True)
    rows = 24
    best, r, ids = call(base.expand(rows, -1), bias.expand(rows, -1), torch.full((rows,), -1.5), rows, 1, 20011, 8)
    assert (best == best[0]).all() and (ids == ids[0]).all()
    assert np.array_equal(r, np.arange(rows)[:, None].repeat(8, 1))


@pytest.mark.gpu
def test_two_streams_and_a_replayed_graph():
    base, bias, scores = drawn(13, 8, 30000, True)
    scores = settled(base, bias, scores, 2, 4, 4)
    want = ref.beams(summed(base, bias), scores.double().numpy(), 2, 4, 4)
    d = [base.cuda(), bias.cuda(), scores.cuda()]

    def outs():
        return (torch.zeros(2, 4, device="cuda"), torch.zeros(2, 4, dtype=torch.int32, device="cuda"),
                torch.zeros(2, 4, dtype=torch.int64, device="cuda"))

    def go(o, stream=None):
        native.xpress_beam_select(*d, *o, 2, 4, 30000, 4, 30000, 30000, stream=stream)
    streams, all_outs = [torch.cuda.Stream() for _ in range(2)], [outs() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, o in zip(streams, all_outs):
            go(o, st)
    torch.cuda.synchronize()
    for o in all_outs:
        assert np.array_equal(o[1].cpu().numpy(), want[1]) and np.array_equal(o[2].cpu().numpy(), want[2])
    stream, graph, o = torch.cuda.Stream(), torch.cuda.CUDAGraph(), outs()
    native.xpress_beam_select_reserve(2, 4, 30000, 4, stream=stream)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        go(o)
    for _ in range(3):
        for x in o:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(o[1].cpu().numpy(), want[1]) and np.array_equal(o[2].cpu().numpy(), want[2])
        go(outs())
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        o[0].add_(0)
        with pytest.raises(native.XpressError) as e:
            go(o)
    assert e.value.status == native.XPRESS_ECAPTURE


@pytest.mark.gpu
@pytest.mark.parametrize("shape,dtype", [((5,), torch.int64), ((3, 7), torch.bfloat16), ((), torch.float32),
                                         ((1001,), torch.uint8), ((4, 4096), torch.float16), ((2, 0), torch.int32),
                                         ((33,), torch.int16)])
def test_states_follow_their_beams(shape, dtype):
    g = torch.Generator().manual_seed(2)
    N, src = 7, torch.tensor([3, 3, -1, 0, 6, 7, 2 ** 31 - 1, 5, 1], dtype=torch.int32)
    old = torch.randint(0, 100, (N,) + shape, generator=g).to(dtype)
    wide = torch.randint(0, 100, (N, 2) + shape, generator=g).to(dtype)
    out = [torch.full((9,) + shape, 9, dtype=dtype, device="cuda") for _ in range(11)]
    olds = [old.cuda() for _ in range(10)] + [wide.cuda()[:, 1]]
    native.xpress_beam_reorder(list(zip(olds, out)), src.cuda())
    torch.cuda.synchronize()
    for o, x in zip([old] * 10 + [wide[:, 1]], out):
        for m, n in enumerate(src.tolist()):
            want = o[n] if 0 <= n < N else torch.zeros(shape, dtype=dtype)
            assert torch.equal(x[m].cpu(), want)


@pytest.mark.gpu
def test_one_state_shared_by_all_rows_and_rows_with_gaps():
    one = torch.arange(24, device="cuda").float().view(1, 24).expand(5, 24)
    wide = torch.full((4, 40), -1.0, device="cuda")
    native.xpress_beam_reorder([(one, wide[:, :24])], torch.tensor([[4, 9], [0, 2]], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert (wide[:, 24:] == -1).all() and (wide[1, :24] == 0).all()
    assert torch.equal(wide[[0, 2, 3], :24].cpu(), one[:3].cpu())
