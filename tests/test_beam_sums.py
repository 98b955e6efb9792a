"""The sums of exponentials behind xpress_beam_select's scores, where their roundings would not
average out: rows of one value, rows in which a few logits tower over a long tail, and rows
whose largest logits come late.  Scores are given so that the results lie near zero, where the
last rounding is small.

A row's sum of 2^(z L - r), L = log2(e) = Lh + Ll with Lh of 15 bits, is off, relatively, by

* 2^-23 at most for the hardware's exponential (one step of its result);
* the rounding of z Lh - r, ln 2 times half a step: r is at most half above the thread's largest
  z Lh and at most 8 below.  Below 8 in magnitude that is 2^-22 ln 2.  Arguments from -8 to -16
  have half steps of 2^-21, and 255 such terms are less than 1 beside one of 2^-1/2 or more:
  .59 of the sum, .59 2^-21 ln 2 < 2^-22; those below -16 are less than 2^-8 of it;
* three roundings of sums of pairs, 3 2^-24 (the eights are added in 64 bits);
* the factor for Ll: eight roundings of sum y z, at most 2^13 2^-17.6 ln 2 8 2^-24 < 2^-25.

So log sum exp is off by less than (2 + 4 + 3 + .5) 2^-24 < 6e-7."""
import numpy as np
import pytest
import torch

from gpu_util import say
from vocab_wide_add_amd import native

OFF = 9.5 * 2.0 ** -24
V = 131072   # one part of a row, 256 logits a thread, where rows are many


def rows_of(n):
    """float32 [kinds, n] of bf16 values."""
    at = np.arange(n)
    first = at < 4096                       # every thread's first logits of a long row
    lead = at == 0
    kinds = [np.full(n, 7.75), np.full(n, 0.625), np.full(n, -0.30078125), np.full(n, 3.0),
             np.where(lead, 0.0, -16.75), np.where(first, 0.0, -16.75), np.where(lead, 8.0, -0.30078125),
             np.where(first, -8.3125, 0.703125), np.where(at < 8, -8191.0, 0.703125),
             np.where(at % 8 == 3, 1.0078125, -0.99609375), np.where(lead, 8191.0, 8160.0),
             np.where(at >= n - 9, 0.0, -12.0625), -at / n * 20.0]
    return torch.from_numpy(np.stack(kinds)).to(torch.bfloat16)


def log_sums(z):
    z = z.double().numpy()
    top = z.max(1, keepdims=True)
    return top[:, 0], np.log(np.exp(z - top).sum(1))     # (sums of 2^17 terms, pairwise: 2^-48)


def select(base, bias, scores, N, beams, K, stride, n=None):
    n = n or base.shape[1]
    best = torch.empty(N, K, device="cuda")
    rows = torch.empty(N, K, dtype=torch.int32, device="cuda")
    ids = torch.empty(N, K, dtype=torch.int64, device="cuda")
    native.xpress_beam_select(base, bias, scores, best, rows, ids, N, beams, n, K, stride, stride)
    torch.cuda.synchronize()
    return best, rows, ids


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 7, 512])
@pytest.mark.parametrize("form", ["vectors", "bias", "one by one"])
@pytest.mark.parametrize("n", [V, V - 3, 5000])
def test_sums_of_rows_whose_roundings_agree(n, form, rows):
    say("sums %d %s %d" % (n, form, rows))
    z = rows_of(n)
    kinds = len(z)
    _, logs = log_sums(z)
    which = np.arange(max(rows, kinds)) % kinds
    stride = n + 8 - n % 8 + (1 if form == "one by one" else 0)
    scores = torch.from_numpy(logs.astype(np.float32))
    want = scores.double().numpy() - logs
    for r0 in range(0, len(which), rows):
        here = torch.from_numpy(which[r0:r0 + rows])
        m = len(here)
        base = torch.full((m, stride), float("nan"), dtype=torch.bfloat16, device="cuda")
        base[:, :n] = z.cuda()[here.cuda()]
        bias = torch.zeros_like(base) if form == "bias" else None
        best, _, _ = select(base, bias, scores[here].cuda(), m, 1, 1, stride, n)
        off = np.abs(best[:, 0].double().cpu().numpy() - want[here])
        assert (off <= OFF + 2.0 ** -24 * np.abs(want[here])).all(), [
            (int(k), float(o)) for k, o in zip(here[:kinds], off[:kinds])]


@pytest.mark.gpu
def test_a_flat_and_a_peaked_beam_keep_their_order():
    """The flat beam's candidates stand 5e-6 above the peaked one's."""
    z = rows_of(V)[[1, 4]]
    _, logs = log_sums(z)
    flat = np.float32(logs[0])
    above = np.float64(flat) - logs[0]
    peaked = np.float32(above - 5e-6 + logs[1])
    assert 4e-6 < above - (np.float64(peaked) - logs[1]) < 6e-6
    N = 256
    scores = torch.tensor([flat, peaked], device="cuda").repeat(N)
    best, rows, ids = select(z.cuda().repeat(N, 1), None, scores, N, 2, 2, V)
    # two of the flat beam's, by the lower id, then the peaked one's
    assert torch.equal(rows.cpu(), (2 * torch.arange(N, dtype=torch.int32))[:, None].expand(N, 2))
    assert ids.tolist() == [[0, 1]] * N
    best, rows, ids = select(z[[1, 0]].cuda().repeat(N, 1), None, scores.view(N, 2).flip(1).reshape(-1), N, 2, 1, V)
    assert torch.equal(rows.cpu()[:, 0], 2 * torch.arange(N, dtype=torch.int32) + 1)
