"""The beam search example where it cannot go on, as pages run out or tokens would pass the
buffers, and started again."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def made(pages=None):
    import beams
    return beams.Beams(3, 3, 80, window=24, sinks=3, page=8, hq=8, hk=2, dim=64, vocab=1000, pages=pages)


def prompts(seed, lens=(40, 1, 17)):
    r = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 1000, (n,), generator=r).tolist() for n in lens]


@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
def test_a_search_that_lacked_pages_says_so(graph):
    """Nine pages hold the prompts and the first parting of their beams; the first token of
    the second sequence's beams needs more.  Steps after that lack none."""
    d = made(9)
    d.start(prompts(7))
    with pytest.raises(RuntimeError, match="pages"):
        d.search(4, graph=graph)
    with pytest.raises(RuntimeError, match="pages"):
        made(6).start(prompts(7))
    d = made()
    d.start(prompts(7))
    d.search(4, graph=graph)


@pytest.mark.gpu
def test_a_second_search_is_as_a_fresh_one():
    a, b = made(), made()
    a.start(prompts(7))
    a.search(12)
    for d in (a, b):
        d.start(prompts(8, (33, 9, 50)))
    got, want = a.search(8), b.search(8)
    torch.cuda.synchronize()
    for row, n in enumerate((33, 9, 50)):
        here = slice(3 * row, 3 * row + 3)
        assert torch.equal(got[0][here, :n + 8], want[0][here, :n + 8])
    assert torch.equal(got[1], want[1])


@pytest.mark.parametrize("steps", [-2, 0, 1, 7, 10, 1000])
def test_steps_past_the_buffers_are_refused_before_any_gpu_call(steps):
    import beams
    d = beams.Beams.__new__(beams.Beams)
    d.max_len, d.longest = 80, 72        # room for 8
    for graph in (False, True):
        with pytest.raises(ValueError, match="steps"):
            d.search(steps, graph=graph)
    assert d.longest == 72


@pytest.mark.parametrize("lens", [(3, 4), (3, 4, 0), (3, 81, 4), (1, 2, 3, 4)])
def test_prompts_that_do_not_fit_are_refused_before_any_gpu_call(lens):
    import beams
    d = beams.Beams.__new__(beams.Beams)
    d.max_len, d.seqs = 80, 3
    with pytest.raises(ValueError, match="prompts"):
        d.start(prompts(1, lens))


@pytest.mark.gpu
def test_a_search_up_to_the_last_place():
    d = made()
    d.start(prompts(7, (70, 80 - 6, 1)))
    d.search(6)
    torch.cuda.synchronize()
    with pytest.raises(ValueError, match="steps"):
        d.search(2)


@pytest.mark.gpu
def test_the_pool_holds_any_parting_of_full_rows():
    """Nine rows of 79 tokens, no page shared, of which each sequence's first goes on as three."""
    from vocab_wide_add_amd import native
    d = made()
    lens = torch.full((9,), 79, dtype=torch.int32, device="cuda")
    native.xpress_kv_grow(d.refs[0], d.tables[0], torch.zeros_like(lens), lens, 8, missing=d.missing[0])
    src = (torch.arange(9, device="cuda") // 3 * 3).to(torch.int32)
    native.xpress_kv_fork(d.refs[0], d.tables[0], lens, src, d.refs[1], d.tables[1], d.copies, 8, missing=d.missing[1])
    assert d.missing.tolist() == [[0], [0]] and int((d.copies[:, 1] >= 0).sum()) == 6
