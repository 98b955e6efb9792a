"""The drafts' operators at sizes past one grid or one pass of a workgroup: whole numbers and bits
equal to the definition's or to a small call's."""
import numpy as np
import pytest
import torch

import drafts_ref as ref
from gpu_util import say
from vocab_wide_add_amd import native


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x).astype(np.int32))).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("N,M", [(65536, 65536), (3, 65536), (65536, 1)])
def test_forks_of_most_rows(N, M):
    say("fork %d %d" % (N, M))
    rng = np.random.default_rng(M)
    pages, width, page = 3 * N + 40000, 3, 4
    table = rng.permutation(pages)[:3 * N].reshape(N, 3)
    table[rng.random((N, 3)) < 0.1] = -1
    refs = np.bincount(table[table >= 0], minlength=pages)
    lens, src = rng.integers(-1, 14, N), rng.integers(-3, N + 3, M)
    new_refs, new_table = torch.empty(pages, dtype=torch.int32, device="cuda"), i32(np.zeros((M, 3)))
    copies, missing = i32(np.zeros((M, 3))), i32([7])
    native.xpress_kv_fork(i32(refs), i32(table), i32(lens), i32(src), new_refs, new_table, copies, page, missing=missing)
    torch.cuda.synchronize()
    want = ref.fork(refs, table, lens, src, page)
    for x, y in zip((new_refs, new_table, copies), want):
        assert np.array_equal(x.cpu().numpy(), y)
    assert int(missing) == want[3]


@pytest.mark.gpu
def test_pages_of_many_sequences():
    """More sequences than a grid's second dimension has, each with a page of its own at first."""
    say("70001 sequences")
    N, width, page, Hk, D = 70001, 3, 4, 1, 16
    pages = 2 * N + 11
    rng = np.random.default_rng(3)
    have, want = rng.integers(0, 5, N), rng.integers(0, 14, N)
    table = np.full((N, width), -1)
    table[:, 0] = np.where(have > 0, rng.permutation(pages)[:N], -1)
    refs = np.bincount(table[table >= 0], minlength=pages)
    r, t, missing = i32(refs), i32(table), i32([3])
    native.xpress_kv_grow(r, t, i32(have), i32(want), page, missing=missing)
    torch.cuda.synchronize()
    refs, table, lack = ref.grow(refs, table, have, want, page)
    assert np.array_equal(r.cpu().numpy(), refs) and np.array_equal(t.cpu().numpy(), table) and int(missing) == lack
    # paths of two nodes: 2 and 3 go to 0 and 1
    k = torch.arange(pages * page, device="cuda", dtype=torch.int32).view(pages, Hk, page, 1).expand(-1, -1, -1, D // 4)
    k = k.contiguous().view(torch.float8_e4m3fn)
    v = k.clone()
    before = k.view(torch.int32).cpu()
    native.xpress_kv_compact(k, v, t, i32(np.zeros(N)), i32([2, 3]).expand(N, 2), i32(np.full(N, 2)))
    torch.cuda.synchronize()
    after = before.clone()
    own = torch.from_numpy(table[:, 0][table[:, 0] >= 0].astype(np.int64))
    after[own, :, :2] = before[own, :, 2:]
    assert torch.equal(k.view(torch.int32).cpu(), after) and torch.equal(v.view(torch.int32).cpu(), after)
    # copies: every page to the one behind the first half
    lines = np.stack([np.arange(N), np.arange(N) + N, rng.integers(-1, 6, N)], 1)
    native.xpress_kv_copy(k, v, i32(lines))
    torch.cuda.synchronize()
    was = after.clone()
    for n in range(5):
        at = torch.from_numpy(np.flatnonzero(np.clip(lines[:, 2], 0, 4) == n))
        after[at + N, :, :n] = was[at, :, :n]
    assert torch.equal(k.view(torch.int32).cpu(), after) and torch.equal(v.view(torch.int32).cpu(), after)
    native.xpress_kv_free(r, t, i32(have), page, window=3, sinks=1)
    torch.cuda.synchronize()
    refs, table = ref.free(refs, table, have, page, 3, 1)
    assert np.array_equal(r.cpu().numpy(), refs) and np.array_equal(t.cpu().numpy(), table)


@pytest.mark.gpu
def test_beams_of_more_rows_than_one_launch_takes():
    say("2^22 + 3 rows")
    N, V = 2 ** 22 + 3, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    base = (torch.randn(N, V, generator=g, device="cuda") * 3).to(torch.bfloat16)
    scores = -torch.rand(N, generator=g, device="cuda")
    best = torch.empty(N, 1, device="cuda")
    rows, ids = torch.empty(N, 1, dtype=torch.int32, device="cuda"), torch.empty(N, 1, dtype=torch.int64, device="cuda")
    native.xpress_beam_select(base, None, scores, best, rows, ids, N, 1, V, 1, V)
    torch.cuda.synchronize()
    z = base.double()
    assert torch.equal(rows[:, 0], torch.arange(N, device="cuda", dtype=torch.int32))
    assert torch.equal(ids[:, 0], (z == z.max(1, keepdim=True)[0]).int().argmax(1))     # the lowest id
    want = scores.double() + z.max(1)[0] - torch.logsumexp(z, 1)
    # the sum's error, and half a step of the result
    assert ((best[:, 0].double() - want).abs() <= 6e-7 + 2.0 ** -24 * want.abs()).all()
    old = torch.arange(N, device="cuda", dtype=torch.int32)
    new = torch.empty_like(old)
    native.xpress_beam_reorder([(old, new)], rows.view(-1).flip(0).contiguous())
    torch.cuda.synchronize()
    assert torch.equal(new, old.flip(0))


@pytest.mark.gpu
@pytest.mark.parametrize("Q,G", [(1, 1), (9, 8)])     # 1 and 72 rows a head
@pytest.mark.parametrize("form", ["tree", "sinks"])
def test_attention_of_more_workgroups_than_one_launch_takes(form, Q, G):
    """Sequences that repeat a few: their rows are the few's, to the bit."""
    if torch.cuda.get_device_properties(0).total_memory < 40 * 2 ** 30:
        pytest.skip("needs 40 GiB of GPU memory")
    say("more workgroups %s %d" % (form, Q))
    N, few, Hk, D, page = 2 ** 19 + 11, 7, 8, 8, 16
    g = torch.Generator(device="cuda").manual_seed(2)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    k, v, q = normal(few, Hk, page, D), normal(few, Hk, page, D), normal(few, Q, Hk * G, D)
    lens = torch.tensor([0, 1, 5, 9, 12, 15, 16], dtype=torch.int32, device="cuda")
    words = torch.randint(0, 512, (few, Q, 1), generator=g, device="cuda").to(torch.int32)
    table = torch.arange(few, dtype=torch.int32, device="cuda")[:, None]

    def go(at):
        out = torch.full((len(at), Q, Hk * G, D), 9.0, dtype=torch.bfloat16, device="cuda")
        args = [q[at], k, v, table[at], lens[at]]
        if form == "tree":
            native.xpress_tree_attention(*args, words[at], out, page, window=6, sinks=2)
        else:
            native.xpress_sink_attention(*args, out, page, 6, 2)
        torch.cuda.synchronize()
        return out
    want = go(torch.arange(few, device="cuda"))
    assert torch.isfinite(want.float()).all() and (want[0] == 0).all() and (want[3] != 9).all()
    at = torch.arange(N, device="cuda") % few
    got = go(at)
    for n in range(few):
        assert (got[n::few] == want[n]).all()
