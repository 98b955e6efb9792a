"""The sparse attention where its arguments lie otherwise than in the plainest call: rows that are
not on 16 bytes, outputs with gaps, no lse, scales of one kind, lengths out of range, pages past
2^32 bytes, a prompt under a window, two streams at once.  Tolerances as in
test_sparse_attention."""
import numpy as np
import pytest
import torch

import drafts_ref as ref
import test_sparse_attention as base
from gpu_util import say
from vocab_wide_add_amd import native

FEW, MANY = 3, 40      # nodes: 6 and 80 rows a head of 2


def odd(q, gap=3):
    """The same values where rows begin at any multiple of 2 bytes."""
    N, Q, H, D = q.shape
    flat = torch.zeros(N * Q * (H * (D + gap) + 1) + 1, dtype=q.dtype)
    view = flat[1:].as_strided(q.shape, (Q * (H * (D + gap) + 1), H * (D + gap) + 1, D + gap, 1), 1)
    return view.copy_(q)


@pytest.mark.gpu
@pytest.mark.parametrize("Q", [1, FEW, MANY])
@pytest.mark.parametrize("dtype,cache,D", [("bf16", "bf16", 64), ("fp16", "e4m3", 96), ("bf16", "bf16", 200)])
@pytest.mark.parametrize("form", ["tree", "sinks"])
def test_queries_and_outputs_on_odd_places(form, dtype, cache, D, Q):
    say("odd %s %s %d %d" % (form, dtype, D, Q))
    (q, kc, vc, table, lens), scales, sees, _ = base.made(200 + Q, [700, 41, 0, 300], Q, 4, 2, D, 16, dtype, cache)
    sees = sees if form == "tree" else None
    want, want_lse = base.call(q, kc, vc, table, lens, 700, 100, 5, ref.words_of(sees) if sees is not None else None,
                               **scales)
    base.verify(odd(q), kc, vc, table, lens, 700, 100, 5, sees, **scales)
    # an output with gaps, which stay as they are, and no lse; the same to the bit
    wide = torch.full((4, Q + 1, 4, D + 5), 9.0, dtype=q.dtype, device="cuda")
    out = wide[:, :Q, :, 2:2 + D]
    args = [base.up(odd(q)), base.up(kc), base.up(vc), base.up(table), base.up(lens)]
    more = {k: base.up(v) for k, v in scales.items()}
    if sees is None:
        native.xpress_sink_attention(*args, out, 700, 100, 5, **more)
    else:
        native.xpress_tree_attention(*args, base.up(ref.words_of(sees)), out, 700, window=100, sinks=5, **more)
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want)
    assert (wide[:, Q] == 9).all() and (wide[..., :2] == 9).all() and (wide[..., 2 + D:] == 9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("Q", [FEW, MANY])
def test_scales_of_keys_or_values_alone_and_of_other_signs(Q):
    (q, kc, vc, table, lens), scales, sees, _ = base.made(210, [300, 64], Q, 4, 2, 64, 16, "bf16", "e4m3")
    args = [base.up(q), base.up(kc), base.up(vc), base.up(table), base.up(lens), base.up(ref.words_of(sees))]
    one = torch.ones(2)
    for ks, vs in ((None, None), (scales["k_scale"], None), (None, scales["v_scale"]),
                   (scales["k_scale"] * torch.tensor([-1.0, 1.0]), scales["v_scale"] * torch.tensor([1.0, -1.0]))):
        want, _ = base.verify(q, kc, vc, table, lens, 300, sees=sees, scale=0.004,
                              k_scale=one if ks is None else ks, v_scale=one if vs is None else vs)
        out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        native.xpress_tree_attention(*args, out, 300, scale=0.004, k_scale=base.up(ks), v_scale=base.up(vs))
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("Q", [FEW, MANY])
def test_lengths_out_of_range_are_clamped(Q):
    (q, kc, vc, table, lens), _, sees, _ = base.made(220, [200, 200, 200, 200], Q, 4, 2, 64, 16)
    lens = torch.tensor([-5, 10 ** 9, -2 ** 31, 150], dtype=torch.int32)
    out, lse = base.verify(q, kc, vc, table, lens, 190, 30, 3, sees=sees)
    assert (out[[0, 2]] == 0).all() and np.isneginf(lse[[0, 2]]).all()
    base.verify(q, kc, vc, table, lens, 190, 30, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("form,window,sinks", [("sinks", 40, 4), ("sinks", 700, 33), ("sinks", 0, 0), ("tree", 100, 3)])
def test_a_prompt(form, window, sinks):
    """All tokens of a sequence are new; another has some before them, a third is shorter."""
    say("prompt %s %d" % (form, window))
    (q, kc, vc, table, lens), _, sees, _ = base.made(230, [300, 420, 90], 300, 4, 1, 64, 16)
    base.verify(q, kc, vc, table, lens, 420, window, sinks, sees if form == "tree" else None)


@pytest.mark.gpu
@pytest.mark.parametrize("Q", [FEW, MANY])
def test_pages_past_32_bits(Q):
    """Pages at the end of pools of 5 GiB each."""
    say("far pages")
    (q, kc, vc, table, lens), _, sees, _ = base.made(240, [300, 77], Q, 4, 2, 64, 16)
    pages = kc.shape[0]
    big = 5 * 2 ** 30 // (2 * 16 * 64 * 2)
    pools = [torch.zeros((big, 2, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for pool, x in zip(pools, (kc, vc)):
        pool[big - pages:] = x.cuda()
    far = torch.where(table >= 0, table + (big - pages), table)
    tree = ref.words_of(sees)
    for words, window in ((tree, 0), (tree, 50), (None, 50)):
        want = base.call(q, kc, vc, table, lens, 300, window, 3, words)
        out, lse = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(q.shape[:3], device="cuda")
        args = [base.up(q), *pools, base.up(far), base.up(lens)]
        if words is None:
            native.xpress_sink_attention(*args, out, 300, window, 3, lse=lse)
        else:
            native.xpress_tree_attention(*args, base.up(words), out, 300, window=window, sinks=3, lse=lse)
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), want[0]) and np.array_equal(lse.double().cpu().numpy(), want[1])
    # copies and moves there too
    native.xpress_kv_copy(*pools, torch.tensor([[big - pages, big - 1, 16], [0, big - 2, 9]], dtype=torch.int32,
                                               device="cuda"))
    native.xpress_kv_compact(*pools, base.up(far), torch.tensor([0, 0], dtype=torch.int32, device="cuda"),
                             torch.tensor([[3, 40], [70, 71]], dtype=torch.int32, device="cuda"),
                             torch.tensor([2, 0], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for pool, x in zip(pools, (kc, vc)):
        y = x.clone()
        y[pages - 1], y[pages - 2, :, :9] = x[0], 0
        for j, node in enumerate((3, 40)):
            y[table[0, j // 16], :, j % 16] = y[table[0, node // 16], :, node % 16].clone()
        assert torch.equal(pool[big - pages:].cpu().view(torch.int16), y.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("Q", [FEW, MANY])
def test_two_streams_at_once(Q):
    """Calls whose parts meet in a workspace, each stream its own."""
    sets = [base.made(250 + i, [3000, 900], Q, 4, 2, 64, 16) for i in range(2)]
    want = [base.call(*x[0], 3000, 0, 0, ref.words_of(x[2])) for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    dev = [[base.up(t) for t in x[0]] + [base.up(ref.words_of(x[2]))] for x in sets]
    outs = [torch.zeros(x[0][0].shape, dtype=x[0][0].dtype, device="cuda") for x in sets]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, o, s in zip(dev, outs, streams):
            native.xpress_tree_attention(*d, o, 3000, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.double().cpu().numpy(), w[0])
