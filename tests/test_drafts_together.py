"""The operators as they are used together: beam search over shared pages, and a drafted
tree that is verified, cut down to one path and decoded on from."""
import os
import sys

import numpy as np
import pytest
import torch

import drafts_ref as ref
from vocab_wide_add_amd import native

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def searcher(cache="bf16", window=24):
    import beams
    d = beams.Beams(3, 3, 80, window=window, sinks=3, page=8, hq=8, hk=2, dim=64, vocab=1000, cache=cache)
    r = torch.Generator().manual_seed(7)
    prompts = [torch.randint(0, 1000, (n,), generator=r).tolist() for n in (40, 1, 17)]
    d.start(prompts)
    return d, prompts


def holders(table, pages):
    table = table.cpu().numpy()
    return np.bincount(table[(table >= 0) & (table < pages)], minlength=pages)


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_replayed_graph_searches_as_eager_steps_do(cache):
    a, b = searcher(cache)[0], searcher(cache)[0]
    want = [x.clone() for x in a.search(12)]
    got = b.search(12, graph=True)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    for d in (a, b):
        assert int(d.missing.sum()) == 0
        assert np.array_equal(d.refs[0].cpu().numpy(), holders(d.tables[0], len(d.refs[0])))
        # what no beam will see again has been given back: three sinks' page, the window's
        assert ((d.tables[0] >= 0).sum(1).cpu() <= 1 + (24 + 7) // 8 + 1).all()


@pytest.mark.gpu
def test_hypotheses_have_the_scores_of_a_plain_model():
    """Each hypothesis' score is the sum of its tokens' log probabilities under the same
    model over a dense history in 64 bits, as far as the bf16 activations allow: a logit sums
    512 products of rounded factors, whose errors (half steps of 2^-8 each in the embedding's,
    the attention's, its projection's and the sum's rounding, and the logit's own) stay below
    2^-8 * 5 of the sum of the products' magnitudes, and a log probability has two such; the
    best of each list is not beaten by another."""
    d, prompts = searcher()
    steps = 6
    history, scores = (x.cpu() for x in d.search(steps))
    E, Wq, Wo, Wv = (x.double().cpu() for x in (d.embed, d.w_qkv, d.w_out, d.w_vocab))
    cs = d.cos_sin.double().cpu()

    def turned(x, n):
        a, b = x[..., :32], x[..., 32:]
        c, s = cs[:n, None, :32], cs[:n, None, 32:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    for n, prompt in enumerate(prompts):
        rows = range(n * 3, n * 3 + 3)
        assert len({tuple(history[r, :len(prompt) + steps].tolist()) for r in rows}) == 3
        assert scores[n * 3] >= scores[n * 3 + 1] >= scores[n * 3 + 2]
        for r in rows:
            tokens = history[r, :len(prompt) + steps].tolist()
            assert tokens[:len(prompt)] == prompt
            total, tol = 0.0, 0.0
            for t in range(len(prompt), len(tokens)):
                L = t
                x = E[tokens[:L]]
                qkv = (x @ Wq.t()).view(L, 12, 64)
                q, k, v = turned(qkv[:, :8], L)[-1], turned(qkv[:, 8:10], L), qkv[:, 10:]
                k, v = k.repeat_interleave(4, 1), v.repeat_interleave(4, 1)
                z = (k * q[None]).sum(-1) / 8.0
                see = torch.from_numpy(ref.visible(L, 1, 24, 3)[0])
                w = torch.softmax(torch.where(see[:, None], z, float("-inf")), 0)
                y = x[-1] + (w[..., None] * v).sum(0).reshape(-1) @ Wo.t()
                total += float(torch.log_softmax(y @ Wv.t(), 0)[tokens[t]])
                tol += 2 * 5 * 2.0 ** -8 * float((Wv.abs() @ y.abs()).max())
            assert abs(float(scores[r]) - total) <= tol, (r, float(scores[r]), total, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 5)])
def test_a_verified_tree_leaves_what_plain_decoding_leaves(cache, window, sinks):
    """A tree's nodes appended at their places and positions; each node's attention is that of
    its own line of tokens in a plain cache; the path that is kept, moved together, is bit for
    bit the cache of a sequence that was decoded token by token; and the pages behind it can be
    given back."""
    rng = np.random.default_rng(3)
    N, Q, Hq, Hk, D, page, width = 3, 12, 4, 2, 64, 8, 16
    past = np.array([50, 7, 0])
    pages = 2 * N * width
    types = dict(bf16=torch.bfloat16, e4m3=torch.float8_e4m3fn)
    scale = torch.full((Hk,), 1.0 / 32, device="cuda") if cache == "e4m3" else None

    def i32(x):
        return torch.from_numpy(np.ascontiguousarray(np.asarray(x).astype(np.int32))).cuda()

    def normal(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()

    angle = rng.uniform(0, 6, (200, D // 2))
    cs = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
    parents, sees = ref.random_trees(rng, N, Q)
    depth = sees.sum(-1) - 1
    old_k, old_v = normal(N, int(past.max()), Hk, D), normal(N, int(past.max()), Hk, D)
    q, k, v = normal(N * Q, Hq, D), normal(N * Q, Hk, D), normal(N * Q, Hk, D)

    def fresh():
        caches = [torch.zeros(pages, Hk, page, D, device="cuda").to(types[cache]) for _ in range(2)]
        refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        table = torch.full((N, width), -1, dtype=torch.int32, device="cuda")
        return caches, refs, table

    def put(caches, table, kk, vv, at, positions, seq, qq=None):
        out = torch.empty_like(qq) if qq is not None else None
        native.xpress_kv_append_at(qq, kk.contiguous(), vv.contiguous(), out, *caches, table, i32(at), i32(positions), cs,
                                   seq_of=i32(seq), k_scale=scale, v_scale=scale)
        return out

    def prompt(caches, table):
        seq = np.repeat(np.arange(N), past)
        pos = np.concatenate([np.arange(p) for p in past])
        put(caches, table, old_k[seq, pos], old_v[seq, pos], pos, pos, seq)

    # the tree
    caches, refs, table = fresh()
    native.xpress_kv_grow(refs, table, i32(np.zeros(N)), i32(past + Q), page)
    prompt(caches, table)
    seq = np.repeat(np.arange(N), Q)
    turned = put(caches, table, k, v, (past[:, None] + np.arange(Q)).ravel(), (past[:, None] + depth).ravel(), seq, q)
    out = torch.empty(N, Q, Hq, D, dtype=torch.bfloat16, device="cuda")
    native.xpress_tree_attention(turned.view(N, Q, Hq, D), *caches, table, i32(past + Q), ref.words_of(sees).cuda(), out,
                                 int(past.max()) + Q, window=window, sinks=sinks, k_scale=scale, v_scale=scale)

    # every node's line in a cache of its own
    for leaf in range(Q):
        line = [np.flatnonzero(sees[n, leaf]) for n in range(N)]
        other, refs2, table2 = fresh()
        lens = past + np.array([len(x) for x in line])
        native.xpress_kv_grow(refs2, table2, i32(np.zeros(N)), i32(lens), page)
        prompt(other, table2)
        rows = np.concatenate([n * Q + x for n, x in enumerate(line)])
        pos = np.concatenate([past[n] + np.arange(len(x)) for n, x in enumerate(line)])
        put(other, table2, k[rows], v[rows], pos, pos, rows // Q)
        one = torch.empty(N, 1, Hq, D, dtype=torch.bfloat16, device="cuda")
        ask = turned.view(N, Q, Hq, D)[:, leaf:leaf + 1]
        native.xpress_sink_attention(ask, *other, table2, i32(lens), one, int(lens.max()), window, sinks, k_scale=scale,
                                     v_scale=scale)
        torch.cuda.synchronize()
        got, want = out[:, leaf].double().cpu(), one[:, 0].double().cpu()
        assert all(len(x) <= 30 for x in line)     # else a line's window would pass over its own first nodes
        # two roundings of sums near each other
        assert torch.allclose(got, want, rtol=2.0 ** -7, atol=2.0 ** -11)
        if leaf in (5, 11):
            # this line is kept
            kept = [c.clone() for c in caches]
            path = np.full((N, Q), -1)
            for n, x in enumerate(line):
                path[n, :len(x)] = x
            native.xpress_kv_compact(*kept, table, i32(past), i32(path), i32([len(x) for x in line]))
            t1, t2 = table.cpu().numpy(), table2.cpu().numpy()
            for a, b in zip(kept, other):
                a, b = (x.view(torch.uint8 if cache == "e4m3" else torch.int16).cpu() for x in (a, b))
                for n in range(N):
                    for j in range(lens[n]):
                        assert torch.equal(a[t1[n, j // page], :, j % page], b[t2[n, j // page], :, j % page]), (n, j)
            left, cut = refs.clone(), table.clone()
            native.xpress_kv_free(left, cut, i32(lens), page)
            torch.cuda.synchronize()
            assert np.array_equal(left.cpu().numpy(), holders(cut, pages))
            assert ((cut >= 0).sum(1).cpu().numpy() == -(-lens // page)).all()
