"""The decoding example: the operators together, eagerly and as a replayed graph."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def made(cache, **kw):
    import decode
    d = decode.Decoder(3, 96, hq=8, hk=2, dim=64, vocab=5000, cache=cache, **kw)
    r = torch.Generator().manual_seed(7)
    d.prompt([torch.randint(0, 5000, (n,), generator=r).tolist() for n in (40, 1, 17)])
    return d


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_replayed_graph_draws_what_eager_steps_draw(cache):
    a, b = made(cache), made(cache)
    want = a.run(20)
    got = b.run(20, graph=True)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert ((want >= 0) & (want < 5000)).all() and len(want.unique()) > 10
    assert torch.equal(a.pos.cpu(), torch.tensor([59, 20, 36], dtype=torch.int32))
    for x, y in ((a.k_cache, b.k_cache), (a.v_cache, b.v_cache)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.gpu
def test_greedy_steps_take_the_likeliest_token_of_a_plain_model():
    """Every greedy token has the largest logit of the same model over a dense history
    in 64 bits, up to the roundings of the bf16 activations: a logit sums 512 products
    of rounded factors, whose errors (half steps of 2^-8 each in the embedding's, the
    attention's, its projection's and the sum's rounding, and the logit's own) stay
    below 2^-8 * 5 of the sum of the products' magnitudes."""
    d = made("bf16", temperature=0.0)
    r = torch.Generator().manual_seed(7)
    history = [torch.randint(0, 5000, (n,), generator=r).tolist() for n in (40, 1, 17)]
    drawn = d.run(6).cpu()
    E, Wq, Wo, Wv = (x.double().cpu() for x in (d.embed, d.w_qkv, d.w_out, d.w_vocab))
    cs = d.cos_sin.double().cpu()

    def turned(x, n):
        a, b = x[..., :32], x[..., 32:]
        c, s = cs[:n, None, :32], cs[:n, None, 32:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    for n, tokens in enumerate(history):
        for t in range(6):
            x = E[tokens]
            L = len(tokens)
            qkv = (x @ Wq.t()).view(L, 12, 64)
            q, k, v = turned(qkv[:, :8], L)[-1], turned(qkv[:, 8:10], L), qkv[:, 10:]
            k, v = k.repeat_interleave(4, 1), v.repeat_interleave(4, 1)
            w = torch.softmax((k * q[None]).sum(-1) / 8.0, 0)
            y = x[-1] + (w[..., None] * v).sum(0).reshape(-1) @ Wo.t()
            logits = y @ Wv.t()
            tol = 5 * 2.0 ** -8 * (Wv.abs() @ y.abs()).max()
            token = int(drawn[t, n])
            assert logits[token] >= logits.max() - 2 * tol, (n, t, logits[token], logits.max(), tol)
            tokens.append(token)
