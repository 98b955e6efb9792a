"""xpress_tree_attention where a sequence is shorter than its tree: no key stands at a negative
place, and a query's row is given out whatever its own place: it sees the nodes that exist and
that its bits name."""
import numpy as np
import pytest
import torch

import drafts_ref as ref
import serving_ref
from gpu_util import say
from vocab_wide_add_amd import native


@pytest.mark.gpu
@pytest.mark.parametrize("Q,Hq,Hk", [(6, 4, 2), (20, 8, 2), (40, 4, 2), (70, 4, 1)])   # 12, 80, 80 and 280 rows a head
@pytest.mark.parametrize("window", [0, 3])
def test_rows_at_negative_places_see_what_their_bits_name(Q, Hq, Hk, window):
    """Compared with the plain definition over the nodes that exist; tolerances: the output's
    rounding, and 2^-14 of the largest value for weights of 16 bits and sums of fewer than 70."""
    say("short %d %d" % (Q, window))
    rng = np.random.default_rng(Q)
    lens = [Q - 4, Q, 1, 0]
    D, page = 64, 16
    kc, vc, table = serving_ref.paged_pool(rng, lens, Hk, D, page, "bf16", "head", fill=float("nan"))
    q = torch.from_numpy(rng.standard_normal((4, Q, Hq, D)).astype(np.float32)).to(torch.bfloat16)
    sees = rng.random((4, Q, Q)) < 0.4
    sees[0, 0] = False
    sees[0, 0, 4] = True             # a row at place -4 that names the first node there is
    sees[0, 1] = False
    sees[0, 1, :4] = True            # and one that names none that is
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, Q, Hq), 7.0, device="cuda")
    native.xpress_tree_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(),
                                 torch.tensor(lens, dtype=torch.int32, device="cuda"), ref.words_of(sees).cuda(), out, Q,
                                 lse=lse, window=window)
    torch.cuda.synchronize()
    got, got_lse = out.double().cpu(), lse.double().cpu()
    G = Hq // Hk
    for n, length in enumerate(lens):
        past = length - Q
        K, V = (torch.stack([x[table[n, j // page], :, j % page] for j in range(length)]).double()
                if length else torch.zeros(0, Hk, D).double() for x in (kc, vc))
        for i in range(Q):
            js = [past + j for j in range(Q) if past + j >= 0 and sees[n, i, j]]
            if not js:
                assert (got[n, i] == 0).all() and torch.isneginf(got_lse[n, i]).all()
                continue
            for h in range(Hq):
                z = K[js, h // G] @ q[n, i, h].double() / 8.0
                want = torch.softmax(z, 0) @ V[js, h // G]
                tol = 2.0 ** -8 * want.abs() + 2.0 ** -14 * V[js, h // G].abs().max()
                assert ((got[n, i, h] - want).abs() <= tol).all(), (n, i, h)
                assert abs(got_lse[n, i, h] - torch.logsumexp(z, 0)) <= 2.0 ** -16
    assert torch.equal(got[0, 0], vc[table[0, 0], :, 0].double().repeat_interleave(G, 0))
    assert (got[0, 1] == 0).all()
    # without a tree such rows see nothing
    native.xpress_sink_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(),
                                 torch.tensor(lens, dtype=torch.int32, device="cuda"), out, Q, window, 2, lse=lse)
    torch.cuda.synchronize()
    assert (out[0, :4] == 0).all() and torch.isneginf(lse[0, :4]).all()
    assert (out[0, 4:] != 0).any() and torch.isfinite(lse[0, 4:]).all()
