"""Decoding with the serving operators: a one-layer attention model with random weights
takes prompts of different lengths and draws tokens after them.

A step of all sequences is: embed the newest tokens, project to queries, keys and values,
append them to the paged cache (``xpress_kv_append``), attend to it
(``xpress_paged_attention``), project to the vocabulary, draw (``xpress_sample_to_blk``).
The projections are torch matmuls.  The step has no host work, so that ``--graph`` captures
it once and replays it.

    python examples/decode.py --seqs 8 --steps 64 --cache e4m3 --graph
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from vocab_wide_add_amd import native  # noqa: E402

CACHES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


class Decoder:
    """Weights, cache and buffers of N sequences that hold up to max_len tokens."""

    def __init__(self, N, max_len, hq=16, hk=4, dim=128, vocab=32000, page=16, cache="bf16",
                 temperature=0.8, top_k=50, top_p=0.95, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.N, self.max_len, self.hq, self.hk, self.dim, self.vocab = N, max_len, hq, hk, dim, vocab
        width = hq * dim

        def weight(*shape):
            return (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).to(torch.bfloat16)

        self.embed = torch.randn(vocab, width, generator=g, device="cuda").to(torch.bfloat16)
        self.w_qkv = weight((hq + 2 * hk) * dim, width)
        self.w_out = weight(width, width)
        self.w_vocab = weight(vocab, width) * 2.0
        angle = torch.arange(max_len, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(dim // 2, device="cuda", dtype=torch.float64) / (dim // 2))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()

        # pages of all sequences in one pool, handed out in any order
        each = -(-max_len // page)
        order = torch.randperm(N * each, generator=torch.Generator().manual_seed(seed))
        self.table = order.view(N, each).to(torch.int32).cuda()
        shape = (N * each, hk, page, dim)
        self.k_cache, self.v_cache = (torch.zeros(shape, device="cuda").to(CACHES[cache]) for _ in range(2))
        self.scale = torch.full((hk,), 1.0 / 32, device="cuda") if cache == "e4m3" else None

        self.blk = torch.zeros(N, 2, dtype=torch.int64, device="cuda")   # newest token, drawn token
        self.pos = torch.zeros(N, dtype=torch.int32, device="cuda")      # of the newest token
        self.step_no = torch.zeros(1, dtype=torch.int64, device="cuda")
        full = dict(device="cuda", dtype=torch.float32)
        self.temperature = torch.full((N,), float(temperature), **full)
        self.top_p, self.min_p = torch.full((N,), float(top_p), **full), torch.zeros(N, **full)
        self.top_k = torch.full((N,), int(top_k), device="cuda", dtype=torch.int32)
        self.prob = torch.zeros(N, **full)

    def append(self, x, positions, seq_of=None):
        """Keys and values of rows x [T, width] into the cache; the rotated queries."""
        qkv = (x @ self.w_qkv.t()).view(-1, self.hq + 2 * self.hk, self.dim)
        q, k, v = qkv.split([self.hq, self.hk, self.hk], 1)
        q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        native.xpress_kv_append(q, k, v, q_out, self.k_cache, self.v_cache, self.table, positions,
                                self.cos_sin, seq_of=seq_of, k_scale=self.scale, v_scale=self.scale)
        return q_out

    def prompt(self, tokens):
        """Lists of token ids, one a sequence: all but each last one go into the cache."""
        lens = [len(t) - 1 for t in tokens]
        ids = torch.tensor([i for t in tokens for i in t[:-1]], dtype=torch.int64, device="cuda")
        seq = torch.repeat_interleave(torch.arange(self.N), torch.tensor(lens)).to(torch.int32).cuda()
        pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
        self.append(self.embed[ids], pos, seq)
        self.blk[:, 0] = torch.tensor([t[-1] for t in tokens], device="cuda")
        self.pos.copy_(torch.tensor(lens, dtype=torch.int32))

    def step(self, u_all, drawn):
        """One token for every sequence, with the uniform numbers u_all[step]; drawn[step]
        receives the tokens."""
        u = u_all.index_select(0, self.step_no)[0]
        x = self.embed[self.blk[:, 0]]
        q = self.append(x, self.pos).view(self.N, 1, self.hq, self.dim)
        lens = self.pos + 1
        out = torch.empty_like(q)
        native.xpress_paged_attention(q, self.k_cache, self.v_cache, self.table, lens, out, self.max_len,
                                      k_scale=self.scale, v_scale=self.scale)
        y = x + out.view(self.N, -1) @ self.w_out.t()
        logits = y @ self.w_vocab.t()
        native.xpress_sample_to_blk(logits, None, self.blk, self.temperature, self.top_k, self.top_p,
                                    self.min_p, u, self.N, 2, self.vocab, self.vocab, prob=self.prob)
        drawn.index_copy_(0, self.step_no, self.blk[None, :, 1])
        self.blk[:, 0].copy_(self.blk[:, 1])
        self.pos.add_(1)
        self.step_no.add_(1)

    def run(self, steps, seed=1, graph=False):
        """Token ids [steps, N]."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        u_all = torch.rand(steps, self.N, generator=g, device="cuda")
        drawn = torch.zeros(steps, self.N, dtype=torch.int64, device="cuda")
        self.step_no.zero_()
        if not graph:
            for _ in range(steps):
                self.step(u_all, drawn)
            return drawn
        self.step(u_all, drawn)       # the libraries' first calls stay out of the graph
        torch.cuda.synchronize()
        stream, captured = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        native.xpress_paged_attention_reserve(self.N, 1, self.hq, self.hk, self.dim, self.max_len,
                                              stream=stream)
        with torch.cuda.graph(captured, stream=stream):
            self.step(u_all, drawn)
        for _ in range(steps - 1):
            captured.replay()
        torch.cuda.synchronize()      # before the graph's memory goes
        return drawn


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--seqs", type=int, default=8)
    p.add_argument("--prompt", type=int, default=200, help="length of the longest prompt")
    p.add_argument("--steps", type=int, default=64, help="2 or more")
    p.add_argument("--cache", choices=sorted(CACHES), default="bf16")
    p.add_argument("--graph", action="store_true")
    a = p.parse_args()
    d = Decoder(a.seqs, a.prompt + a.steps, cache=a.cache)
    r = torch.Generator().manual_seed(5)
    lens = torch.randint(max(1, a.prompt // 4), a.prompt + 1, (a.seqs,), generator=r).tolist()
    d.prompt([torch.randint(0, d.vocab, (n,), generator=r).tolist() for n in lens])
    d.run(1)                          # loads the libraries
    torch.cuda.synchronize()
    t = time.perf_counter()
    drawn = d.run(a.steps - 1, graph=a.graph)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print("%d sequences, %d steps: %.1f us a step; first sequence: %s"
          % (a.seqs, a.steps - 1, t / (a.steps - 1) * 1e6, drawn[:8, 0].tolist()))


if __name__ == "__main__":
    main()
