"""Beam search over a paged cache whose beams share pages: the one-layer model of decode.py
takes prompts and keeps the best hypotheses of each.

A step of all beams is: pages for one more token (``xpress_kv_grow``), the newest tokens'
keys and values (``xpress_kv_append``), attention with a window and sinks
(``xpress_sink_attention``), project to the vocabulary, the best continuations
(``xpress_beam_select``), and the beams that go on: their page tables and the copies of
part-filled pages (``xpress_kv_fork``, ``xpress_kv_copy``), their tokens
(``xpress_beam_reorder``), and the pages that left the window (``xpress_kv_free``).  Two
steps, from one set of buffers to the other and back, have no host work, so that
``--graph`` captures them once and replays them.

    python examples/beams.py --seqs 4 --beams 4 --steps 32 --graph
"""
import argparse
import time

import torch

from decode import Decoder, native


class Beams(Decoder):
    """Beams of N sequences over a pool of `pages` pages."""

    def __init__(self, N, beams, max_len, window=64, sinks=4, page=16, pages=None, **kw):
        # a page more a row than its tokens need: where all rows hold all of theirs, a fork takes
        # new ones for the beams that part before those which it gives back are free
        super().__init__(N * beams, max_len + page, page=page, **kw)
        self.max_len = max_len
        self.seqs, self.beams, self.window, self.sinks, self.page = N, beams, window, sinks, page
        rows, width = N * beams, self.table.shape[1]
        pages = self.k_cache.shape[0] if pages is None else pages
        i32 = dict(device="cuda", dtype=torch.int32)
        self.refs = [torch.zeros(pages, **i32) for _ in range(2)]
        self.tables = [torch.full((rows, width), -1, **i32) for _ in range(2)]
        self.lens = torch.zeros(rows, **i32)
        self.copies, self.missing = torch.zeros(rows, 3, **i32), torch.zeros(2, 1, **i32)
        self.lacked = torch.zeros(1, **i32)   # of all calls since the start
        self.scores = torch.zeros(rows, device="cuda")
        self.best, self.rows = torch.zeros(N, beams, device="cuda"), torch.zeros(N, beams, **i32)
        self.ids = torch.zeros(N, beams, device="cuda", dtype=torch.int64)
        self.history = [torch.zeros(rows, max_len, device="cuda", dtype=torch.int64) for _ in range(2)]

    def start(self, prompts):
        """Lists of token ids, one a sequence: all but each last one go into the cache once, and
        are forked to the beams, of which the first alone counts at first."""
        self.longest = max(len(p) for p in prompts)
        if len(prompts) != self.seqs or min(len(p) for p in prompts) < 1 or self.longest > self.max_len:
            raise ValueError("%d prompts of 1 to %d tokens expected" % (self.seqs, self.max_len))
        lens = torch.tensor([len(p) - 1 for p in prompts], dtype=torch.int32, device="cuda")
        rows = torch.arange(self.seqs, dtype=torch.int32, device="cuda")
        self.refs[1].zero_()                  # the pages of an earlier search are free
        table = torch.full_like(self.tables[1][:self.seqs], -1)
        native.xpress_kv_grow(self.refs[1], table, torch.zeros_like(lens), lens, self.page, missing=self.missing[0])
        self.table = table
        ids = torch.tensor([i for p in prompts for i in p[:-1]], dtype=torch.int64, device="cuda")
        seq = torch.repeat_interleave(rows, lens.long())
        pos = torch.cat([torch.arange(len(p) - 1) for p in prompts]).to(torch.int32).cuda()
        if len(ids):
            self.append(self.embed[ids], pos, seq)
        src = rows.repeat_interleave(self.beams)
        native.xpress_kv_fork(self.refs[1], table, lens, src, self.refs[0], self.tables[0], self.copies, self.page,
                              missing=self.missing[1])
        native.xpress_kv_copy(self.k_cache, self.v_cache, self.copies)
        self.lens.copy_(lens[src.long()])
        for i, p in enumerate(prompts):
            self.history[0][i * self.beams:(i + 1) * self.beams, :len(p)] = torch.tensor(p, device="cuda")
        self.scores.fill_(float("-inf"))
        self.scores[::self.beams] = 0.0
        self.lacked.zero_()
        self.count_missing()
        self.check()

    def count_missing(self):
        """Adds what the last xpress_kv_grow and xpress_kv_fork lacked, which the next ones write
        over."""
        self.lacked.add_(self.missing[0]).add_(self.missing[1])

    def check(self):
        """Tokens without a page are not stored, and hypotheses over them mean nothing."""
        if int(self.lacked):
            raise RuntimeError("the pool lacked %d pages" % int(self.lacked))

    def half(self, a, b):
        """One token for every beam, from buffers a to buffers b."""
        rows, longer = self.N, self.lens + 1
        self.table = self.tables[a]
        native.xpress_kv_grow(self.refs[a], self.table, self.lens, longer, self.page, missing=self.missing[0])
        x = self.embed[self.history[a].gather(1, self.lens.long()[:, None])[:, 0]]
        q = self.append(x, self.lens).view(rows, 1, self.hq, self.dim)
        out = torch.empty_like(q)
        native.xpress_sink_attention(q, self.k_cache, self.v_cache, self.table, longer, out, self.max_len, self.window,
                                     self.sinks, k_scale=self.scale, v_scale=self.scale)
        logits = (x + out.view(rows, -1) @ self.w_out.t()) @ self.w_vocab.t()
        native.xpress_beam_select(logits, None, self.scores, self.best, self.rows, self.ids, self.seqs, self.beams,
                                  self.vocab, self.beams, self.vocab)
        native.xpress_kv_free(self.refs[a], self.table, longer, self.page, window=self.window, sinks=self.sinks)
        native.xpress_kv_fork(self.refs[a], self.table, longer, self.rows, self.refs[b], self.tables[b], self.copies,
                              self.page, missing=self.missing[1])
        self.count_missing()
        native.xpress_kv_copy(self.k_cache, self.v_cache, self.copies)
        native.xpress_beam_reorder([(self.history[a], self.history[b])], self.rows)
        self.scores.copy_(self.best.view(-1))
        self.lens.add_(1)
        self.history[b].scatter_(1, self.lens.long()[:, None], self.ids.view(-1, 1))

    def search(self, steps, graph=False):
        """`steps` (even, 2 or more) tokens; the hypotheses [rows, max_len] and their scores."""
        # (past max_len a token's place in the history is out of range on the device)
        if steps < 2 or steps % 2 or self.longest + steps > self.max_len:
            raise ValueError("an even number of 2 or more steps expected, and %d tokens with the longest "
                             "prompt's %d at most" % (self.max_len, self.longest))
        self.longest += steps
        pairs = steps // 2
        if graph:
            self.half(0, 1)           # the libraries' first calls stay out of the graph
            self.half(1, 0)
            torch.cuda.synchronize()
            stream, captured = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            native.xpress_sparse_attention_reserve(self.N, 1, self.hq, self.hk, self.dim, self.max_len, self.window,
                                                   self.sinks, stream=stream)
            native.xpress_beam_select_reserve(self.seqs, self.beams, self.vocab, self.beams, stream=stream)
            with torch.cuda.graph(captured, stream=stream):
                self.half(0, 1)
                self.half(1, 0)
            for _ in range(pairs - 1):
                captured.replay()
            torch.cuda.synchronize()
        else:
            for _ in range(pairs):
                self.half(0, 1)
                self.half(1, 0)
        self.check()
        return self.history[0], self.scores


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--seqs", type=int, default=4)
    p.add_argument("--beams", type=int, default=4)
    p.add_argument("--prompt", type=int, default=100, help="length of the longest prompt")
    p.add_argument("--steps", type=int, default=32, help="even, 2 or more")
    p.add_argument("--graph", action="store_true")
    a = p.parse_args()
    d = Beams(a.seqs, a.beams, a.prompt + a.steps + 4)
    r = torch.Generator().manual_seed(5)
    lens = torch.randint(max(1, a.prompt // 4), a.prompt + 1, (a.seqs,), generator=r).tolist()
    d.start([torch.randint(0, d.vocab, (n,), generator=r).tolist() for n in lens])
    torch.cuda.synchronize()
    t = time.perf_counter()
    history, scores = d.search(a.steps, graph=a.graph)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print("%d sequences of %d beams, %d steps: %.1f us a step; best of the first: %s, score %.3f"
          % (a.seqs, a.beams, a.steps, t / a.steps * 1e6, history[0, lens[0]:lens[0] + 8].tolist(), float(scores[0])))


if __name__ == "__main__":
    main()
