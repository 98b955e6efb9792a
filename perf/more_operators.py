"""Operators of drafts that branch and of beams, as measured: attention of a tree of drafted tokens over
the paged cache, attention with a window and sinks, the cache's pages (forked, copied, grown, freed,
compacted), and beam search's selection with its states.

``run`` computes a pass in plain torch operations, or (``own``) through the framework's entry points;
``exact`` computes the same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "fp16": 2, "e4m3": 1}
_E4M3_MAX = 448.0


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _attend(name, op, N, Q, Hq, Hk, D, page, longest, ragged, dtype="bf16", cache="bf16", layout="head",
            window=0, sinks=0):
    """op "tree": Q nodes of a tree; "sinks": Q tokens in a row."""
    return dict(name=name, op=op, N=N, Q=Q, Hq=Hq, Hk=Hk, D=D, page=page, longest=longest, ragged=ragged,
                dtype=dtype, cache=cache, layout=layout, window=window, sinks=sinks)


def _fork(name, N, beams, prompt, drawn, Hk, D, page, dtype="bf16", layout="head"):
    """N sequences of `beams` beams each, that share a prompt and have `drawn` tokens of their own."""
    return dict(name=name, op="fork", N=N, beams=beams, prompt=prompt, drawn=drawn, Hk=Hk, D=D, page=page,
                dtype=dtype, cache=dtype, layout=layout)


def _turn(name, N, longest, more, page, window=0, sinks=0):
    return dict(name=name, op="turn", N=N, longest=longest, more=more, page=page, window=window, sinks=sinks)


def _compact(name, N, Q, depth, past, Hk, D, page, dtype="bf16", cache="bf16", layout="head"):
    return dict(name=name, op="compact", N=N, Q=Q, depth=depth, past=past, Hk=Hk, D=D, page=page, dtype=dtype,
                cache=cache, layout=layout)


def _beams(name, N, beams, K, V, pad, bias, history, hidden):
    return dict(name=name, op="beams", N=N, beams=beams, K=K, V=V, pad=pad, bias=bias, history=history,
                hidden=hidden)


def listed():
    return [
        # one user's drafted tree of 8 nodes after one chat turn: latency
        _attend("tree_one", "tree", 1, 8, 32, 8, 128, 16, 1009, False),
        # trees of 16 nodes (the framework's B) for 32 sequences, ragged lengths
        _attend("tree_32", "tree", 32, 16, 32, 8, 128, 16, 4096, True),
        # wide trees: 64 nodes, 256 rows a key-value head
        _attend("tree_wide", "tree", 32, 64, 32, 8, 128, 32, 4096, True),
        # an 8-bit cache in token-major pages that end inside every tile, an odd number of nodes, small heads
        _attend("tree_e4m3", "tree", 48, 11, 28, 4, 64, 24, 6001, True, cache="e4m3", layout="token"),
        # chats far longer than their window of 4096, four sinks; the pages between are freed
        _attend("sinks_32", "sinks", 32, 1, 32, 8, 128, 16, 32768, True, window=4096, sinks=4),
        # a drafted block over a short window, odd sizes everywhere
        _attend("sinks_block", "sinks", 24, 5, 35, 5, 80, 24, 9001, True, dtype="fp16", cache="fp16",
                layout="token", window=1777, sinks=37),
        # the pages of one sequence's four beams: latency
        _fork("fork_one", 1, 4, 1009, 19, 8, 128, 16),
        # a step of 32 sequences with 8 beams each
        _fork("fork_256", 32, 8, 1009, 301, 8, 128, 16),
        # 256 sequences that drop rejected tokens and what left their window, then take pages for new ones
        _turn("turn_256", 256, 8192, 64, 16, window=4096, sinks=4),
        # trees of 64 nodes appended, the accepted path moved to its places
        _compact("compact_64", 64, 64, 12, 2000, 8, 128, 16),
        # one sequence's next token over 4 beams
        _beams("beams_one", 1, 4, 8, 152064, 0, False, 256, 4096),
        # the framework's 480 rows as 60 sequences of 8 beams
        _beams("beams_480", 60, 8, 8, 152064, 0, True, 256, 4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "sinks", "sinks", "fork", "fork", "turn", "compact", "compact",
                     "beams", "beams"])
    if op == "beams":
        beams = rng.choice([1, 2, 3, 4, 8, 16])
        rows = _log_int(rng, 1, 480)
        return dict(op=op, N=max(1, rows // beams), beams=beams, K=rng.choice([beams, 2 * beams, 1, 5]),
                    V=_log_int(rng, 1000, 152064), pad=rng.choice([0, 0, 64, 7]), bias=rng.random() < 0.6,
                    history=_log_int(rng, 1, 1000), hidden=_log_int(rng, 16, 4096))
    window, sinks = rng.choice([(0, 0), (_log_int(rng, 16, 4096), rng.choice([0, 1, 4, 33, 128]))])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "turn":
        return dict(op=op, N=_log_int(rng, 1, 256), longest=_log_int(rng, 20, 8192), more=rng.choice([1, 1, 17, 64]),
                    page=page, window=window, sinks=sinks)
    G = rng.choice([1, 2, 4, 5, 7, 8, 16])
    Hk = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 80, 96, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    layout = rng.choice(["head", "token"])
    if op == "fork":
        beams = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, N=_log_int(rng, 1, 256 // beams), beams=beams, prompt=_log_int(rng, 1, 1009),
                    drawn=_log_int(rng, 1, 301), Hk=Hk, D=min(D, 128), page=page, dtype=dtype, cache=dtype,
                    layout=layout)
    if op == "compact":
        Q = _log_int(rng, 2, 64)
        return dict(op=op, N=_log_int(rng, 1, 64), Q=Q, depth=rng.randint(1, min(Q, 16)),
                    past=_log_int(rng, 1, 2000), Hk=Hk, D=min(D, 128), page=page, dtype=dtype, cache=cache,
                    layout=layout)
    Q = _log_int(rng, 1, 64) if op == "tree" else rng.choice([1, 1, 1, 5, 16])
    if op == "sinks" and not window:
        window, sinks = _log_int(rng, 16, 4096), rng.choice([1, 4, 33, 128])
    N = _log_int(rng, 1, 64)
    most = 32 * 4096 * 8 * 128 // (N * Hk * D)          # cached values as in the listed cases
    work = 32 * 4096 * 64 * 32 * 128 // (N * Q * G * Hk * D)
    longest = _log_int(rng, Q + 17, max(Q + 18, min(65536, most, work)))
    return dict(op=op, N=N, Q=Q, Hq=G * Hk, Hk=Hk, D=D, page=page, longest=longest, ragged=rng.random() < 0.7,
                dtype=dtype, cache=cache, layout=layout, window=window, sinks=sinks)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _pool(case, pages, r, gen):
    """Key and value pools with finite values everywhere, viewed [pages, Hk, page, D], and their scales."""
    ps, Hk, D, cache = case["page"], case["Hk"], case["D"], case["cache"]
    shape = (pages, ps, Hk, D) if case["layout"] == "token" else (pages, Hk, ps, D)

    def one():
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        if cache == "e4m3":
            y = torch.empty(shape, dtype=_TYPES[cache], device="cuda")
            y.view(-1).copy_((x.view(-1) * 24.0).clamp_(-_E4M3_MAX, _E4M3_MAX))
            x = y
        else:
            x = x.to(_TYPES[cache])
        return x.transpose(1, 2) if case["layout"] == "token" else x

    k, v = one(), one()
    ks = vs = None
    if cache == "e4m3":
        ks, vs = (torch.from_numpy((r.uniform(0.6, 1.4, Hk) / 24.0).astype(np.float32)).cuda() for _ in "kv")
    return k, v, ks, vs


def _trees(N, Q, r):
    """Random trees of Q nodes whose parents come before them: parents [N, Q] (-1: the root), and who sees whom."""
    back = 1 + (r.random((N, Q)) ** 2 * 8).astype(np.int64)
    parents = np.maximum(np.arange(Q) - back, 0)
    parents[:, 0] = -1
    at = np.broadcast_to(np.arange(Q), (N, Q))
    sees = np.zeros((N, Q, Q), bool)
    while (at >= 0).any():
        n, i = np.nonzero(at >= 0)
        sees[n, i, at[n, i]] = True
        at = np.where(at >= 0, np.take_along_axis(parents, np.maximum(at, 0), 1), -1)
    return parents, sees


def prepare(case, seed):
    r = np.random.default_rng([seed, 78])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 2 + 1)

    def normal(shape, sigma, dtype):
        x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, sigma, generator=gen)
        return x.to(dtype)

    def up(x, dtype=np.int32):
        return torch.from_numpy(np.ascontiguousarray(np.asarray(x).astype(dtype))).cuda()

    s = dict(case=case)
    op, N = case["op"], case["N"]
    if op == "beams":
        rows, stride, K = N * case["beams"], case["V"] + case["pad"], case["K"]
        s["base"] = normal((rows, stride), 4.0, torch.bfloat16)
        s["bias"] = normal((rows, stride), 0.5, torch.bfloat16) if case["bias"] else None
        s["scores"] = up(-r.gamma(4.0, 2.0, rows), np.float32)
        s["history"] = up(r.integers(0, case["V"], (rows, case["history"])), np.int64)
        s["hidden"] = normal((rows, case["hidden"]), 1.0, torch.bfloat16)
        s["new_history"] = torch.empty((N * K, case["history"]), dtype=torch.int64, device="cuda")
        s["new_hidden"] = torch.empty((N * K, case["hidden"]), dtype=torch.bfloat16, device="cuda")
        s["best"] = torch.empty((N, K), dtype=torch.float32, device="cuda")
        s["rows"] = torch.empty((N, K), dtype=torch.int32, device="cuda")
        s["ids"] = torch.empty((N, K), dtype=torch.int64, device="cuda")
        return s

    ps = case["page"]
    if op == "turn":
        old = r.integers(max(1, case["longest"] // 8), case["longest"] + 1, N)
        s["keep"] = up(np.maximum(old - r.integers(0, case["more"] + 1, N), 0))   # rejected tokens go
        s["want"] = s["keep"] + case["more"]
        width = -(-(case["longest"] + case["more"]) // ps)
        need = -(-old // ps)
        pages = N * width + 5
        order = r.permutation(pages)
        slots = np.arange(width)[None] < need[:, None]
        table = np.full((N, width), -1)
        table[slots] = order[:need.sum()]
        s["table"] = up(table)
        s["refs"] = up(np.bincount(order[:need.sum()], minlength=pages))
        s["missing"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s

    Hk, D = case["Hk"], case["D"]
    if op == "fork":
        b, total = case["beams"], case["prompt"] + r.integers(0, case["drawn"] + 1, N)
        whole, need = case["prompt"] // ps, -(-total // ps)
        # a prompt's whole pages are shared, what follows is each beam's own
        width = -(-(case["prompt"] + case["drawn"]) // ps) + 1
        pages = N * (whole + b * (width - whole + 1)) + 7
        order = r.permutation(pages)
        table = np.full((N, b, width), -1)
        table[:, :, :whole] = order[:N * whole].reshape(N, 1, whole)
        slots = np.arange(whole, width)[None, None] < need[:, None, None]
        tail = order[N * whole:N * whole + N * b * (width - whole)].reshape(N, b, width - whole)
        table[:, :, whole:] = np.where(slots, tail, -1)
        table = table.reshape(N * b, width)
        s["table"], s["lens"] = up(table), up(np.repeat(total, b))
        s["src"] = up(np.arange(N)[:, None] * b + np.minimum(r.geometric(0.4, (N, b)) - 1, b - 1))
        s["src"] = s["src"].view(-1)
        s["refs"] = up(np.bincount(table[table >= 0], minlength=pages))
        s["new_table"], s["new_refs"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        s["copies"] = torch.empty((N * b, 3), dtype=torch.int32, device="cuda")
        s["missing"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["k_cache"], s["v_cache"], _, _ = _pool(case, pages, r, gen)
        return s

    Q, dtype = case["Q"], _TYPES[case["dtype"]]
    if op == "compact":
        lens = r.integers(max(1, case["past"] // 2), case["past"] + 1, N) + Q
        most = case["past"] + Q
    else:
        lens = np.full(N, case["longest"])
        if case["ragged"]:
            lens = r.integers(max(Q, case["longest"] // 8), case["longest"] + 1, N)
            lens[r.integers(0, N)] = case["longest"]
        most = case["longest"]
    width = -(-most // ps)
    slots = np.arange(width)[None] < -(-lens // ps)[:, None]
    if op != "compact" and case["window"]:      # pages that no query sees any more were freed
        at = np.arange(width)[None]
        slots &= (at * ps < case["sinks"]) | ((at + 1) * ps > (lens - Q - case["window"] + 1)[:, None])
    pages = (N * width if op == "compact" else int(slots.sum())) + 3     # outputs: the same size whatever the lengths
    table = np.full((N, width), -1)
    table[slots] = r.permutation(pages)[:slots.sum()]
    s["table"], s["lens"] = up(table), up(lens)
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _pool(case, pages, r, gen)
    parents, sees = _trees(N, Q, r)
    if op == "compact":
        kv = normal((N * Q, 2 * Hk, D), 1.0, dtype)
        s["k"], s["v"] = kv[:, :Hk], kv[:, Hk:]
        depth = sees.sum(-1) - 1
        s["places"] = up((lens[:, None] - Q + np.arange(Q)).reshape(-1))
        s["positions"] = up((lens[:, None] - Q + depth).reshape(-1))
        half = D // 2
        angle = np.arange(most)[:, None] * 10000.0 ** (-np.arange(half) / half)
        s["cos_sin"] = up(np.concatenate([np.cos(angle), np.sin(angle)], 1), np.float32)
        # the accepted path ends at a node drawn among those no deeper than `depth`
        fits = np.where(depth < case["depth"], r.random((N, Q)) + depth, -1.0)
        seen = np.take_along_axis(sees, fits.argmax(1)[:, None, None], 1)[:, 0]
        count = seen.sum(1)
        path = np.full((N, case["depth"]), -1)
        path[np.arange(case["depth"])[None] < count[:, None]] = np.nonzero(seen)[1]
        s["path"], s["count"], s["start"] = up(path), up(count), up(lens - Q)
        return s
    s["q"] = normal((N, Q, case["Hq"], D), 1.5, dtype)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((N, Q, case["Hq"]), dtype=torch.float32, device="cuda")
    s["longest"] = int(case["longest"])
    if op == "tree":
        words = -(-Q // 32)
        bits = np.zeros((N, Q, words * 32), np.uint64)
        bits[:, :, :Q] = sees
        bits = (bits.reshape(N, Q, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
        s["tree"] = up(bits.astype(np.uint32).view(np.int32))
        s["parents"] = up(parents)
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------

def _bits(x):
    """The same values as whole numbers, for indexing any type."""
    return x.view(torch.uint8 if x.element_size() == 1 else torch.int16)


def _plain_attend(s):
    case = s["case"]
    N, Q, Hq, Hk, D, ps = (case[x] for x in ("N", "Q", "Hq", "Hk", "D", "page"))
    G, L = Hq // Hk, s["longest"]
    table = s["table"].long()

    def dense(cache, scale):
        x = _bits(cache)[table.clamp(min=0)].view(cache.dtype).float()   # [N, P, Hk, ps, D]
        x = x.permute(0, 2, 1, 3, 4).reshape(N, Hk, -1, D)[:, :, :L]
        return x if scale is None else x * scale[None, :, None, None]

    past = s["lens"].long()[:, None] - Q                                            # [N, 1]
    node = torch.arange(Q, device="cuda")
    key = torch.arange(L, device="cuda")
    new = key[None] - past                                                          # [N, L]
    if case["op"] == "tree":
        words = s["tree"].long()                                                    # [N, Q, words]
        which = new.clamp(0, Q - 1)[:, None].expand(N, Q, L)
        bit = (words.gather(2, which // 32) >> (which % 32)) & 1
        within = (bit == 1) & ((new >= 0) & (new < Q))[:, None]
        size = ((words[..., None] >> torch.arange(32, device="cuda")) & 1).sum((2, 3))
        pos = past + size - 1
        seen = (new < 0)[:, None].expand(N, Q, L)
    else:
        pos = past + node
        within = torch.zeros((), dtype=torch.bool, device="cuda")
        seen = key <= pos[..., None]
    if case["window"]:
        seen = seen & ((key > pos[..., None] - case["window"]) | (key < case["sinks"]))
    seen = (seen | within) & (table.repeat_interleave(ps, 1)[:, :L] >= 0)[:, None]
    k, v = dense(s["k_cache"], s["k_scale"]), dense(s["v_cache"], s["v_scale"])
    v = torch.where((key < s["lens"][:, None])[:, None, :, None], v, torch.zeros((), device="cuda"))
    q = s["q"].float().view(N, Q, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(N * Hk, Q * G, D)
    z = torch.bmm(q, k.reshape(N * Hk, L, D).transpose(1, 2).contiguous()) * (1.0 / math.sqrt(D))
    z = z.view(N, Hk, Q, G, L).masked_fill(~seen[:, None, :, None], float("-inf"))
    top = z.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), torch.zeros_like(top), top)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    out = torch.bmm(e.view(N * Hk, Q * G, L), v.reshape(N * Hk, L, D)).view(N, Hk, Q, G, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + torch.log(total))[..., 0]
    s["out"].copy_(out.permute(0, 2, 1, 3, 4).reshape(N, Q, Hq, D))
    s["lse"].copy_(lse.permute(0, 2, 1, 3).reshape(N, Q, Hq))
    return s["out"], s["lse"]


def _holders(table, pages):
    """How many entries of the table name each page."""
    ids = table.long().flatten()
    ids = torch.where((ids >= 0) & (ids < pages), ids, pages)
    return torch.zeros(pages + 1, dtype=torch.int32, device="cuda").index_add_(
        0, ids, torch.ones_like(ids, dtype=torch.int32))[:pages]


def _plain_fork(s):
    table, src, refs, ps = s["table"], s["src"].long(), s["refs"], s["case"]["page"]
    (N, W), M, pages = table.shape, src.numel(), refs.numel()
    ok = (src >= 0) & (src < N)
    n = src.clamp(0, N - 1)
    row, length = table[n], s["lens"].long()[n].clamp(0, W * ps)
    full, part = length // ps, length % ps
    slot, m = torch.arange(W, device="cuda"), torch.arange(M, device="cuda")
    new = torch.where(ok[:, None] & (slot * ps < length[:, None]), row, -1)
    last = full.clamp(max=W - 1)[:, None]
    p = row.gather(1, last)[:, 0].long()
    has = ok & (part > 0) & (p >= 0) & (p < pages)
    first = torch.full((N,), M, device="cuda").scatter_reduce_(0, n, torch.where(ok, m, M), "amin")
    stays = (first[n] == m) & (refs[p.clamp(0, pages - 1)] == 1)
    want = has & ~stays
    free = torch.sort((refs != 0).to(torch.int8), stable=True).indices
    rank = torch.cumsum(want, 0) - 1
    got = want & (rank < (refs == 0).sum())
    fresh = free[rank.clamp(0, pages - 1)]
    new.scatter_(1, last, torch.where(want, torch.where(got, fresh, -1), new.gather(1, last)[:, 0])[:, None].int())
    s["new_table"].copy_(new)
    s["new_refs"].copy_(refs - _holders(table, pages) + _holders(new, pages))
    none = torch.tensor([-1, -1, 0], device="cuda")
    s["copies"].copy_(torch.where(got[:, None], torch.stack([p, fresh, part], 1), none))
    s["missing"].copy_((want & ~got).sum())
    p, fresh, part = p[got], fresh[got], part[got]
    within = (torch.arange(ps, device="cuda") < part[:, None])[:, None, :, None]
    k, v = _bits(s["k_cache"]), _bits(s["v_cache"])
    k[fresh] = torch.where(within, k[p], k[fresh])
    v[fresh] = torch.where(within, v[p], v[fresh])
    return s["new_table"], s["new_refs"], s["copies"], s["missing"], s["k_cache"], s["v_cache"]


def _plain_turn(s):
    table, refs, case = s["table"], s["refs"], s["case"]
    ps, (N, W), pages = case["page"], table.shape, refs.numel()
    slot = torch.arange(W, device="cuda")
    keep, want = s["keep"].long()[:, None], s["want"].long()[:, None]
    stays = slot * ps < keep
    if case["window"]:
        stays = stays & ((slot * ps < case["sinks"]) | ((slot + 1) * ps > keep - case["window"] + 1))
    refs.sub_(_holders(torch.where(stays, -1, table), pages))
    table.copy_(torch.where(stays, table, -1))
    wanted = (slot * ps >= keep) & (slot * ps < want) & ((table < 0) | (table >= pages))
    rank = (torch.cumsum(wanted.flatten(), 0) - 1).view(N, W)
    free = torch.sort((refs != 0).to(torch.int8), stable=True).indices
    got = wanted & (rank < (refs == 0).sum())
    table.copy_(torch.where(got, free[rank.clamp(0, pages - 1)].int(), table))
    refs.add_(_holders(torch.where(got, table, -1), pages))
    s["missing"].copy_((wanted & ~got).sum())
    return table, refs, s["missing"]


def _plain_compact(s):
    case, table = s["case"], s["table"].long()
    ps, Q, N = case["page"], case["Q"], case["N"]
    cs = s["cos_sin"][s["positions"].long()][:, None]
    c, sn = cs.chunk(2, -1)
    a, b = s["k"].float().chunk(2, -1)
    turned = torch.cat([a * c - b * sn, b * c + a * sn], -1)

    def stored(x, scale, like):
        if scale is None:
            return x.to(like.dtype)
        return (x / scale[None, :, None]).clamp(-_E4M3_MAX, _E4M3_MAX).to(like.dtype)

    seq = torch.arange(N, device="cuda").repeat_interleave(Q)
    at = s["places"].long()
    page, off = table[seq, at // ps], at % ps
    k, v = _bits(s["k_cache"]), _bits(s["v_cache"])
    k[page, :, off] = _bits(stored(turned, s["k_scale"], s["k_cache"]))
    v[page, :, off] = _bits(stored(s["v"].float(), s["v_scale"], s["v_cache"]))
    j = torch.arange(case["depth"], device="cuda")
    there = j < s["count"][:, None]
    seq = torch.arange(N, device="cuda")[:, None].expand_as(there)[there]
    start = s["start"].long()[:, None]
    old, new = (start + s["path"].long())[there], (start + j)[there]
    fp, fo, tp, to = table[seq, old // ps], old % ps, table[seq, new // ps], new % ps
    k[tp, :, to] = k[fp, :, fo]
    v[tp, :, to] = v[fp, :, fo]
    return s["k_cache"], s["v_cache"]


def _plain_beams(s):
    case = s["case"]
    N, beams, K, V = case["N"], case["beams"], case["K"], case["V"]
    z = s["base"][:, :V].float()
    if s["bias"] is not None:
        z = (z + s["bias"][:, :V].float()).to(torch.bfloat16).float()
    top = z.amax(-1, keepdim=True)
    total = torch.exp((z - top).double()).sum(-1, keepdim=True)
    z, ids = torch.sort(z, dim=-1, descending=True, stable=True)
    k = min(K, V)
    logp = (z[:, :k].double() - top.double()) - torch.log(total)
    score = (s["scores"].double()[:, None] + logp).view(N, beams * k)
    score, at = torch.sort(score, dim=-1, descending=True, stable=True)
    at, score = at[:, :K], score[:, :K]
    s["best"].copy_(score)
    s["rows"].copy_(at // k + torch.arange(N, device="cuda")[:, None] * beams)
    s["ids"].copy_(ids[:, :k].reshape(N, beams * k).gather(1, at))
    rows = s["rows"].long().flatten()
    s["new_history"].copy_(s["history"][rows])
    s["new_hidden"].copy_(s["hidden"][rows])
    return s["best"], s["rows"], s["ids"], s["new_history"], s["new_hidden"]


def run(state):
    case, s = state["case"], state
    op = case["op"]
    if not own:
        return {"tree": _plain_attend, "sinks": _plain_attend, "fork": _plain_fork, "turn": _plain_turn,
                "compact": _plain_compact, "beams": _plain_beams}[op](state)
    from vocab_wide_add_amd import native
    if op == "tree":
        native.xpress_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["tree"],
                                     s["out"], s["longest"], lse=s["lse"], window=case["window"],
                                     sinks=case["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"], s["lse"]
    if op == "sinks":
        native.xpress_sink_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["out"],
                                     s["longest"], case["window"], case["sinks"], lse=s["lse"],
                                     k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"], s["lse"]
    if op == "fork":
        native.xpress_kv_fork(s["refs"], s["table"], s["lens"], s["src"], s["new_refs"], s["new_table"],
                              s["copies"], case["page"], missing=s["missing"])
        native.xpress_kv_copy(s["k_cache"], s["v_cache"], s["copies"])
        return s["new_table"], s["new_refs"], s["copies"], s["missing"], s["k_cache"], s["v_cache"]
    if op == "turn":
        native.xpress_kv_free(s["refs"], s["table"], s["keep"], case["page"], window=case["window"],
                              sinks=case["sinks"])
        native.xpress_kv_grow(s["refs"], s["table"], s["keep"], s["want"], case["page"], missing=s["missing"])
        return s["table"], s["refs"], s["missing"]
    if op == "compact":
        native.xpress_kv_append_at(None, s["k"], s["v"], None, s["k_cache"], s["v_cache"], s["table"],
                                   s["places"], s["positions"], s["cos_sin"], k_scale=s["k_scale"],
                                   v_scale=s["v_scale"])
        native.xpress_kv_compact(s["k_cache"], s["v_cache"], s["table"], s["start"], s["path"], s["count"])
        return s["k_cache"], s["v_cache"]
    stride = case["V"] + case["pad"]
    native.xpress_beam_select(s["base"], s["bias"], s["scores"], s["best"], s["rows"], s["ids"], case["N"],
                              case["beams"], case["V"], case["K"], stride, stride)
    native.xpress_beam_reorder([(s["history"], s["new_history"]), (s["hidden"], s["new_hidden"])], s["rows"])
    return s["best"], s["rows"], s["ids"], s["new_history"], s["new_hidden"]


# ---------------------------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------------------------

def work(case):
    op, N = case["op"], case["N"]
    if op == "beams":
        rows, K = N * case["beams"], case["K"]
        state = case["history"] * 8 + case["hidden"] * 2
        return {"bytes": rows * (case["V"] * (4 if case["bias"] else 2) + 4) + N * K * (16 + 2 * state),
                "flops": rows * case["V"] * 5}
    ps = case["page"]
    if op == "turn":
        width = -(-(case["longest"] + case["more"]) // ps)
        return {"bytes": N * width * 8 + (N * width + 5) * 8 + N * 8, "flops": N * width}
    Hk, D, cb = case["Hk"], case["D"], _BYTES[case["cache"]]
    if op == "fork":
        b, width = case["beams"], -(-(case["prompt"] + case["drawn"]) // ps) + 1
        whole = case["prompt"] // ps
        pages = N * (whole + b * (width - whole + 1)) + 7
        copied = N * b * 0.6 * ps / 2                      # tokens: about so many beams share a parent
        return {"bytes": 2 * N * b * width * 4 + 2 * pages * 4 + N * b * 20 + copied * Hk * D * 4 * cb,
                "flops": N * b * width}
    Q = case["Q"]
    if op == "compact":
        moved = N * case["depth"] * 0.7
        return {"bytes": N * Q * (2 * Hk * D * (_BYTES[case["dtype"]] + cb) + 8 + D * 4) + moved * 4 * Hk * D * cb,
                "flops": N * Q * Hk * D * 3}
    Hq, b = case["Hq"], _BYTES[case["dtype"]]
    span = case["longest"] * (9 / 16 if case["ragged"] else 1)   # the mean drawn length
    if case["window"]:
        span = min(span, case["window"] + case["sinks"] + Q - 1)
    return {"bytes": N * (2 * span * Hk * D * cb + Q * Hq * (2 * D * b + 4)), "flops": N * Q * Hq * span * D * 4}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_attend(s):
    case = s["case"]
    N, Q, Hq, Hk, D, ps = (case[x] for x in ("N", "Q", "Hq", "Hk", "D", "page"))
    out = torch.zeros((N, Q, Hq, D), dtype=torch.float64)
    lse = torch.full((N, Q, Hq), float("-inf"), dtype=torch.float64)
    table = s["table"].cpu().numpy()
    parents = s["parents"].cpu().numpy() if case["op"] == "tree" else None
    for n, length in enumerate(s["lens"].tolist()):
        past = length - Q
        there = np.repeat(table[n] >= 0, ps)[:length]
        sets = []                                            # the keys that each query sees
        for i in range(Q):
            line = list(range(i + 1))
            if parents is not None:                          # a node and those above it
                line = [i]
                while parents[n, line[-1]] >= 0:
                    line.append(int(parents[n, line[-1]]))
            pos = past + len(line) - 1
            key = np.arange(length)
            see = key < past
            if parents is None:
                see = key <= pos
            if case["window"]:
                see &= (key >= pos - case["window"] + 1) | (key < case["sinks"])
            if parents is not None:
                see[past + np.array(line)] = True
            sets.append(see & there)
        used = np.flatnonzero(np.any(sets, 0))
        at = torch.from_numpy(used).cuda()
        page, off = torch.from_numpy(table[n, used // ps].astype(np.int64)).cuda(), at % ps
        k, v = (_bits(c)[page, :, off].view(c.dtype).double() for c in (s["k_cache"], s["v_cache"]))  # [keys, Hk, D]
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
        see = torch.from_numpy(np.array(sets)[:, used]).cuda()
        for h in range(Hk):
            q = s["q"][n, :, h * (Hq // Hk):(h + 1) * (Hq // Hk)].double()                # [Q, G, D]
            z = (q.reshape(-1, D) @ k[:, h].t().contiguous()).view(Q, -1, len(used)) / math.sqrt(D)
            z = torch.where(see[:, None], z, float("-inf"))
            total = torch.logsumexp(z, -1)
            w = torch.nan_to_num(torch.exp(z - total[..., None]), nan=0.0)
            o = (w.view(-1, len(used)) @ v[:, h].contiguous()).view(Q, -1, D)
            out[n, :, h * (Hq // Hk):(h + 1) * (Hq // Hk)] = o.cpu()
            lse[n, :, h * (Hq // Hk):(h + 1) * (Hq // Hk)] = total.cpu()
    return out, lse


def _exact_fork(s):
    table, lens, src, refs = (s[x].cpu().numpy() for x in ("table", "lens", "src", "refs"))
    ps, free = s["case"]["page"], list(np.flatnonzero(refs == 0)[::-1])
    new, copies, missing = np.full((len(src), table.shape[1]), -1), [], 0
    taken = set()
    for m, n in enumerate(src):
        full, part = divmod(int(lens[n]), ps)
        new[m, :full] = table[n, :full]
        copies.append((-1, -1, 0))
        if part:
            p = int(table[n, full])
            if n not in taken and refs[p] == 1:
                new[m, full] = p
            elif free:
                new[m, full] = free.pop()
                copies[-1] = (p, int(new[m, full]), part)
            else:
                missing += 1
        taken.add(n)
    count = refs.copy()
    np.subtract.at(count, table[table >= 0], 1)
    np.add.at(count, new[new >= 0], 1)
    caches = []
    for c in (s["k_cache"], s["v_cache"]):
        x = c.double()
        for a, b, t in copies:
            if b >= 0:
                x[b, :, :t] = x[a, :, :t].clone()
        caches.append(x.cpu())
    whole = [torch.from_numpy(np.asarray(x).astype(np.int32)) for x in (new, count, copies, [missing])]
    return (*whole, *caches)


def _exact_turn(s):
    case = s["case"]
    table, refs = s["table"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy()
    keep, want, ps = s["keep"].tolist(), s["want"].tolist(), case["page"]
    missing = 0
    for n, row in enumerate(table):
        for slot, p in enumerate(row):
            tokens = range(slot * ps, min((slot + 1) * ps, keep[n]))
            seen = len(tokens) > 0
            if case["window"] and seen:      # by the next token, at position keep[n]
                seen = tokens[0] < case["sinks"] or (slot + 1) * ps - 1 > keep[n] - case["window"]
            if p >= 0 and not seen:
                refs[p] -= 1
                row[slot] = -1
    free = list(np.flatnonzero(refs == 0)[::-1])
    for n, row in enumerate(table):
        for slot in range(-(-keep[n] // ps), -(-want[n] // ps)):
            if row[slot] < 0 and free:
                row[slot] = free.pop()
                refs[row[slot]] = 1
            elif row[slot] < 0:
                missing += 1
    return torch.from_numpy(table), torch.from_numpy(refs), torch.tensor([missing], dtype=torch.int32)


def _exact_compact(s):
    case = s["case"]
    ps, Q = case["page"], case["Q"]
    table, places = s["table"].cpu().numpy(), s["places"].cpu().numpy()
    cs = s["cos_sin"].cpu().double()[s["positions"].cpu().long()]
    turn = torch.complex(*cs.chunk(2, -1))[:, None]                  # a pair is one complex number
    y = torch.complex(*(x.contiguous() for x in s["k"].cpu().double().chunk(2, -1))) * turn
    seq = np.arange(len(places)) // Q
    page, off = table[seq, places // ps], places % ps
    caches = []
    for old, x, scale in ((s["k_cache"], torch.cat([y.real, y.imag], -1), s["k_scale"]),
                          (s["v_cache"], s["v"].cpu().double(), s["v_scale"])):
        if scale is not None:
            x = (x / scale.cpu().double()[:, None]).clamp(-_E4M3_MAX, _E4M3_MAX)
        got = old.cpu().to(torch.float64).numpy()
        got[page, :, off] = x.numpy()
        for n, (start, count) in enumerate(zip(s["start"].tolist(), s["count"].tolist())):
            for j, node in enumerate(s["path"][n, :count].tolist()):
                a, b = start + node, start + j
                got[table[n, b // ps], :, b % ps] = got[table[n, a // ps], :, a % ps]
        caches.append(torch.from_numpy(got))
    return caches[0], caches[1]


def _exact_beams(s):
    case = s["case"]
    N, beams, K, V = case["N"], case["beams"], case["K"], case["V"]
    z = s["base"][:, :V].double()
    if s["bias"] is not None:
        z = (z + s["bias"][:, :V].double()).float().to(torch.bfloat16).double()
    z, scores = z.cpu().numpy(), s["scores"].double().cpu().numpy()
    best, rows, ids = [], [], []
    for n in range(N):
        found = []
        for r in range(n * beams, (n + 1) * beams):
            x = z[r]
            total = math.log(np.exp(x - x.max()).sum()) + x.max()
            least = np.partition(x, V - min(K, V))[V - min(K, V)]
            found += [(-(scores[r] + x[v] - total), r, int(v)) for v in np.flatnonzero(x >= least)]
        found = sorted(found)[:K]
        best.append([-f[0] for f in found])
        rows.append([f[1] for f in found])
        ids.append([f[2] for f in found])
    rows = torch.tensor(rows, dtype=torch.int32)
    at = rows.long().flatten()
    return (torch.tensor(best, dtype=torch.float64), rows, torch.tensor(ids), s["history"].cpu()[at],
            s["hidden"].cpu().double()[at])


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_attend, "sinks": _exact_attend, "fork": _exact_fork, "turn": _exact_turn,
            "compact": _exact_compact, "beams": _exact_beams}[case["op"]](s)
