"""Plain implementations in 64 bits of the operators for drafts that branch and for beams:
attention of a tree, attention with a window and sinks, the pages of a cache, and beam
search's selection."""
from __future__ import annotations

import math

import numpy as np
import torch


def words_of(sees) -> torch.Tensor:
    """int32 words [..., Q, ceil(Q / 32)] of truth values [..., Q, Q]."""
    sees = np.asarray(sees, bool)
    Q = sees.shape[-1]
    words = -(-Q // 32)
    bits = np.zeros(sees.shape[:-1] + (words * 32,), np.uint64)
    bits[..., :Q] = sees
    bits = (bits.reshape(sees.shape[:-1] + (words, 32)) << np.arange(32, dtype=np.uint64)).sum(-1)
    return torch.from_numpy(bits.astype(np.uint32).view(np.int32))


def random_trees(rng, N, Q):
    """(parents [N, Q], sees [N, Q, Q]): a node sees itself and those above it."""
    parents = np.full((N, Q), -1)
    sees = np.zeros((N, Q, Q), bool)
    for n in range(N):
        for i in range(Q):
            if i:
                parents[n, i] = rng.integers(max(0, i - 5), i)
                sees[n, i] = sees[n, parents[n, i]]
            sees[n, i, i] = True
    return parents, sees


def visible(length, Q, window, sinks, sees=None):
    """Truth values [Q, length]: which places each query sees."""
    past = length - Q
    out = np.zeros((Q, length), bool)
    for i in range(Q):
        pos = past + (i if sees is None else int(sees[i].sum()) - 1)
        for j in range(length):
            if sees is not None and j >= past:
                out[i, j] = sees[i, j - past]
            else:
                ok = j <= pos if sees is None else True
                out[i, j] = ok and (window == 0 or j > pos - window or j < sinks)
    return out


def attention64(q, kc, vc, table, lens, max_len, scale, window=0, sinks=0, sees=None, k_scale=None,
                v_scale=None):
    """(out, lse, |.|-weighted values, largest sum of |q_d k_d| * scale) in float64; sees
    [N, Q, Q] for a tree."""
    N, Q, Hq, D = q.shape
    pages, Hk, page, _ = kc.shape
    G = Hq // Hk
    out, absv = np.zeros(q.shape), np.zeros(q.shape)
    lse, reach = np.full((N, Q, Hq), -np.inf), np.zeros((N, Q, Hq))
    kd, vd = kc.double().numpy(), vc.double().numpy()
    for n in range(N):
        length = min(max(int(lens[n]), 0), max_len)
        see = visible(length, Q, window, sinks, None if sees is None else sees[n])
        for i in range(Q):
            js = np.array([j for j in np.flatnonzero(see[i]) if 0 <= int(table[n, j // page]) < pages], int)
            if not len(js):
                continue
            g = np.array([int(table[n, j // page]) for j in js])
            o = js % page
            for h in range(Hq):
                K, V = kd[g, h // G, o], vd[g, h // G, o]
                if k_scale is not None:
                    K, V = K * float(k_scale[h // G]), V * float(v_scale[h // G])
                x = q[n, i, h].double().numpy()
                z = K @ x * scale
                top = z.max()
                w = np.exp(z - top)
                lse[n, i, h] = top + math.log(w.sum())
                out[n, i, h] = w @ V / w.sum()
                absv[n, i, h] = w @ np.abs(V) / w.sum()
                reach[n, i, h] = (np.abs(K) @ np.abs(x)).max() * abs(scale)
    return out, lse, absv, reach


def fork(refs, table, lens, src, page):
    """(new refs, new table, copies, missing) of int arrays."""
    refs, table, pages, width = np.asarray(refs), np.asarray(table), len(refs), np.asarray(table).shape[1]
    free = [p for p in range(pages) if refs[p] == 0][::-1]
    new, copies = np.full((len(src), width), -1), np.tile([-1, -1, 0], (len(src), 1))
    missing, seen = 0, set()
    for m, n in enumerate(np.asarray(src).tolist()):
        if not 0 <= n < len(table):
            continue
        whole, part = divmod(min(max(int(lens[n]), 0), width * page), page)
        new[m, :whole] = table[n, :whole]
        if part:
            p = int(table[n, whole])
            if not 0 <= p < pages or (n not in seen and refs[p] == 1):
                new[m, whole] = p
            elif free:
                new[m, whole] = free.pop()
                copies[m] = p, new[m, whole], part
            else:
                missing += 1
        seen.add(n)
    count = refs.astype(np.int64).copy()
    for t, by in ((table, -1), (new, 1)):
        for p in t.flatten().tolist():
            if 0 <= p < pages:
                count[p] += by
    return count, new, copies, missing


def copy(cache, copies):
    """The cache [pages, heads, page, dim] after the copies, in its own type."""
    out = cache.clone()
    pages, _, page, _ = cache.shape
    for a, b, t in np.asarray(copies).tolist():
        if 0 <= a < pages and 0 <= b < pages:
            t = min(max(t, 0), page)
            out[b, :, :t] = cache[a, :, :t]
    return out


def grow(refs, table, have, want, page):
    refs, table = np.asarray(refs).copy(), np.asarray(table).copy()
    free = [p for p in range(len(refs)) if refs[p] == 0][::-1]
    missing = 0
    for n in range(len(table)):
        for s in range(-(-max(int(have[n]), 0) // page), min(-(-max(int(want[n]), 0) // page), table.shape[1])):
            if 0 <= table[n, s] < len(refs):
                continue
            if free:
                table[n, s] = free.pop()
                refs[table[n, s]] = 1
            else:
                missing += 1
    return refs, table, missing


def free(refs, table, lens, page, window=0, sinks=0):
    refs, table = np.asarray(refs).copy(), np.asarray(table).copy()
    for n in range(len(table)):
        length = int(lens[n])
        for s in range(table.shape[1]):
            held = [j for j in range(s * page, (s + 1) * page) if j < length]
            # the token at position `length` and those after it see nothing earlier
            if held and (window == 0 or held[0] < sinks or (s + 1) * page - 1 > length - window):
                continue
            if 0 <= table[n, s] < len(refs):
                refs[table[n, s]] -= 1
            table[n, s] = -1
    return refs, table


def compact(cache, table, start, path, count):
    """The cache after the moves, in its own type."""
    out = cache.clone()
    pages, _, page, _ = cache.shape
    width = table.shape[1]

    def find(n, place):
        if place // page >= width or not 0 <= int(table[n, place // page]) < pages:
            return None
        return int(table[n, place // page]), place % page

    for n in range(len(start)):
        if int(start[n]) < 0:
            continue
        before = -1
        for j in range(min(int(count[n]), path.shape[1])):
            node = int(path[n, j])
            if node <= before:
                break
            before = node
            a, b = find(n, int(start[n]) + node), find(n, int(start[n]) + j)
            if a and b:
                out[b[0], :, b[1]] = cache[a[0], :, a[1]]
    return out


def beams(z, scores, N, beams, K):
    """(scores, rows, ids) [N, K] of float64 logits [N * beams, V]."""
    best, rows, ids = np.full((N, K), -np.inf), np.full((N, K), -1), np.full((N, K), -1)
    for n in range(N):
        found = []
        for r in range(n * beams, (n + 1) * beams):
            x = np.where(np.isnan(z[r]), -np.inf, z[r])
            top = x.max()
            if top == -np.inf or not np.isfinite(scores[r]):
                continue
            with np.errstate(invalid="ignore"):
                d = np.where(x == top, 0.0, x - top)
            total = math.log(math.fsum(np.exp(d)))
            order = np.lexsort((np.arange(len(x)), -x))[:K]
            found += [(-((float(scores[r]) - total) + d[v]), r, -x[v], int(v)) for v in order if d[v] > -np.inf]
        for k, f in enumerate(sorted(found)[:K]):
            best[n, k], rows[n, k], ids[n, k] = -f[0], f[1], f[3]
    return best, rows, ids
