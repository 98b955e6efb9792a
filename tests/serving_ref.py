"""Plain implementations in 64 bits of the serving operators (append to a paged
cache, attention over it, sampled readout), and the inputs the tests give them."""
from __future__ import annotations

import math

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


def half_step(dtype) -> float:
    """Largest relative error of one rounding to the type."""
    return torch.finfo(dtype).eps / 2


def paged_pool(rng, lens, Hk, D, page, cache, layout="head", fill=None, spare=2, table_extra=1):
    """Random pages for sequences of the given lengths: (k, v) CPU caches viewed
    [pages, Hk, page, D], an int32 page table (unused entries -1) and the pages'
    number.  Every place is drawn; `fill`, if given, goes into all places that
    hold no token."""
    need = [-(-int(x) // page) for x in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(need), max(max(need, default=0), 1) + table_extra), -1, np.int32)
    at = 0
    used = np.zeros((pages, page), bool)
    for n, c in enumerate(need):
        table[n, :c] = order[at:at + c]
        at += c
        for j in range(int(lens[n])):
            used[table[n, j // page], j % page] = True
    caches = []
    for _ in range(2):
        x = torch.from_numpy(rng.standard_normal((pages, Hk, page, D)).astype(np.float32))
        if cache == "e4m3":
            x = x * 16
        if fill is not None:
            x = torch.where(torch.from_numpy(used)[:, None, :, None], x, torch.tensor(float(fill)))
        x = x.to(TYPES[cache])
        if layout == "token":
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        caches.append(x)
    return caches[0], caches[1], torch.from_numpy(table)


def append64(q, k, v, kc, vc, table, pos, seq, cos_sin, k_scale, v_scale, interleaved):
    """(q_out, k cache, v cache, places written [pages, page]) in float64; caches as
    stored codes before their rounding."""
    rot = cos_sin.shape[1] if cos_sin is not None else 0
    pages, Hk, page, D = kc.shape
    out = np.zeros(q.shape)
    kcd, vcd = kc.double().numpy().copy(), vc.double().numpy().copy()
    written = np.zeros((pages, page), bool)
    for t in range(k.shape[0]):
        p, n = int(pos[t]), int(seq[t])
        if (p < 0 or (cos_sin is not None and p >= cos_sin.shape[0]) or not 0 <= n < table.shape[0]
                or p // page >= table.shape[1]):
            continue

        def rotated(x):
            x = x.double().numpy().copy()
            for i in range(rot // 2):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
                c, s = float(cos_sin[p, i]), float(cos_sin[p, rot // 2 + i])
                x[:, a], x[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
            return x
        out[t] = rotated(q[t])
        g = int(table[n, p // page])
        if 0 <= g < pages:
            ks = k_scale.double().numpy()[:, None] if k_scale is not None else 1.0
            vs = v_scale.double().numpy()[:, None] if v_scale is not None else 1.0
            kcd[g, :, p % page] = rotated(k[t]) / ks
            vcd[g, :, p % page] = v[t].double().numpy() / vs
            written[g, p % page] = True
    return out, kcd, vcd, written


def attention64(q, kc, vc, table, lens, max_len, scale, window=0, k_scale=None, v_scale=None):
    """(out, lse, |.|-weighted values, largest sum of |q_d k_d| * scale) in float64."""
    N, Q, Hq, D = q.shape
    pages, Hk, page, _ = kc.shape
    G = Hq // Hk
    out, absv = np.zeros(q.shape), np.zeros(q.shape)
    lse, reach = np.full((N, Q, Hq), -np.inf), np.zeros((N, Q, Hq))
    kd, vd = kc.double().numpy(), vc.double().numpy()
    for n in range(N):
        length = min(max(int(lens[n]), 0), max_len)
        for i in range(Q):
            pos = length - Q + i
            js = [j for j in range(max(0, pos - window + 1) if window > 0 else 0, pos + 1)
                  if 0 <= int(table[n, j // page]) < pages]
            if not js:
                continue
            g = np.array([int(table[n, j // page]) for j in js])
            o = np.array([j % page for j in js])
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


def sample64(z, temperature, top_k, top_p, min_p, u):
    """(ids, probs) of float64 logits [rows, V] by sorting."""
    ids, probs = [], []
    for r in range(z.shape[0]):
        x = np.where(np.isnan(z[r]), -np.inf, z[r])
        top = x.max()
        if top == -np.inf:
            ids.append(0)
            probs.append(0.0)
            continue
        t = float(temperature[r])
        order = np.lexsort((np.arange(len(x)), -x))
        if not t > 0:
            ids.append(int(order[0]))
            probs.append(1.0)
            continue
        y = x[order]
        with np.errstate(invalid="ignore", over="ignore"):
            w = np.where(y == top, 1.0, np.where(y == -np.inf, 0.0, np.exp((y - top) / t)))
        k, p, m = int(top_k[r]), float(top_p[r]), float(min_p[r])
        keep = len(y)
        if k > 0:
            keep = min(keep, k)
        before = np.concatenate([[0.0], np.cumsum(w[:keep])])
        if p < 1:
            keep = min(keep, max(1, int((before[:-1] < p * before[-1]).sum())))
        if m > 0:
            keep = min(keep, max(1, int((w >= m).sum())))
        c = np.cumsum(w[:keep])
        g = float(u[r])
        g = 0.0 if not g > 0 else min(g, 1 - 2.0 ** -24)
        j = int((c <= g * c[-1]).sum())
        ids.append(int(order[j]))
        probs.append(w[j] / c[-1])
    return np.array(ids), np.array(probs)
