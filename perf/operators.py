"""The serving operators next to the drafting pass, as measured: the append to a paged key-value cache
with position rotation, attention of new tokens over that cache, and the sampled readout.

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

def _append(name, N, T, Hq, Hk, D, rot, page, dtype="bf16", cache="bf16", layout="head",
            interleaved=False, prompt=False, past=0):
    """N sequences; T new tokens each (prompt: packed prompts of different lengths, T in all)."""
    return dict(name=name, op="append", N=N, T=T, Hq=Hq, Hk=Hk, D=D, rot=rot, page=page, dtype=dtype,
                cache=cache, layout=layout, interleaved=interleaved, prompt=prompt, past=past)


def _attend(name, N, Q, Hq, Hk, D, page, longest, ragged, dtype="bf16", cache="bf16", layout="head",
            window=0):
    return dict(name=name, op="attend", N=N, Q=Q, Hq=Hq, Hk=Hk, D=D, page=page, longest=longest,
                ragged=ragged, dtype=dtype, cache=cache, layout=layout, window=window)


def _sample(name, N, B, V, pad, bias, filters):
    return dict(name=name, op="sample", N=N, B=B, V=V, pad=pad, bias=bias, filters=filters)


def listed():
    return [
        # one sequence's next token: pure latency
        _append("append_one", 1, 1, 32, 8, 128, 128, 16, past=1000),
        # a drafted block of 16 for 32 sequences (the framework's N and B) into an 8-bit cache
        _append("append_blocks_e4m3", 32, 16, 32, 8, 128, 128, 64, cache="e4m3", past=2000),
        # packed prompts of different lengths, half of each head rotated in adjacent pairs, token-major pages
        _append("append_prompts", 9, 20011, 32, 8, 128, 64, 16, layout="token", interleaved=True,
                prompt=True),
        # one chat turn of one user: the smallest attention call
        _attend("attend_one", 1, 1, 32, 8, 128, 16, 1009, False),
        # 32 sequences decoding one token each, ragged lengths
        _attend("attend_32", 32, 1, 32, 8, 128, 16, 4096, True),
        # one very long context, few heads: all parallelism comes from the split
        _attend("attend_long", 1, 1, 32, 4, 128, 64, 131072, False),
        # verifying a drafted block of 16 tokens per sequence
        _attend("attend_block", 32, 16, 32, 8, 128, 32, 4096, True),
        # many sequences on an 8-bit cache with small heads
        _attend("attend_e4m3", 128, 1, 32, 8, 64, 64, 6000, True, cache="e4m3"),
        # odd head size and group, a sliding window, token-major pages that end inside every tile
        _attend("attend_window", 24, 3, 35, 5, 80, 24, 9001, True, dtype="fp16", cache="fp16",
                layout="token", window=1777),
        # the next token of one sequence
        _sample("sample_one", 1, 2, 152064, 0, False, "mixed"),
        # one drafted block, rows padded apart, nucleus only
        _sample("sample_block", 1, 16, 151936, 64, True, "top_p"),
        # the framework's own readout shape, sampled
        _sample("sample_480", 32, 16, 152064, 0, True, "mixed"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "sample", "sample"])
    if op == "sample":
        rows = _log_int(rng, 1, 480)
        B = rng.choice([2, 5, 8, 16])
        return dict(op=op, N=max(1, rows // (B - 1)), B=B, V=_log_int(rng, 1000, 152064),
                    pad=rng.choice([0, 0, 64, 7]), bias=rng.random() < 0.6,
                    filters=rng.choice(["none", "top_p", "mixed"]))
    G = rng.choice([1, 2, 4, 5, 7, 8, 16])
    Hk = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 80, 96, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    layout = rng.choice(["head", "token"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "append":
        prompt = rng.random() < 0.5
        N = _log_int(rng, 1, 64)
        most = max(1, 20000 * 48 * 128 // ((G * Hk + 2 * Hk) * D))
        T = _log_int(rng, N, max(N, min(20000, most))) if prompt else rng.choice([1, 1, 4, 16])
        return dict(op=op, N=N, T=T, Hq=G * Hk, Hk=Hk, D=D, rot=rng.choice([D, D, D // 2]), page=page,
                    dtype=dtype, cache=cache, layout=layout, interleaved=rng.random() < 0.4,
                    prompt=prompt, past=_log_int(rng, 1, 5000))
    Q = rng.choice([1, 1, 1, 2, 5, 8, 16])
    N = _log_int(rng, 1, 128)
    most = 32 * 4096 * 8 * 128 // (N * Hk * D)          # cached values as in the listed cases
    work = 32 * 4096 * 16 * 32 * 128 // (N * Q * G * Hk * D)
    longest = _log_int(rng, 17, max(18, min(131072, most, work)))
    return dict(op=op, N=N, Q=Q, Hq=G * Hk, Hk=Hk, D=D, page=page, longest=longest,
                ragged=rng.random() < 0.7, dtype=dtype, cache=cache, layout=layout,
                window=rng.choice([0, 0, 0, _log_int(rng, 16, 4096)]))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _lengths(case, r):
    """Lengths of the sequences, new tokens included."""
    N = case["N"]
    if case["op"] == "append":
        if case["prompt"]:
            cuts = np.sort(r.choice(np.arange(1, max(2, case["T"])), size=N - 1, replace=False)) if N > 1 else []
            return np.diff(np.concatenate([[0], cuts, [case["T"]]])).astype(np.int64)
        return r.integers(0, case["past"] + 1, N) + case["T"]
    if not case["ragged"]:
        return np.full(N, case["longest"], np.int64)
    got = r.integers(max(1, case["longest"] // 8), case["longest"] + 1, N)
    got[r.integers(0, N)] = case["longest"]
    return np.maximum(got, min(case["Q"], case["longest"]))


def _paged(case, lens, r, gen):
    """A pool of pages in random order with stale finite values everywhere, and the sequences' page tables."""
    ps, Hk, D, cache = case["page"], case["Hk"], case["D"], case["cache"]
    need = -(-lens // ps)
    pages = int(need.sum()) + 3
    if case["op"] == "append":   # the same pool whatever the lengths
        pages = (case["T"] // ps + case["N"] if case["prompt"] else
                 case["N"] * -(-(case["past"] + case["T"]) // ps)) + 3
    order = r.permutation(pages).astype(np.int32)
    table = np.full((len(lens), int(need.max())), -1, np.int32)
    at = 0
    for n, c in enumerate(need):
        table[n, :c] = order[at:at + c]
        at += c
    shape = (pages, ps, Hk, D) if case["layout"] == "token" else (pages, Hk, ps, D)
    both = []
    for _ in range(2):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        if cache == "e4m3":
            y = torch.empty(shape, dtype=_TYPES[cache], device="cuda")
            flat, into = x.view(-1), y.view(-1)
            into.copy_((flat * 24.0).clamp_(-_E4M3_MAX, _E4M3_MAX))
            x = y
        else:
            x = x.to(_TYPES[cache])
        both.append(x.transpose(1, 2) if case["layout"] == "token" else x)
    scales = None
    if cache == "e4m3":
        scales = [torch.from_numpy((r.uniform(0.6, 1.4, Hk) / 24.0).astype(np.float32)).cuda() for _ in range(2)]
    return both, scales, torch.from_numpy(table).cuda()


def prepare(case, seed):
    r = np.random.default_rng([seed, 77])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 2 + 1)

    def normal(shape, sigma, dtype):
        x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, sigma, generator=gen)
        return x.to(dtype)

    s = dict(case=case)
    if case["op"] == "sample":
        N, B, V = case["N"], case["B"], case["V"]
        rows = N * (B - 1)
        stride = V + case["pad"]
        s["base"] = normal((rows, stride), 4.0, torch.bfloat16)
        s["bias"] = normal((rows, stride), 0.5, torch.bfloat16) if case["bias"] else None
        s["blk"] = torch.from_numpy(r.integers(0, V, (N, B))).cuda()
        t = r.uniform(0.5, 1.3, rows)
        k = np.zeros(rows, np.int32)
        p = np.ones(rows)
        m = np.zeros(rows)
        if case["filters"] == "top_p":
            p = r.uniform(0.8, 0.98, rows)
        elif case["filters"] == "mixed":   # rows of requests with settings of their own
            kind = r.integers(0, 6, rows)
            k = np.where((kind == 1) | (kind == 3), r.choice([1, 20, 50, 1000], rows), 0).astype(np.int32)
            p = np.where((kind == 2) | (kind == 3), r.uniform(0.7, 0.98, rows), 1.0)
            m = np.where(kind == 4, r.uniform(0.02, 0.2, rows), 0.0)
            t = np.where(kind == 5, 0.0, t)
        for name, v in (("temperature", t), ("top_p", p), ("min_p", m), ("u", r.random(rows, np.float32))):
            s[name] = torch.from_numpy(np.asarray(v, np.float32)).cuda()
        s["top_k"] = torch.from_numpy(k).cuda()
        s["prob"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        return s

    lens = _lengths(case, r)
    (s["k_cache"], s["v_cache"]), scales, s["table"] = _paged(case, lens, r, gen)
    s["k_scale"], s["v_scale"] = scales if scales else (None, None)
    N, Hq, Hk, D, dtype = case["N"], case["Hq"], case["Hk"], case["D"], _TYPES[case["dtype"]]
    if case["op"] == "attend":
        s["q"] = normal((N, case["Q"], Hq, D), 1.5, dtype)
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((N, case["Q"], Hq), dtype=torch.float32, device="cuda")
        s["longest"] = int(case["longest"])
        return s
    if case["prompt"]:
        seq = np.repeat(np.arange(N), lens)
        pos = np.concatenate([np.arange(c) for c in lens])
    else:
        seq = np.repeat(np.arange(N), case["T"])
        pos = (lens[:, None] - case["T"] + np.arange(case["T"])).reshape(-1)
    T = len(pos)
    # q, k and v are slices of one projection's rows
    qkv = normal((T, Hq + 2 * Hk, D), 1.0, dtype)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    s["q_out"] = torch.empty((T, Hq, D), dtype=dtype, device="cuda")
    s["seq"] = torch.from_numpy(seq.astype(np.int32)).cuda()
    s["pos"] = torch.from_numpy(pos.astype(np.int32)).cuda()
    half = case["rot"] // 2
    angle = np.arange(int(lens.max()))[:, None] * 10000.0 ** (-np.arange(half) / half)
    s["cos_sin"] = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------

def _bits(x):
    """The same values as whole numbers, for indexing any type."""
    return x.view(torch.uint8 if x.element_size() == 1 else torch.int16)


def _plain_append(s):
    case = s["case"]
    rot, half, ps = case["rot"], case["rot"] // 2, case["page"]
    cs = s["cos_sin"][s["pos"].long()][:, None]
    c, sn = cs[..., :half], cs[..., half:]

    def rotated(x):
        x = x.float()
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:rot]
            y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
        return torch.cat([y, x[..., rot:]], -1)

    def stored(x, scale, like):
        if scale is None:
            return x.to(like.dtype)
        return (x / scale[None, :, None]).clamp(-_E4M3_MAX, _E4M3_MAX).to(like.dtype)

    page = s["table"][s["seq"].long(), s["pos"].long() // ps].long()
    off = s["pos"].long() % ps
    s["q_out"].copy_(rotated(s["q"]))
    _bits(s["k_cache"])[page, :, off] = _bits(stored(rotated(s["k"]), s["k_scale"], s["k_cache"]))
    _bits(s["v_cache"])[page, :, off] = _bits(stored(s["v"].float(), s["v_scale"], s["v_cache"]))
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_attend(s):
    case = s["case"]
    N, Q, Hq, Hk, D, ps = (case[x] for x in ("N", "Q", "Hq", "Hk", "D", "page"))
    G, L = Hq // Hk, s["longest"]
    table = s["table"].long()

    def dense(cache, scale):
        x = _bits(cache)[table.clamp(min=0)].view(cache.dtype).float()   # [N, P, Hk, ps, D]
        x = x.permute(0, 2, 1, 3, 4).reshape(N, Hk, -1, D)[:, :, :L]
        return x if scale is None else x * scale[None, :, None, None]

    pos = s["lens"].long()[:, None] - Q + torch.arange(Q, device="cuda")          # [N, Q]
    key = torch.arange(L, device="cuda")
    seen = key <= pos[..., None]                                                    # [N, Q, L]
    if case["window"]:
        seen = seen & (key > pos[..., None] - case["window"])
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


def _plain_sample(s):
    case = s["case"]
    N, B, V = case["N"], case["B"], case["V"]
    z = s["base"][:, :V].float()
    if s["bias"] is not None:
        z = (z + s["bias"][:, :V].float()).to(torch.bfloat16).float()
    z = torch.where(z.isnan(), float("-inf"), z)
    z, ids = torch.sort(z, dim=-1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    greedy = ~(t > 0)
    w = torch.exp((z.double() - z[:, :1].double()) / torch.where(greedy, 1.0, t))
    w = torch.where(z == z[:, :1], 1.0, w)
    rank = torch.arange(V, device="cuda")
    k = s["top_k"].long()[:, None]
    keep = ((rank < k) | (k <= 0)) & (~greedy | (rank < 1))
    w = w * keep
    before = torch.cumsum(w, -1) - w
    whole = (before + w)[:, -1:]
    p, m = s["top_p"].double()[:, None], s["min_p"].double()[:, None]
    keep &= (before < p * whole) | (p >= 1) | (rank < 1)
    keep &= (w >= m) | (rank < 1)
    w = w * keep
    c = torch.cumsum(w, -1)
    j = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(-1, keepdim=True)
    last = (w > 0).sum(-1, keepdim=True) - 1
    j = torch.minimum(j, last)
    s["blk"][:, 1:] = ids.gather(-1, j).view(N, B - 1)
    s["prob"].copy_((w.gather(-1, j) / c[:, -1:])[:, 0])
    return s["blk"], s["prob"]


def run(state):
    case = state["case"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "sample": _plain_sample}[case["op"]](state)
    from vocab_wide_add_amd import native
    s = state
    if case["op"] == "append":
        native.xpress_kv_append(s["q"], s["k"], s["v"], s["q_out"], s["k_cache"], s["v_cache"], s["table"],
                                s["pos"], s["cos_sin"], seq_of=s["seq"], k_scale=s["k_scale"],
                                v_scale=s["v_scale"], interleaved=case["interleaved"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if case["op"] == "attend":
        native.xpress_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["out"],
                                      s["longest"], lse=s["lse"], window=case["window"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"], s["lse"]
    stride = case["V"] + case["pad"]
    native.xpress_sample_to_blk(s["base"], s["bias"], s["blk"], s["temperature"], s["top_k"], s["top_p"],
                                s["min_p"], s["u"], case["N"], case["B"], case["V"], stride, stride,
                                prob=s["prob"])
    return s["blk"], s["prob"]


# ---------------------------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "sample":
        rows = case["N"] * (case["B"] - 1)
        return {"bytes": rows * (case["V"] * (4 if case["bias"] else 2) + 32), "flops": rows * case["V"] * 8}
    Hq, Hk, D, b, cb = case["Hq"], case["Hk"], case["D"], _BYTES[case["dtype"]], _BYTES[case["cache"]]
    if case["op"] == "append":
        T = case["T"] if case["prompt"] else case["N"] * case["T"]
        return {"bytes": T * ((2 * Hq + 2 * Hk) * D * b + 2 * Hk * D * cb + 12 + case["rot"] * 4),
                "flops": T * (Hq + Hk) * case["rot"] * 3}
    Q, span = case["Q"], case["longest"] * (9 / 16 if case["ragged"] else 1)   # the mean drawn length
    if case["window"]:
        span = min(span, case["window"] + Q - 1)
    return {"bytes": case["N"] * (2 * span * Hk * D * cb + Q * Hq * (2 * D * b + 4)),
            "flops": case["N"] * Q * Hq * span * D * 4}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_append(s):
    case = s["case"]
    rot = case["rot"]
    pos, seq = s["pos"].cpu().numpy(), s["seq"].cpu().numpy()
    cs = s["cos_sin"].cpu().double()[torch.from_numpy(pos).long()]
    turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None]    # a pair is one complex number

    def rotated(x):
        x = x.cpu().double()
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["interleaved"] else x[..., :rot].chunk(2, -1)
        y = torch.complex(a.contiguous(), b.contiguous()) * turn
        y = torch.view_as_real(y).flatten(-2) if case["interleaved"] else torch.cat([y.real, y.imag], -1)
        return torch.cat([y, x[..., rot:]], -1)

    table = s["table"].cpu().numpy()
    page, off = table[seq, pos // case["page"]], pos % case["page"]
    caches = []
    for old, new, scale in ((s["k_cache"], rotated(s["k"]), s["k_scale"]),
                            (s["v_cache"], s["v"].cpu().double(), s["v_scale"])):
        if scale is not None:
            new = (new / scale.cpu().double()[:, None]).clamp(-_E4M3_MAX, _E4M3_MAX)
        got = old.cpu().to(torch.float64).numpy()
        got[page, :, off] = new.numpy()
        caches.append(torch.from_numpy(got))
    return rotated(s["q"]), caches[0], caches[1]


def _exact_attend(s):
    case = s["case"]
    N, Q, Hq, Hk, D, ps = (case[x] for x in ("N", "Q", "Hq", "Hk", "D", "page"))
    out = torch.zeros((N, Q, Hq, D), dtype=torch.float64)
    lse = torch.full((N, Q, Hq), float("-inf"), dtype=torch.float64)
    for n, length in enumerate(s["lens"].tolist()):
        pages = s["table"][n, :-(-length // ps)].long()
        k, v = (_bits(c)[pages].view(c.dtype).transpose(0, 1).double().reshape(Hk, -1, D)[:, :length]
                for c in (s["k_cache"], s["v_cache"]))
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"].double()[:, None, None], v * s["v_scale"].double()[:, None, None]
        k, v = (x.repeat_interleave(Hq // Hk, 0) for x in (k, v))
        for i in range(Q):
            last = length - Q + i
            first = max(0, last - case["window"] + 1) if case["window"] else 0
            if last < first:
                continue
            z = (k[:, first:last + 1] * s["q"][n, i].double()[:, None]).sum(-1) / math.sqrt(D)
            total = torch.logsumexp(z, -1)
            out[n, i] = ((z - total[:, None]).exp()[..., None] * v[:, first:last + 1]).sum(1).cpu()
            lse[n, i] = total.cpu()
    return out, lse


def _exact_sample(s):
    case = s["case"]
    N, B, V = case["N"], case["B"], case["V"]
    z = s["base"][:, :V].double()
    if s["bias"] is not None:
        z = (z + s["bias"][:, :V].double()).float().to(torch.bfloat16).double()   # both roundings exact enough
    z = z.cpu().numpy()
    per = {x: s[x].double().cpu().numpy() for x in ("temperature", "top_k", "top_p", "min_p", "u")}
    ids, probs = [], []
    for row in range(N * (B - 1)):
        x, t = z[row], per["temperature"][row]
        values, counts = np.unique(x[x == x], return_counts=True)          # groups of equal logits
        values, counts = values[::-1], counts[::-1].astype(np.float64)
        if not t > 0:
            ids.append(int(np.argmax(x == values[0])))
            probs.append(1.0)
            continue
        w = np.exp((values - values[0]) / t)
        k, p, m = per["top_k"][row], per["top_p"][row], per["min_p"][row]
        n = counts if k <= 0 else np.diff(np.concatenate([[0.0], np.minimum(np.cumsum(counts), k)]))
        before = np.concatenate([[0.0], np.cumsum(n * w)])
        if p < 1:
            left = np.ceil((p * before[-1] - before[:-1]) / np.maximum(w, 1e-300))
            n = np.minimum(n, np.maximum(left, 0.0))
            n[0] = max(n[0], 1.0)
        n = n * (w >= m)
        n[0] = max(n[0], 1.0)
        c = np.cumsum(n * w)
        goal = per["u"][row] * c[-1]
        g = min(int(np.searchsorted(c, goal, side="right")), int(np.flatnonzero(n * w)[-1]))
        j = min(int((goal - (c[g] - n[g] * w[g])) / w[g]), int(n[g]) - 1)
        ids.append(int(np.flatnonzero(x == values[g])[max(j, 0)]))
        probs.append(w[g] / c[-1])
    blk = s["blk"].cpu().clone()
    blk[:, 1:] = torch.tensor(ids).view(N, B - 1)
    return blk, torch.tensor(probs, dtype=torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attend":
        # the listed block case is the most that the loop over queries does in time
        if case["N"] * case["Q"] * case["Hq"] * case["longest"] * case["D"] > 32 * 16 * 32 * 4096 * 128:
            return None
        return _exact_attend(s)
    return _exact_sample(s)
