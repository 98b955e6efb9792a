"""The pages of a cache: xpress_kv_fork, xpress_kv_copy, xpress_kv_grow, xpress_kv_free,
xpress_kv_compact and xpress_kv_append_at.  Whole numbers and copied bytes: equal."""
import numpy as np
import pytest
import torch

import drafts_ref as ref
import serving_ref
from gpu_util import say
from vocab_wide_add_amd import native

TYPES = serving_ref.TYPES


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x).astype(np.int32)))


def holders(table, pages):
    table = np.asarray(table)
    return np.bincount(table[(table >= 0) & (table < pages)], minlength=pages)


def shared_table(rng, N, width, pages, share=0.4, holes=0.1):
    """Rows that share pages here and there, with entries that name none, and the counts."""
    table = np.full((N, width), -1)
    order = rng.permutation(pages)
    at = 0
    for n in range(N):
        for s in range(width):
            if n and rng.random() < share:
                table[n, s] = table[rng.integers(0, n), s]
            elif rng.random() < holes:
                table[n, s] = rng.choice([-1, -7, pages, 2 ** 31 - 1])
            elif at < pages:
                table[n, s] = order[at]
                at += 1
    return table, holders(table, pages)


def run_fork(refs, table, lens, src, page, missing=True, stride=0):
    pages, (N, W), M = len(refs), np.asarray(table).shape, len(src)
    new_refs = torch.full((pages,), 99, dtype=torch.int32, device="cuda")
    wide = torch.full((M, W + stride), 77, dtype=torch.int32, device="cuda")
    copies = torch.full((M, 3), 55, dtype=torch.int32, device="cuda")
    short = torch.full((1,), 44, dtype=torch.int32, device="cuda") if missing else None
    r, t = i32(refs).cuda(), i32(table).cuda()
    native.xpress_kv_fork(r, t, i32(lens).cuda(), i32(src).cuda(), new_refs, wide[:, :W], copies, page, missing=short)
    torch.cuda.synchronize()
    assert np.array_equal(r.cpu().numpy(), refs) and np.array_equal(t.cpu().numpy(), table)
    if stride:
        assert (wide[:, W:] == 77).all()
    return (new_refs.cpu().numpy(), wide[:, :W].cpu().numpy(), copies.cpu().numpy(),
            int(short) if missing else None)


def check_fork(refs, table, lens, src, page, **kw):
    got = run_fork(refs, table, lens, src, page, **kw)
    want = ref.fork(refs, table, lens, src, page)
    for x, y, what in zip(got, want, ("refs", "table", "copies", "missing")):
        if x is not None:
            assert np.array_equal(x, y), what
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("seed,N,M,width,page,pages", [
    (0, 1, 1, 1, 1, 1), (1, 1, 8, 3, 16, 40), (2, 8, 8, 5, 16, 100), (3, 7, 20, 9, 5, 60), (4, 30, 3, 4, 64, 200),
    (5, 40, 40, 300, 16, 13000), (6, 1500, 2100, 2, 3, 9000), (7, 3, 1300, 2, 8, 1500), (8, 5, 5, 7, 16, 36),
    (9, 9000, 9000, 1, 4, 20000),
])
def test_forks(seed, N, M, width, page, pages):
    say("fork %d" % seed)
    rng = np.random.default_rng([seed, 61])
    table, refs = shared_table(rng, N, width, pages - pages // 3 if pages > 3 else pages)
    refs = np.concatenate([refs, np.zeros(pages - len(refs), int)])
    table[table >= pages] = pages + 3
    refs = holders(table, pages)
    lens = rng.integers(-2, width * page + 4, N)
    src = rng.integers(-1, N + 1, M)
    check_fork(refs, table, lens, src, page, stride=seed % 3)


@pytest.mark.gpu
def test_beams_that_go_on_alone_touch_nothing():
    table, pages = np.arange(12).reshape(3, 4), 20
    refs = holders(table, pages)
    got = check_fork(refs, table, [50, 64, 33], [0, 1, 2], 16)
    assert np.array_equal(got[0], holders(got[1], pages))
    assert (got[2] == [-1, -1, 0]).all() and got[3] == 0


@pytest.mark.gpu
def test_a_part_filled_page_that_others_name_is_copied_by_all():
    """The page of a prompt's last tokens under two rows: neither may write to it."""
    table = np.array([[0, 1], [0, 1]])
    got = check_fork(holders(table, 6), table, [20, 20], [0, 1, 0], 16)
    assert got[2].tolist() == [[1, 2, 4], [1, 3, 4], [1, 4, 4]]
    assert got[0].tolist() == [3, 0, 1, 1, 1, 0]


@pytest.mark.gpu
def test_pages_run_out():
    table = np.array([[3]])
    refs = np.array([1, 0, 7, 1, 1])
    got = check_fork(refs, table, [5], [0, 0, 0, 0], 16)
    assert got[3] == 2 and got[1][:, 0].tolist() == [3, 1, -1, -1]
    check_fork(refs, table, [5], [0, 0, 0, 0], 16, missing=False)


@pytest.mark.gpu
def test_no_rows_on_either_side():
    refs, table = holders([[0, 1]], 4), np.array([[0, 1]])
    got = check_fork(refs, table, [20], [], 16)        # all pages come back
    assert (got[0] == 0).all()
    empty = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    new = torch.full((2, 2), 9, dtype=torch.int32, device="cuda")
    new_refs, copies = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty((2, 3), dtype=torch.int32, device="cuda")
    native.xpress_kv_fork(i32(refs).cuda(), empty, empty[:, 0], i32([0, 1]).cuda(), new_refs, new, copies, 16)
    torch.cuda.synchronize()
    assert (new == -1).all() and np.array_equal(new_refs.cpu().numpy(), refs)
    assert copies.tolist() == [[-1, -1, 0]] * 2


@pytest.mark.gpu
def test_a_captured_fork_is_replayed():
    rng = np.random.default_rng(5)
    table, refs = shared_table(rng, 20, 6, 150)
    lens, src = rng.integers(0, 96, 20), rng.integers(0, 20, 20)
    want = ref.fork(refs, table, lens, src, 16)
    r, t, l, s = (i32(x).cuda() for x in (refs, table, lens, src))
    out = [torch.zeros(150, dtype=torch.int32, device="cuda"), torch.zeros((20, 6), dtype=torch.int32, device="cuda"),
           torch.zeros((20, 3), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        native.xpress_kv_fork(r, t, l, s, out[0], out[1], out[2], 16, missing=out[3])
    for _ in range(3):
        for x in out:
            x.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert np.array_equal(x.cpu().numpy().reshape(np.shape(y)), y)


def pool(rng, pages, Hk, page, D, dtype, layout, pad=0):
    """Two caches of random bits (NaN among them), a view of rows with `pad` more elements."""
    e = torch.empty(0, dtype=TYPES[dtype]).element_size()
    both = []
    for _ in range(2):
        shape = (pages, page, Hk, D + pad) if layout == "token" else (pages, Hk, page, D + pad)
        x = torch.from_numpy(rng.integers(0, 256, shape[:-1] + (shape[-1] * e,), dtype=np.uint8).astype(np.uint8))
        x = x.view(TYPES[dtype])[..., :D]
        both.append(x.transpose(1, 2) if layout == "token" else x)
    return both


def bits(x):
    return x.contiguous().view(torch.uint8)


def on_gpu(x):
    """The same strides, whole storage."""
    flat = torch.as_strided(x.view(torch.uint8 if x.element_size() == 1 else torch.int16),
                            (x.untyped_storage().nbytes() // x.element_size(),), (1,), 0).cuda()
    return torch.as_strided(flat.view(x.dtype), x.shape, x.stride(), x.storage_offset()), flat


LAYOUTS = [("bf16", 128, "head", 0), ("bf16", 64, "token", 0), ("fp16", 80, "head", 8), ("e4m3", 64, "token", 0),
           ("bf16", 5, "head", 0), ("fp16", 6, "token", 0), ("e4m3", 7, "head", 0), ("bf16", 12, "head", 4),
           ("e4m3", 8, "head", 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,layout,pad", LAYOUTS)
@pytest.mark.parametrize("page", [16, 24, 1])
def test_copies(dtype, D, layout, pad, page):
    rng = np.random.default_rng([D, page])
    k, v = pool(rng, 40, 3, page, D, dtype, layout, pad)
    to = rng.permutation(np.arange(20, 40))
    copies = np.stack([rng.integers(0, 20, 20), to, rng.integers(-1, page + 3, 20)], 1)
    copies[3, 0], copies[5, 1], copies[7, 0], copies[8, 1], copies[9, :2] = -1, -1, 40, 2 ** 31 - 1, 33
    copies[9, 1] = copies[9, 0] = to[9]
    (kd, kf), (vd, vf) = on_gpu(k), on_gpu(v)
    before = kf.clone()
    native.xpress_kv_copy(kd, vd, i32(copies).cuda())
    torch.cuda.synchronize()
    assert torch.equal(bits(kd.cpu()), bits(ref.copy(k, copies)))
    assert torch.equal(bits(vd.cpu()), bits(ref.copy(v, copies)))
    if pad:     # nothing beside the rows
        gaps = torch.ones(kf.shape, dtype=torch.bool, device="cuda")
        torch.as_strided(gaps, kd.shape, kd.stride(), 0)[:] = False
        assert torch.equal(before[gaps], kf[gaps])


@pytest.mark.gpu
@pytest.mark.parametrize("seed,N,width,page,pages,most", [
    (0, 1, 1, 1, 1, 1), (1, 3, 10, 16, 30, 160), (2, 1, 3000, 4, 7000, 12000), (3, 1500, 7, 16, 6000, 112),
    (4, 256, 300, 16, 40000, 900), (5, 2500, 3, 5, 4500, 15), (6, 4, 20, 8, 10, 200),
])
def test_growth(seed, N, width, page, pages, most):
    say("grow %d" % seed)
    rng = np.random.default_rng([seed, 62])
    table, _ = shared_table(rng, N, width, pages // 2, holes=0.7)
    refs = holders(table, pages)
    refs[rng.integers(0, pages, pages // 10)] += 1          # pages of other tables
    have = rng.integers(-3, most + 1, N)
    want = have + rng.integers(-2, 3 * page + 2, N)
    r, t, short = i32(refs).cuda(), i32(table).cuda(), torch.full((1,), 9, dtype=torch.int32, device="cuda")
    native.xpress_kv_grow(r, t, i32(have).cuda(), i32(want).cuda(), page, missing=short)
    torch.cuda.synchronize()
    for x, y in zip((r.cpu().numpy(), t.cpu().numpy(), int(short)), ref.grow(refs, table, have, want, page)):
        assert np.array_equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (20, 0), (33, 5), (500, 16), (7, 1000)])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_pages_given_back(window, sinks, page):
    rng = np.random.default_rng([window, sinks, page])
    N, width, pages = 40, 30, 2000
    table, refs = shared_table(rng, N, width, pages)
    lens = rng.integers(-1, width * page + 50, N)
    lens[:3] = 0
    r, t = i32(refs).cuda(), i32(table).cuda()
    for _ in range(2):       # a second time there is nothing left to give
        native.xpress_kv_free(r, t, i32(lens).cuda(), page, window=window, sinks=sinks)
        torch.cuda.synchronize()
        want = ref.free(refs, table, lens, page, window, sinks)
        assert np.array_equal(r.cpu().numpy(), want[0]) and np.array_equal(t.cpu().numpy(), want[1])
    assert np.array_equal(want[0], holders(want[1], pages))


@pytest.mark.gpu
def test_what_is_freed_is_what_no_later_query_sees():
    """Freed pages against the attention's own rule, for the next token."""
    for length in (0, 1, 15, 16, 17, 100, 161):
        for window, sinks in ((1, 0), (16, 3), (40, 17), (1000, 0)):
            see = ref.visible(length + 1, 1, window, sinks)[0]
            table = np.arange(12)[None]
            _, kept = ref.free(holders(table, 12), table, [length], 16, window, sinks)
            for s in range(12):
                seen = see[s * 16:(s + 1) * 16][:max(0, length - s * 16)].any()
                assert not (seen and kept[0, s] < 0), (length, window, sinks, s)
                # what is kept is seen, or a window's page whose seen token is to come
                assert seen or kept[0, s] < 0 or s == (length - 1) // 16


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,layout,pad", LAYOUTS)
@pytest.mark.parametrize("page,Q", [(16, 16), (24, 40), (1, 9), (8, 600)])
def test_paths_move_together(dtype, D, layout, pad, page, Q):
    rng = np.random.default_rng([D, page, Q])
    N, Hk = 9, 3
    start = rng.integers(0, 40, N)
    start[4] = -1
    need = -(-(40 + Q) // page)
    pages = N * need + 2
    k, v = pool(rng, pages, Hk, page, D, dtype, layout, pad)
    table = rng.permutation(pages)[:N * need].reshape(N, need)
    table[2, need // 2], table[3, 0] = -1, pages          # moves from and to there are left out
    longest = min(Q, 300)
    path, count = np.full((N, longest), -1), rng.integers(0, longest + 1, N)
    for n in range(N):
        path[n] = np.sort(rng.permutation(Q)[:longest])
    count[5], count[6] = longest + 9, -3
    path[7, min(3, longest - 1):] = path[7, 2]                # ends before its count
    path[8] = np.arange(longest) * 1000                       # leaves the table
    (kd, kf), (vd, _) = on_gpu(k), on_gpu(v)
    before = kf.clone()
    native.xpress_kv_compact(kd, vd, i32(table).cuda(), i32(start).cuda(), i32(path).cuda(), i32(count).cuda())
    torch.cuda.synchronize()
    assert torch.equal(bits(kd.cpu()), bits(ref.compact(k, table, start, path, count)))
    assert torch.equal(bits(vd.cpu()), bits(ref.compact(v, table, start, path, count)))
    if pad:
        gaps = torch.ones(kf.shape, dtype=torch.bool, device="cuda")
        torch.as_strided(gaps, kd.shape, kd.stride(), 0)[:] = False
        assert torch.equal(before[gaps], kf[gaps])


@pytest.mark.gpu
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_append_at_places(cache):
    """Each key is the one that xpress_kv_append makes at its position, put elsewhere."""
    rng = np.random.default_rng(8)
    T, Hq, Hk, D, page, width = 60, 4, 2, 64, 16, 8
    pages = 2 * width
    q, k, v = (torch.from_numpy(rng.standard_normal((T, h, D)).astype(np.float32)).to(torch.bfloat16).cuda()
               for h in (Hq, Hk, Hk))
    angle = rng.uniform(0, 6, (100, D // 2))
    cs = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
    seq = np.repeat([0, 1], T // 2)
    places = np.concatenate([rng.permutation(width * page)[:T // 2] for _ in range(2)])
    positions = rng.integers(0, 100, T)
    places[3], places[4], positions[5], positions[6], places[7], seq[8] = -1, width * page, -1, 100, 2 ** 31 - 1, 2
    table = rng.permutation(pages).reshape(2, width)
    table[1, 3] = -1
    scale = torch.full((Hk,), 0.01, device="cuda") if cache == "e4m3" else None
    shape = (pages, Hk, page, D)
    got = [torch.zeros(shape, device="cuda").to(TYPES[cache]) for _ in range(2)]
    out = torch.full_like(q, 7)
    native.xpress_kv_append_at(q, k, v, out, *got, i32(table).cuda(), i32(places).cuda(), i32(positions).cuda(), cs,
                               seq_of=i32(seq).cuda(), k_scale=scale, v_scale=scale)
    # every token alone in a sequence of its own, at its position
    flat = [torch.zeros((T * 7, Hk, page, D), device="cuda").to(TYPES[cache]) for _ in range(2)]
    each = i32(np.arange(T * 7).reshape(T, 7)).cuda()
    ok = (positions >= 0) & (positions < 100) & (seq < 2)
    want_out = torch.full_like(q, 7)
    native.xpress_kv_append(q, k, v, want_out, *flat, each, i32(np.where(ok, positions, -1)).cuda(), cs,
                            k_scale=scale, v_scale=scale)
    torch.cuda.synchronize()
    assert torch.equal(out, want_out)
    for a, b in zip(got, flat):
        want = torch.zeros(shape, device="cuda").to(TYPES[cache])
        for t in range(T):
            if ok[t] and 0 <= places[t] < width * page and table[seq[t], places[t] // page] >= 0:
                x = b.view(torch.uint8)[t * 7 + positions[t] // page, :, positions[t] % page]
                want.view(torch.uint8)[table[seq[t], places[t] // page], :, places[t] % page] = x
        assert torch.equal(a.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.gpu
def test_pages_past_32_bits():
    """Pages more than 2^32 bytes apart: copies and moves there."""
    say("far pages")
    step = (1 << 32) // 2 + 64            # elements
    flat = torch.zeros(2 * step + 4096, dtype=torch.bfloat16, device="cuda")
    k = torch.as_strided(flat, (3, 1, 16, 64), (step, 1024, 64, 1))
    v = torch.as_strided(torch.zeros(2 * step + 4096, dtype=torch.bfloat16, device="cuda"), (3, 1, 16, 64),
                         (step, 1024, 64, 1))
    k[1] = torch.arange(1024, device="cuda").view(1, 16, 64).to(torch.bfloat16)
    v[1] = -k[1]
    native.xpress_kv_copy(k, v, i32([[1, 2, 16]]).cuda())
    native.xpress_kv_compact(k, v, i32([[2, 0]]).cuda(), i32([14]).cuda(), i32([[1, 3]]).cuda(), i32([2]).cuda())
    torch.cuda.synchronize()
    assert torch.equal(k[2, :, :14], k[1, :, :14]) and torch.equal(v[2, :, :14], v[1, :, :14])
    assert torch.equal(k[2, :, 14], k[1, :, 15]) and (k[2, :, 15] == 0).all()
