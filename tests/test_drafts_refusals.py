"""What the operators for drafts that branch, for pages and for beams refuse, on the CPU:
every status comes back before any HIP call, and the binding's own checks run before the
library is asked."""
import struct

import pytest
import torch

from conftest import gpu_available
from test_serving_refusals import (APPEND, ATTENTION, BAD_CACHE, CACHE, GOOD_APPEND, GOOD_ATTENTION, GOOD_CACHE, MiB)
from vocab_wide_add_amd import native

# made-up addresses: only where no kernel could be put on a device with them
no_gpu_only = pytest.mark.skipif(gpu_available(), reason="fake-pointer checks run without a GPU")
BAD = native.XPRESS_EINVAL


def cache(**change):
    d = dict(GOOD_CACHE, **change)
    return struct.pack(native._KV_CACHE, *[d[x] for x in CACHE])


def sink(sinks=4, **change):
    d = dict(GOOD_ATTENTION, **change)
    return native.load().xpress_sink_attention(native._ATTENTION_ARGS.pack(*[d[x] for x in ATTENTION]), sinks, None)


def tree(at=64 * MiB, tn=3, ti=1, sinks=0, **change):
    d = dict(GOOD_ATTENTION, **change)
    return native.load().xpress_tree_attention(native._ATTENTION_ARGS.pack(*[d[x] for x in ATTENTION]), at, tn, ti,
                                               sinks, None)


BAD_ATTENTION = [
    dict(Q=-1), dict(Hq=0), dict(Hq=3), dict(dtype=2), dict(max_len=0), dict(max_len=65), dict(window=-1),
    dict(scale=float("nan")), dict(scale=1e300), dict(cache_dtype=2, dim=56), dict(k=16 * MiB + 8), dict(q=0),
    dict(out=0), dict(lens=0), dict(q=2 * MiB + 1), dict(lse=4 * MiB + 2), dict(q_n=-1), dict(o_n=0),
    dict(out=2 * MiB), dict(out=16 * MiB), dict(lse=5 * MiB), dict(lse=3 * MiB), dict(Q=2 ** 30), dict(sinks=-1),
    dict(sinks=2 ** 31),
]


@no_gpu_only
@pytest.mark.parametrize("change", BAD_CACHE + BAD_ATTENTION)
def test_sink_attention_refuses(change):
    assert sink(**change) == BAD


@no_gpu_only
@pytest.mark.parametrize("change", BAD_CACHE + BAD_ATTENTION + [
    dict(at=0), dict(at=64 * MiB + 2), dict(tn=-1), dict(ti=-1), dict(tn=2 ** 61), dict(at=3 * MiB), dict(at=4 * MiB),
    dict(at=3 * MiB - 20),                                   # reaches into out
])
def test_tree_attention_refuses(change):
    assert tree(**change) == BAD


@no_gpu_only
def test_attention_of_nothing_is_ok():
    lib = native.load()
    assert sink(seqs=0, q=0, out=0) == 0 and sink(Q=0, q=0, out=0) == 0
    assert tree(seqs=0, q=0, out=0, at=0) == 0 and tree(Q=0, at=0) == 0
    assert lib.xpress_sink_attention(None, 0, None) == BAD
    assert lib.xpress_tree_attention(None, 64 * MiB, 3, 1, 0, None) == BAD
    assert lib.xpress_tree_attention(None, None, 3, 1, 0, None) == BAD


def test_sparse_reserve_checks_its_sizes():
    lib = native.load()
    good = [2, 3, 4, 2, 64, 100, 0, 0]
    for i, bad in ((0, -1), (1, -1), (2, 3), (3, 0), (4, 60), (5, 0), (6, -1), (7, -1), (7, 2 ** 31)):
        args = list(good)
        args[i] = bad
        assert lib.xpress_sparse_attention_reserve(*args, 1, None) == BAD
    assert lib.xpress_sparse_attention_reserve(0, *good[1:], 1, None) == 0


def append_at(places=40 * MiB, **change):
    d = dict(GOOD_APPEND, **change)
    return native.load().xpress_kv_append_at(native._APPEND_ARGS.pack(*[d[x] for x in APPEND]), places, None)


@no_gpu_only
@pytest.mark.parametrize("change", [dict(places=40 * MiB + 2), dict(places=16 * MiB), dict(places=32 * MiB + 64),
                                    dict(T=-1), dict(positions=0), dict(rot_dim=3), dict(q_out=0)])
def test_append_at_refuses(change):
    assert append_at(**change) == BAD


# refs, pages, table, stride, lens, N, src, M, width, page_size, new_refs, new_table, stride, copies, missing
FORK = [MiB, 100, 2 * MiB, 8, 3 * MiB, 4, 4 * MiB, 6, 8, 16, 5 * MiB, 6 * MiB, 8, 7 * MiB, 8 * MiB]
GROW = [MiB, 100, 2 * MiB, 8, 4, 8, 16, 3 * MiB, 4 * MiB, 5 * MiB]
FREE = [MiB, 100, 2 * MiB, 8, 4, 8, 16, 3 * MiB, 0, 0]
SELECT = [MiB, 4 * MiB, 2 * MiB, 3 * MiB, 5 * MiB, 6 * MiB, 2, 3, 100, 4, 100, 100]


def changed(base, at):
    args = list(base)
    for i, v in at.items():
        args[i] = v
    return args


@no_gpu_only
@pytest.mark.parametrize("at", [
    {0: 0}, {0: MiB + 2}, {1: 0}, {1: 2 ** 31}, {2: 0}, {2: 2 * MiB + 1}, {3: 7}, {3: -1}, {4: 0}, {5: -1},
    {5: 2 ** 24}, {5: 65537}, {6: 0}, {7: -1}, {7: 2 ** 24}, {7: 65537}, {8: 0}, {8: 2 ** 28, 3: 2 ** 28, 12: 2 ** 28}, {9: 0}, {9: -16},
    {10: 0}, {11: 0}, {12: 7}, {13: 0}, {13: 7 * MiB + 2}, {14: 8 * MiB + 1},
    {10: MiB}, {10: MiB + 396}, {11: 2 * MiB}, {11: 2 * MiB + 100}, {13: 6 * MiB + 100}, {14: 6 * MiB}, {14: MiB},
    {13: 4 * MiB}, {11: 3 * MiB}, {10: 4 * MiB},
])
def test_fork_refuses(at):
    assert native.load().xpress_kv_fork(*changed(FORK, at), None) == BAD


@no_gpu_only
@pytest.mark.parametrize("at", [
    {0: 0}, {0: MiB + 1}, {1: 0}, {1: 2 ** 31}, {2: 0}, {3: 7}, {4: -1}, {4: 2 ** 31}, {5: 0},
    {5: 2 ** 21, 3: 2 ** 21, 6: 1}, {6: 0}, {7: 0}, {8: 0}, {8: 4 * MiB + 2}, {9: 5 * MiB + 1}, {2: MiB + 40},
    {7: MiB + 40}, {8: 2 * MiB}, {9: 2 * MiB + 4}, {9: MiB},
])
def test_grow_refuses(at):
    assert native.load().xpress_kv_grow(*changed(GROW, at), None) == BAD


@no_gpu_only
@pytest.mark.parametrize("at", [
    {0: 0}, {1: 0}, {2: 0}, {3: 7}, {4: -1}, {5: 0}, {6: 0}, {7: 0}, {7: 3 * MiB + 2}, {8: -1}, {9: -1},
    {8: 2 ** 31}, {9: 2 ** 31}, {2: MiB}, {7: MiB + 4}, {7: 2 * MiB},
])
def test_free_refuses(at):
    assert native.load().xpress_kv_free(*changed(FREE, at), None) == BAD


POOL_ONLY = [x for x in BAD_CACHE if not set(x) & {"seqs", "table_width", "stride_table", "page_table"}
             and x not in (dict(cache_dtype=1),)]


@no_gpu_only
@pytest.mark.parametrize("change", POOL_ONLY)
def test_copy_and_compact_refuse_the_cache(change):
    lib = native.load()
    assert lib.xpress_kv_copy(cache(**change), 40 * MiB, 3, None) == BAD
    assert lib.xpress_kv_compact(cache(**change), 40 * MiB, 41 * MiB, 4, 42 * MiB, 4, None) == BAD


@no_gpu_only
def test_copy_and_compact_refuse():
    lib = native.load()
    for copies, count in ((0, 3), (40 * MiB + 2, 3), (16 * MiB, 3), (40 * MiB, -1), (40 * MiB, 2 ** 31)):
        assert lib.xpress_kv_copy(cache(), copies, count, None) == BAD
    assert lib.xpress_kv_copy(None, 40 * MiB, 3, None) == BAD
    assert lib.xpress_kv_copy(cache(page_table=0, seqs=0, table_width=0), 0, 0, None) == 0
    # a page of 2^31 pieces
    assert lib.xpress_kv_copy(cache(page_size=2 ** 25, stride_head=2 ** 31, stride_page=2 ** 33, dim=8, heads=65536,
                                    stride_token=8, k=2 ** 50, v=2 ** 55), 40 * MiB, 3, None) == BAD
    good = [40 * MiB, 41 * MiB, 4, 42 * MiB, 4]
    for at in ({0: 0}, {1: 0}, {3: 0}, {0: 40 * MiB + 2}, {1: 41 * MiB + 1}, {2: 3}, {2: -4}, {4: -1}, {4: 2 ** 31},
               {0: 16 * MiB}, {1: 32 * MiB}, {3: 16 * MiB + 64}, {2: 2 ** 60}):
        assert lib.xpress_kv_compact(cache(), *changed(good, at), None) == BAD
    assert lib.xpress_kv_compact(cache(page_table=16 * MiB), *good, None) == BAD
    for change in (dict(page_table=0), dict(seqs=-1), dict(table_width=0), dict(stride_table=3)):
        assert lib.xpress_kv_compact(cache(**change), *good, None) == BAD
    assert lib.xpress_kv_compact(None, *good, None) == BAD
    assert lib.xpress_kv_compact(cache(seqs=0), 0, 0, 0, 0, 4, None) == 0
    assert lib.xpress_kv_compact(cache(), 0, 0, 0, 0, 0, None) == 0


@no_gpu_only
@pytest.mark.parametrize("at", [
    {6: -1}, {7: 0}, {7: 4097}, {8: 0}, {8: 2 ** 31}, {9: 0}, {9: 129}, {10: 99}, {11: 99}, {0: 0}, {2: 0}, {3: 0},
    {4: 0}, {5: 0}, {0: MiB + 1}, {1: 4 * MiB + 1}, {2: 2 * MiB + 2}, {3: 3 * MiB + 2}, {4: 5 * MiB + 1},
    {5: 6 * MiB + 4}, {3: MiB}, {4: MiB + 4}, {5: 4 * MiB}, {3: 2 * MiB}, {4: 3 * MiB}, {5: 5 * MiB}, {10: 2 ** 61},
    {6: 2 ** 31, 7: 1}, {6: 2 ** 20, 7: 4096},
])
def test_beam_select_refuses(at):
    assert native.load().xpress_beam_select(*changed(SELECT, at), None) == BAD


@no_gpu_only
def test_beam_select_of_nothing_is_ok():
    assert native.load().xpress_beam_select(*changed(SELECT, {6: 0, 0: 0}), None) == 0
    lib = native.load()
    assert lib.xpress_beam_select_reserve(0, 4, 1000, 4, None) == 0
    for args in ((-1, 4, 1000, 4), (1, 0, 1000, 4), (1, 4, 0, 4), (1, 4, 1000, 0), (1, 4, 1000, 129)):
        assert lib.xpress_beam_select_reserve(*args, None) == BAD


@no_gpu_only
def test_beam_reorder_refuses():
    lib = native.load()

    def go(states, src=MiB, N=4, M=6, count=None):
        return lib.xpress_beam_reorder(b"".join(native._STATE.pack(*s) for s in states),
                                       len(states) if count is None else count, src, N, M, None)
    good = (2 * MiB, 3 * MiB, 64, 64, 64)
    for i, bad in ((0, 0), (1, 0), (2, -1), (3, -1), (3, 63), (4, -1), (4, 2 ** 61), (1, 2 * MiB), (1, 2 * MiB + 100),
                   (1, MiB), (2, 2 ** 60), (3, 2 ** 60)):
        s = list(good)
        s[i] = bad
        assert go([tuple(s)]) == BAD
    assert go([good, good]) == BAD                                  # written twice
    assert go([good, (3 * MiB, 5 * MiB, 64, 64, 64)]) == BAD        # read where the other writes
    assert go([good], src=0) == BAD and go([good], src=MiB + 2) == BAD
    assert go([good], N=-1) == BAD and go([good], M=-1) == BAD and go([good], count=-1) == BAD
    assert go([good], count=4097) == BAD
    assert go([], src=0) == 0 and go([good], M=0, src=0) == 0


@no_gpu_only
@pytest.mark.parametrize("count", [2, 33, 300, 4096])
def test_beam_reorder_refuses_overlaps_among_many_states(count):
    lib = native.load()

    def go(states):
        return lib.xpress_beam_reorder(b"".join(native._STATE.pack(*s) for s in states), count, MiB, 4, 6, None)
    good = [((2 * i + 2) * MiB, (2 * i + 3) * MiB, 64, 64, 64) for i in range(count)]
    for at, other in ((0, count - 1), (count - 1, 0), (count // 2, 0)):
        if at == other:
            continue
        for to in (good[other][1], good[other][1] + 383, good[other][1] - 383,     # written twice
                   good[other][0], good[other][0] + 255, good[other][0] - 383):    # written where another reads
            s = list(good)
            s[at] = (s[at][0], to, 64, 64, 64)
            assert go(s) == BAD
    # a long span that ends past the ones which begin after it
    s = list(good)
    s[0] = (s[0][0], s[0][1], 64, MiB, 64)
    assert go(s) == BAD


def test_the_binding_refuses_tensors_on_the_cpu():
    t = torch.zeros(4, 8, dtype=torch.int32)
    one = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        native.xpress_kv_fork(one, t, one, one, one, t, torch.zeros(4, 3, dtype=torch.int32), 16)
    with pytest.raises(ValueError, match="GPU"):
        native.xpress_kv_grow(one, t, one, one, 16)
    with pytest.raises(ValueError, match="GPU"):
        native.xpress_kv_free(one, t, one, 16)
    with pytest.raises(ValueError, match="GPU"):
        native.xpress_beam_reorder([(t, t)], one)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        native.xpress_kv_copy(k, k.clone(), torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        native.xpress_kv_compact(k, k.clone(), t, one, t, one)
    with pytest.raises(ValueError, match="GPU"):
        native.xpress_kv_append_at(None, torch.zeros(4, 2, 64, dtype=torch.bfloat16),
                                   torch.zeros(4, 2, 64, dtype=torch.bfloat16), None, k, k.clone(), t, one, one, None)


@pytest.mark.gpu
def test_the_binding_refuses_other_shapes_and_types():
    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32, device="cuda")
    refs, table, lens = i32(20), i32(4, 8), i32(4)

    def fork(**c):
        d = dict(refs=refs, table=table, lens=lens, src=i32(6), new_refs=i32(20), new_table=i32(6, 8), copies=i32(6, 3))
        d.update(c)
        native.xpress_kv_fork(*d.values(), 16)
    fork()
    for c in (dict(refs=refs.long()), dict(refs=i32(20, 1)), dict(table=i32(4)), dict(table=table.float()),
              dict(lens=i32(5)), dict(src=i32(5)), dict(new_refs=i32(19)), dict(new_table=i32(6, 7)),
              dict(copies=i32(6, 2)), dict(copies=i32(7, 3)), dict(lens=lens.cpu()), dict(table=i32(8, 4).t())):
        with pytest.raises(ValueError):
            fork(**c)
    for c in (dict(new_refs=refs), dict(src=None)):
        with pytest.raises((native.XpressError, AttributeError)):
            fork(**c)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    for bad in (i32(2, 2), i32(3), torch.zeros(2, 3, device="cuda")):
        with pytest.raises(ValueError):
            native.xpress_kv_copy(k, v, bad)
    with pytest.raises(ValueError):
        native.xpress_kv_copy(k, v[:3], i32(2, 3))
    for start, path, count in ((i32(3), i32(4, 5), lens), (lens, i32(3, 5), lens), (lens, i32(4, 5), i32(5)),
                               (lens, i32(4, 5).float(), lens), (lens, i32(5, 4).t(), lens)):
        with pytest.raises(ValueError):
            native.xpress_kv_compact(k, v, table, start, path, count)
    x = torch.zeros(6, 100, dtype=torch.bfloat16, device="cuda")
    out = [torch.zeros(2, 4, device="cuda"), i32(2, 4), torch.zeros(2, 4, dtype=torch.int64, device="cuda")]
    s = torch.zeros(6, device="cuda")
    native.xpress_beam_select(x, None, s, *out, 2, 3, 100, 4, 100)
    for args in ((x.float(), None, s, *out), (x, None, s[:5], *out), (x, None, s.double(), *out),
                 (x, None, s, out[0][:1], *out[1:]), (x, None, s, out[0], out[1].long(), out[2]),
                 (x, None, s, *out[:2], out[2].int()), (x[:5].clone(), None, s, *out), (x, x.cpu(), s, *out)):
        with pytest.raises(ValueError):
            native.xpress_beam_select(*args, 2, 3, 100, 4, 100, 100)
    src = i32(3)
    for pair in ((x, x[:2].clone()), (x, x[:3].float()), (x, x[:3, :50].clone()), (x, torch.zeros(3, 100, dtype=torch.bfloat16)),
                 (x.t(), torch.zeros(3, 6, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            native.xpress_beam_reorder([pair], src)
    with pytest.raises(ValueError):
        native.xpress_beam_reorder([(x, x[:3].clone()), (x[:5], x[:3].clone())], src)
