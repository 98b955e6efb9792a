"""xpress_kv_append against the definition in 64 bits.

Tolerances.  A stored value is rounded once (half a step of its type, relative);
before that the rotation rounds two products and their sum in fp32, and the
e4m3 form a quotient: at most 2^-24 each, of |a c| + |b s|.  Copied values
(v, dimensions past rot_dim) in a 16-bit cache are exact."""
import numpy as np
import pytest
import torch

import serving_ref as ref
from gpu_util import say
from vocab_wide_add_amd import native


def build(rng, lens, new, Hq, Hk, D, rot, page, dtype, cache, layout="head", pad=0, max_pos=None):
    """Packed rows [T, Hq + 2 Hk, D + pad] with `new[n]` last tokens of each sequence."""
    kc, vc, table = ref.paged_pool(rng, lens, Hk, D, page, cache, layout)
    seq = np.repeat(np.arange(len(lens)), new).astype(np.int32)
    pos = np.concatenate([np.arange(x - y, x) for x, y in zip(lens, new)]).astype(np.int32)
    T = len(pos)
    rows = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hk, D + pad)).astype(np.float32))
    rows = rows.to(ref.TYPES[dtype])
    cs = None
    if rot:
        n = max_pos or int(max(lens))
        angle = np.arange(n)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
        cs = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32))
    scales = [None, None]
    if cache == "e4m3":
        scales = [torch.from_numpy(rng.uniform(0.02, 0.1, Hk).astype(np.float32)) for _ in range(2)]
    return rows, kc, vc, table, torch.from_numpy(pos), torch.from_numpy(seq), cs, scales


def check(rows, kc, vc, table, pos, seq, cs, scales, Hq, Hk, D, interleaved, give_seq=True,
          in_place=False, off=0):
    q, k, v = rows[:, :Hq, off:off + D], rows[:, Hq:Hq + Hk, off:off + D], rows[:, Hq + Hk:, off:off + D]
    want_q, want_k, want_v, written = ref.append64(q, k, v, kc, vc, table, pos, seq, cs, *scales,
                                                   interleaved)
    dev = rows.cuda()
    qd, kd, vd = dev[:, :Hq, off:off + D], dev[:, Hq:Hq + Hk, off:off + D], dev[:, Hq + Hk:, off:off + D]
    q_out = qd if in_place else torch.full((len(pos), Hq, D), 7.0, dtype=rows.dtype, device="cuda")
    kcd, vcd = (torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)
                for x in (kc, vc))
    native.xpress_kv_append(qd, kd, vd, q_out, kcd, vcd, table.cuda(), pos.cuda(),
                            cs.cuda() if cs is not None else None,
                            seq_of=seq.cuda() if give_seq else None,
                            k_scale=scales[0].cuda() if scales[0] is not None else None,
                            v_scale=scales[1].cuda() if scales[1] is not None else None,
                            interleaved=interleaved)
    torch.cuda.synchronize()

    def near(got, want, size, dtype):
        tol = ref.half_step(dtype) * np.abs(want) + 4 * 2.0 ** -24 * size
        if dtype == torch.float8_e4m3fn:
            tol = np.maximum(tol, 2.0 ** -10 + 4 * 2.0 ** -24 * size)   # half of the smallest step
            want = np.clip(want, -ref.E4M3_MAX, ref.E4M3_MAX)
        elif dtype == torch.float16:
            tol = np.maximum(tol, 2.0 ** -25)
        bad = ~(np.abs(got - want) <= tol * (1 + 2.0 ** -20))
        assert not bad.any(), (int(bad.sum()), np.abs(got - want).max())

    size = 2.0 * max(1.0, float(rows.double().abs().max()))
    near(q_out.double().cpu().numpy(), want_q, size, rows.dtype)
    for got, want, old, sc in ((kcd, want_k, kc, scales[0]), (vcd, want_v, vc, scales[1])):
        inv = 1.0 if sc is None else (1.0 / sc.double().numpy())[None, :, None]
        w = written[:, None, :, None] & np.ones(got.shape, bool)
        g = got.double().cpu().numpy()
        near(np.where(w, g, 0.0), np.where(w, want, 0.0),
             size * np.broadcast_to(np.asarray(inv)[..., None], got.shape) if sc is not None else size,
             got.dtype)
        # what no token went to keeps its bits
        bits = torch.uint8 if got.element_size() == 1 else torch.int16
        same = got.view(bits).cpu().numpy() == old.view(bits).numpy()
        assert same[~w].all()
        if sc is None and want is want_v:
            assert np.array_equal(g[w], want[w])
    return q_out, kcd, vcd


SHAPES = [
    # lens, new, Hq, Hk, D, rot, page, layout
    ([1], [1], 4, 1, 64, 64, 16, "head"),
    ([1000], [1], 32, 8, 128, 128, 16, "head"),
    ([5, 17, 33], [5, 1, 7], 8, 2, 128, 64, 16, "token"),
    ([40, 16, 31], [16, 16, 16], 6, 3, 80, 80, 24, "token"),
    ([9, 70], [9, 64], 5, 1, 96, 32, 7, "head"),
    ([12], [12], 2, 2, 8, 8, 1, "head"),
    ([30, 3], [11, 3], 3, 1, 20, 6, 5, "token"),
    ([8], [8], 1, 1, 256, 0, 8, "head"),
    ([300], [300], 7, 7, 40, 16, 128, "head"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"),
                                         ("fp16", "e4m3")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_against_64_bits(shape, dtype, cache, interleaved):
    lens, new, Hq, Hk, D, rot, page, layout = SHAPES[shape]
    say("append %d %s %s %s" % (shape, dtype, cache, interleaved))
    rng = np.random.default_rng([shape, 5])
    made = build(rng, lens, new, Hq, Hk, D, rot, page, dtype, cache, layout)
    check(*made, Hq, Hk, D, interleaved)


@pytest.mark.gpu
def test_uniform_tokens_need_no_sequence_ids():
    rng = np.random.default_rng(1)
    made = build(rng, [20, 40, 33], [4, 4, 4], 8, 2, 64, 64, 16, "bf16", "bf16")
    check(*made, 8, 2, 64, False, give_seq=False)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_queries_rotated_in_place(interleaved):
    rng = np.random.default_rng(2)
    made = build(rng, [20, 40], [4, 9], 8, 2, 128, 128, 16, "bf16", "bf16")
    check(*made, 8, 2, 128, interleaved, in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("off,pad", [(1, 3), (8, 8), (0, 5)])
def test_rows_of_any_alignment(off, pad):
    rng = np.random.default_rng(3)
    made = build(rng, [20, 40], [4, 9], 4, 2, 64, 32, 16, "bf16", "e4m3", pad=pad)
    a = check(*made, 4, 2, 64, False, off=off)
    # the aligned copy gives the same bits
    rows = made[0][:, :, off:off + 64].contiguous()
    b = check(rows, *made[1:], 4, 2, 64, False)
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.gpu
def test_padding_and_missing_pages():
    """Tokens out of any range leave the caches alone and give zero queries; a page
    outside the pool takes nothing, but its token's query is rotated."""
    rng = np.random.default_rng(4)
    rows, kc, vc, table, pos, seq, cs, sc = build(rng, [20, 40, 33], [6, 6, 6], 4, 2, 64, 64, 16,
                                                  "bf16", "bf16", max_pos=41)
    pos, seq, table = pos.clone(), seq.clone(), table.clone()
    pos[0], pos[1], pos[2] = -1, 41, 2 ** 31 - 1
    pos[3] = -2 ** 31
    seq[4], seq[5] = -1, 3
    pos[6] = table.shape[1] * 16 - 1                    # a -1 entry of the table (or past cos_sin)
    table[2, 1] = kc.shape[0]                           # one past the pool
    table[1, 2] = -7
    check(rows, kc, vc, table, pos, seq, cs, sc, 4, 2, 64, False)


@pytest.mark.gpu
def test_e4m3_saturates_and_keeps_nan():
    rng = np.random.default_rng(6)
    rows, kc, vc, table, pos, seq, cs, sc = build(rng, [4], [4], 1, 1, 16, 0, 16, "bf16", "e4m3")
    rows[0, 2, :4] = torch.tensor([float("nan"), float("inf"), float("-inf"), 3e38])
    vcd = vc.cuda()
    native.xpress_kv_append(None, rows[:, 1:2].cuda(), rows[:, 2:3].cuda(), None, kc.cuda(), vcd,
                            table.cuda(), pos.cuda(), None)
    got = vcd[int(table[0, 0]), 0, 0, :4].float().cpu()
    assert torch.isnan(got[0]) and got[1:].tolist() == [448.0, -448.0, 448.0]


@pytest.mark.gpu
def test_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(7)
    rows, kc, vc, table, pos, seq, cs, sc = build(rng, [50, 70], [1, 1], 8, 2, 128, 128, 16, "bf16",
                                                  "bf16")
    dev = rows.cuda()
    q, k, v = dev[:, :8], dev[:, 8:10], dev[:, 10:]
    t, p, c = table.cuda(), pos.cuda(), cs.cuda()
    want = [torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda"), kc.cuda(), vc.cuda()]
    native.xpress_kv_append(q, k, v, *want, t, p, c)
    got = [torch.zeros_like(want[0]), kc.cuda(), vc.cuda()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        native.xpress_kv_append(q, k, v, *got, t, p, c)
    for _ in range(3):
        for x, y in zip(got, (torch.zeros_like(want[0]), kc, vc)):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot", [(80, 40), (12, 8), (12, 12), (20, 8), (7, 2), (24, 0), (1, 0), (520, 512)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_sizes_of_every_access_width(D, rot, cache, interleaved):
    """Pieces of 8, 4 and 1 elements, with and without a half piece at a head's end."""
    say("append widths %d %d %s %s" % (D, rot, cache, interleaved))
    rng = np.random.default_rng([D, rot])
    made = build(rng, [20, 40], [4, 9], 5, 2, D, rot, 16, "bf16", cache)
    check(*made, 5, 2, D, interleaved)


@pytest.mark.gpu
@pytest.mark.parametrize("cache,layout", [("bf16", "token"), ("e4m3", "head")])
def test_prompts_with_more_work_than_threads(cache, layout):
    """Past the size at which a workgroup takes a whole token."""
    rng = np.random.default_rng([8, 1])
    made = build(rng, [700, 1, 901], [700, 1, 901], 32, 8, 128, 32, 16, "bf16", cache, layout)
    assert sum((700, 1, 901)) * 48 * 8 > 1 << 19
    check(*made, 32, 8, 128, True)


@pytest.mark.gpu
def test_places_past_32_bits():
    """A pool of more than 2^32 elements with the sequence on its last pages."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GiB of GPU memory")
    rng = np.random.default_rng(9)
    rows, kc, vc, table, pos, seq, cs, sc = build(rng, [60], [9], 4, 2, 128, 128, 16, "bf16", "bf16")
    pages = (2 ** 32) // (2 * 16 * 128) + 64
    shift = pages - kc.shape[0]
    dev = rows.cuda()
    q, k, v = dev[:, :4], dev[:, 4:6], dev[:, 6:]
    small = [torch.zeros(9, 4, 128, dtype=torch.bfloat16, device="cuda"), kc.cuda(), vc.cuda()]
    native.xpress_kv_append(q, k, v, *small, table.cuda(), pos.cuda(), cs.cuda())
    big = [torch.zeros(pages, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for b, x in zip(big, (kc, vc)):
        b[shift:] = x.cuda()
    out = torch.zeros_like(small[0])
    native.xpress_kv_append(q, k, v, out, *big, torch.where(table >= 0, table + shift, table).cuda(), pos.cuda(),
                            cs.cuda())
    torch.cuda.synchronize()
    assert torch.equal(out, small[0])
    for b, x in zip(big, small[1:]):
        assert torch.equal(b[shift:], x) and not b[:shift].any()


@pytest.mark.gpu
def test_two_tokens_at_one_place():
    """Not for use: each element comes from one of them.  Nothing else changes."""
    rng = np.random.default_rng(10)
    rows, kc, vc, table, pos, seq, cs, sc = build(rng, [40], [2], 4, 8, 128, 0, 16, "bf16", "bf16")
    pos = torch.tensor([37, 37], dtype=torch.int32)
    dev, kcd, vcd = rows.cuda(), kc.cuda(), vc.cuda()
    native.xpress_kv_append(None, dev[:, 4:12], dev[:, 12:], None, kcd, vcd, table.cuda(), pos.cuda(), None,
                            seq_of=seq.cuda())
    torch.cuda.synchronize()
    page = int(table[0, 37 // 16])
    for got, old, new in ((kcd.cpu(), kc, rows[:, 4:12]), (vcd.cpu(), vc, rows[:, 12:])):
        here = got[page, :, 37 % 16]
        assert ((here == new[0]) | (here == new[1])).all()
        got[page, :, 37 % 16] = old[page, :, 37 % 16]
        assert torch.equal(got, old)


@pytest.mark.gpu
def test_one_token_in_place_under_another_stride():
    """q_out on q for one token, and for one head: the strides that address nothing may differ."""
    rng = np.random.default_rng(11)
    for Hq, lens, new in ((4, [40], [1]), (1, [40], [5])):
        rows, kc, vc, table, pos, seq, cs, sc = build(rng, lens, new, Hq, 2, 64, 64, 16, "bf16", "bf16")
        dev = rows.cuda()
        q, k, v = dev[:, :Hq], dev[:, Hq:Hq + 2], dev[:, Hq + 2:]
        want = torch.empty(len(pos), Hq, 64, dtype=torch.bfloat16, device="cuda")
        native.xpress_kv_append(q, k, v, want, kc.cuda(), vc.cuda(), table.cuda(), pos.cuda(), cs.cuda())
        st = (q.stride(0) + 8, q.stride(1)) if len(pos) == 1 else (q.stride(0), q.stride(1) + 8)
        onto = q.as_strided(q.shape, (*st, 1))
        native.xpress_kv_append(q, k, v, onto, kc.cuda(), vc.cuda(), table.cuda(), pos.cuda(), cs.cuda())
        torch.cuda.synchronize()
        assert torch.equal(q, want)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [682, 683])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_either_side_of_a_workgroup_a_token(T, cache):
    """A thread a piece up to 2^18 pieces, a workgroup a token beyond: 48 heads of 8 pieces each."""
    assert (682 * 48 * 8 <= 1 << 18) and (683 * 48 * 8 > 1 << 18)
    rng = np.random.default_rng([12, T])
    made = build(rng, [T - 40, 40], [T - 40, 40], 32, 8, 128, 128, 16, "bf16", cache)
    check(*made, 32, 8, 128, False)
