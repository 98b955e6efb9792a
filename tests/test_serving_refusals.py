"""What the serving operators refuse, on the CPU: every status comes back before any
HIP call, and the binding's own checks run before the library is asked."""
import pytest
import torch

from conftest import gpu_available
from vocab_wide_add_amd import native

# made-up addresses: only where no kernel could be put on a device with them
no_gpu_only = pytest.mark.skipif(gpu_available(), reason="fake-pointer checks run without a GPU")

CACHE = ["k", "v", "k_scale", "v_scale", "page_table", "pages", "page_size", "heads", "dim",
         "stride_page", "stride_head", "stride_token", "cache_dtype", "seqs", "table_width",
         "stride_table"]
APPEND = CACHE + ["q", "key", "value", "q_out", "positions", "seq_of", "cos_sin", "T", "Hq", "dtype",
                  "rot_dim", "max_pos", "interleaved", "q_t", "q_h", "k_t", "k_h", "v_t", "v_h", "o_t",
                  "o_h"]
ATTENTION = CACHE + ["q", "out", "lse", "lens", "Q", "Hq", "dtype", "max_len", "window", "scale", "q_n",
                     "q_i", "q_h", "o_n", "o_i", "o_h"]

MiB = 1 << 20
GOOD_CACHE = dict(k=16 * MiB, v=32 * MiB, k_scale=0, v_scale=0, page_table=MiB, pages=8, page_size=16,
                  heads=2, dim=64, stride_page=2048, stride_head=1024, stride_token=64, cache_dtype=0,
                  seqs=2, table_width=4, stride_table=4)
GOOD_APPEND = dict(GOOD_CACHE, q=2 * MiB, key=3 * MiB, value=4 * MiB, q_out=5 * MiB, positions=6 * MiB,
                   seq_of=7 * MiB, cos_sin=8 * MiB, T=6, Hq=4, dtype=0, rot_dim=64, max_pos=100,
                   interleaved=0, q_t=256, q_h=64, k_t=128, k_h=64, v_t=128, v_h=64, o_t=256, o_h=64)
GOOD_ATTENTION = dict(GOOD_CACHE, q=2 * MiB, out=3 * MiB, lse=4 * MiB, lens=5 * MiB, Q=3, Hq=4, dtype=0,
                      max_len=64, window=0, scale=0.125, q_n=768, q_i=256, q_h=64, o_n=768, o_i=256,
                      o_h=64)


def append(**change):
    d = dict(GOOD_APPEND, **change)
    return native.load().xpress_kv_append(native._APPEND_ARGS.pack(*[d[x] for x in APPEND]), None)


def attend(**change):
    d = dict(GOOD_ATTENTION, **change)
    return native.load().xpress_paged_attention(native._ATTENTION_ARGS.pack(*[d[x] for x in ATTENTION]),
                                                None)


BAD_CACHE = [
    dict(pages=0), dict(page_size=0), dict(heads=0), dict(dim=0), dict(pages=2 ** 31),
    dict(cache_dtype=3), dict(cache_dtype=-1), dict(stride_page=0), dict(stride_head=-64),
    dict(stride_token=0), dict(seqs=-1), dict(table_width=0), dict(stride_table=3), dict(stride_table=-4),
    dict(table_width=2 ** 28, stride_table=2 ** 28),      # 2^32 tokens
    dict(stride_page=2047), dict(stride_head=1000),       # elements share addresses
    dict(stride_token=32), dict(stride_page=2 ** 62),
    dict(k=0), dict(v=0), dict(k=32 * MiB), dict(page_table=0), dict(page_table=MiB + 2),
    dict(k=16 * MiB + 1), dict(k_scale=9 * MiB), dict(v_scale=9 * MiB),    # scales with a 16-bit cache
    dict(cache_dtype=2, k_scale=9 * MiB + 1), dict(cache_dtype=1),         # another 16-bit type than q
]


@no_gpu_only
@pytest.mark.parametrize("change", BAD_CACHE + [
    dict(T=-1), dict(T=2 ** 31), dict(Hq=-1), dict(dtype=2), dict(dtype=5), dict(rot_dim=-2),
    dict(rot_dim=3), dict(rot_dim=66), dict(max_pos=0), dict(cos_sin=0), dict(cos_sin=8 * MiB + 1),
    dict(positions=0), dict(positions=6 * MiB + 2), dict(seq_of=7 * MiB + 1),
    dict(seq_of=0, T=5),                                  # not a whole number of tokens a sequence
    dict(seq_of=0, seqs=0),
    dict(q=0), dict(key=0), dict(value=0), dict(q_out=0), dict(q=2 * MiB + 1), dict(q_out=5 * MiB + 1),
    dict(q_t=-1), dict(k_h=-64), dict(v_t=-1), dict(o_t=0), dict(o_h=63), dict(o_t=255),
    dict(q_out=2 * MiB, o_t=512), dict(q_out=2 * MiB + 128),    # on q, but not as q itself
    dict(key=16 * MiB), dict(value=32 * MiB + 4096), dict(q=16 * MiB), dict(q_out=32 * MiB - 64),
    dict(positions=16 * MiB), dict(seq_of=32 * MiB), dict(page_table=16 * MiB),
    dict(q_t=2 ** 62),
])
def test_append_refuses(change):
    assert append(**change) == native.XPRESS_EINVAL


@no_gpu_only
@pytest.mark.parametrize("change", BAD_CACHE + [
    dict(Q=-1), dict(Hq=0), dict(Hq=3), dict(Hq=2 ** 20), dict(dtype=2), dict(max_len=0),
    dict(max_len=65), dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(scale=1e300), dict(dim=68, stride_token=68, stride_head=1088, stride_page=2176),
    dict(dim=264, stride_token=264, stride_head=4224, stride_page=8448),
    dict(cache_dtype=2, dim=56),                          # 8-bit rows of 56 bytes
    dict(k=16 * MiB + 8), dict(v=32 * MiB + 2), dict(stride_token=68, stride_head=1088, stride_page=2176),
    dict(stride_head=1028, stride_page=2056), dict(stride_page=2052),
    dict(q=0), dict(out=0), dict(lens=0), dict(q=2 * MiB + 1), dict(out=3 * MiB + 1), dict(lse=4 * MiB + 2),
    dict(lens=5 * MiB + 1), dict(q_n=-1), dict(q_i=-1), dict(q_h=-1), dict(o_n=0), dict(o_i=255),
    dict(o_h=32), dict(o_n=700), dict(out=2 * MiB), dict(out=5 * MiB - 64), dict(out=16 * MiB),
    dict(out=32 * MiB + 4096), dict(lse=2 * MiB), dict(lse=5 * MiB), dict(lse=3 * MiB), dict(lse=MiB),
    dict(out=MiB), dict(lse=32 * MiB), dict(q_n=2 ** 62), dict(Q=2 ** 30),
])
def test_attention_refuses(change):
    assert attend(**change) == native.XPRESS_EINVAL


@no_gpu_only
def test_nothing_to_do_is_ok():
    assert append(T=0, key=0, value=0, q=0, q_out=0) == 0
    assert attend(seqs=0, q=0, out=0) == 0
    assert attend(Q=0, q=0, out=0) == 0
    lib = native.load()
    assert lib.xpress_kv_append(None, None) == native.XPRESS_EINVAL
    assert lib.xpress_paged_attention(None, None) == native.XPRESS_EINVAL


# base, bias, blk, prob, temperature, top_k, top_p, min_p, u, N, B, V, stride_base, stride_bias
_SAMPLE = [MiB, 2 * MiB, 3 * MiB, 4 * MiB, 5 * MiB, 6 * MiB, 7 * MiB, 8 * MiB, 9 * MiB, 2, 4, 100, 100, 100]


def _sample(**at):
    args = list(_SAMPLE)
    for i, v in at.items():
        args[int(i[1:])] = v
    return native.load().xpress_sample_to_blk(*args, None)


@no_gpu_only
@pytest.mark.parametrize("at", [
    dict(_9=-1), dict(_10=0), dict(_11=0), dict(_11=2 ** 31, _12=2 ** 31, _13=2 ** 31), dict(_12=99),
    dict(_13=99), dict(_0=0), dict(_2=0), dict(_4=0), dict(_5=0), dict(_6=0), dict(_7=0), dict(_8=0),
    dict(_0=MiB + 1), dict(_1=2 * MiB + 1), dict(_2=3 * MiB + 4), dict(_3=4 * MiB + 2),
    dict(_4=5 * MiB + 2), dict(_5=6 * MiB + 1), dict(_8=9 * MiB + 3), dict(_2=MiB), dict(_2=2 * MiB + 1192),
    dict(_2=MiB - 8), dict(_3=MiB), dict(_3=9 * MiB), dict(_3=3 * MiB + 8), dict(_2=9 * MiB - 56),
    dict(_2=5 * MiB), dict(_9=2 ** 62), dict(_9=2 ** 31, _10=2), dict(_12=2 ** 61),
])
def test_sample_refuses(at):
    assert _sample(**at) == native.XPRESS_EINVAL


@no_gpu_only
def test_sample_with_no_rows_is_ok():
    assert _sample(_9=0, _0=0, _2=0) == 0
    assert _sample(_10=1, _0=0, _2=0) == 0


def test_plan_and_reserve_check_their_sizes():
    p = native.xpress_paged_attention_plan(32, 1, 32, 8, 128, 4096)
    assert p["launches"] in (1, 2) and p["splits"] * p["chunk"] >= 4096
    assert native.xpress_paged_attention_plan(0, 1, 32, 8, 128, 4096)["launches"] == 0
    assert native.xpress_paged_attention_plan(1, 1, 8, 8, 64, 1)["launches"] == 1
    # a window bounds what is planned for
    w = native.xpress_paged_attention_plan(1, 1, 8, 8, 64, 100000, 100)
    assert w["splits"] * w["chunk"] < 1000
    for bad in ((-1, 1, 8, 8, 64, 10), (1, -1, 8, 8, 64, 10), (1, 1, 8, 3, 64, 10), (1, 1, 0, 8, 64, 10),
                (1, 1, 8, 8, 60, 10), (1, 1, 8, 8, 512, 10), (1, 1, 8, 8, 64, 0), (1, 1, 8, 8, 64, 10, -1)):
        with pytest.raises(native.XpressError):
            native.xpress_paged_attention_plan(*bad)
        assert native.load().xpress_paged_attention_reserve(
            *(list(bad) + [0] * (7 - len(bad))), None) == native.XPRESS_EINVAL


def test_binding_checks_tensors():
    """Shapes, types and devices are looked at before the library is called."""
    bf = dict(dtype=torch.bfloat16)
    kc, vc = torch.zeros(4, 2, 16, 64, **bf), torch.zeros(4, 2, 16, 64, **bf)
    table = torch.zeros(1, 4, dtype=torch.int32)
    q, k = torch.zeros(3, 4, 64, **bf), torch.zeros(3, 2, 64, **bf)
    pos = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        native.xpress_kv_append(q, k, k, q, kc, vc, table, pos, None)
    for a, b, t, why in ((kc, vc[:, :, :8], table, "one type, shape"), (kc, vc.half(), table, "one type"),
                         (kc.float(), vc.float(), table, "bf16, fp16"), (kc, vc, table.long(), "int32"),
                         (kc, vc, table[0], "int32"),
                         (kc.transpose(2, 3), vc.transpose(2, 3), table, "unit stride")):
        with pytest.raises(ValueError, match=why):
            native.xpress_kv_append(q, k, k, q, a, b, t, pos, None)
        with pytest.raises(ValueError, match=why):
            native.xpress_paged_attention(q[None], a, b, t, pos[:1], q[None], 16)
    base = torch.zeros(3, 100, **bf)
    row = torch.zeros(3)
    blk = torch.zeros(1, 4, dtype=torch.int64)
    with pytest.raises(ValueError, match="base"):
        native.xpress_sample_to_blk(base, None, blk, row, row.int(), row, row, row, 1, 4, 101, 101)
    with pytest.raises(ValueError, match="top_k"):
        native.xpress_sample_to_blk(base, None, blk, row, row[:2].clone().int(), row, row, row, 1, 4, 100, 100)
    with pytest.raises(ValueError, match="prob"):
        native.xpress_sample_to_blk(base, None, blk, row, row.int(), row, row, row, 1, 4, 100, 100,
                                    prob=row[1:])


@pytest.mark.gpu
def test_binding_checks_shapes_on_the_gpu():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    kc, vc = torch.zeros(4, 2, 16, 64, **bf), torch.zeros(4, 2, 16, 64, **bf)
    table = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    q, k = torch.zeros(3, 4, 64, **bf), torch.zeros(3, 2, 64, **bf)
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    for args, why in (((q, k[:, :, :32], k, q, kc, vc, table, pos, None), "k:"),
                      ((q, k, k[:2], q, kc, vc, table, pos, None), "v:"),
                      ((q, k, k, q[:2], kc, vc, table, pos, None), "q_out"),
                      ((q, k, k, q.half(), kc, vc, table, pos, None), "q_out"),
                      ((q, k, k, q, kc, vc, table, pos[:2], None), "positions"),
                      ((q, k, k, q, kc, vc, table, pos.long(), None), "positions"),
                      ((q, k, k, q, kc, vc, table, pos, torch.zeros(9, 64, **bf)), "cos_sin"),
                      ((q, k, k, q, kc, vc, table, pos.cpu(), None), "positions")):
        with pytest.raises(ValueError, match=why):
            native.xpress_kv_append(*args)
    q4 = q[None]
    lens = pos[:1]
    for args, kw, why in (((q4, kc, vc, table, lens, q4[:, :2], 16), {}, "out"),
                          ((q4, kc, vc, table, pos, q4, 16), {}, "lens"),
                          ((torch.cat([q4, q4]), kc, vc, table, lens, q4, 16), {}, "q:"),
                          ((q4, kc, vc, table, lens, q4, 16), dict(lse=torch.zeros(1, 3, 4, **bf)), "lse"),
                          ((q4, kc, vc, table, lens, q4, 16), dict(k_scale=torch.zeros(3, device="cuda")),
                           "k_scale")):
        with pytest.raises(ValueError, match=why):
            native.xpress_paged_attention(*args, **kw)
    with pytest.raises(native.XpressError):
        native.xpress_paged_attention(q4, kc, vc, table, lens, torch.empty_like(q4), 65)
    with pytest.raises(native.XpressError):      # out on q
        native.xpress_paged_attention(q4, kc, vc, table, lens, q4, 16)


def test_sample_reserve_checks_its_sizes():
    for bad in ((-1, 2, 1000), (1, 0, 1000), (1, 2, 0), (1, 2, 2 ** 31), (2 ** 31, 3, 1000), (2 ** 62, 2, 10)):
        with pytest.raises(native.XpressError):
            native.xpress_sample_reserve(*bad, stream=0)
    # nothing is needed: no HIP call either
    for none in ((0, 2, 152064), (5, 1, 152064), (100, 2, 152064), (1, 2, 20000)):
        native.xpress_sample_reserve(*none, stream=0)


def sample_inputs(device):
    f = dict(device=device)
    return dict(base=torch.zeros(3, 100, dtype=torch.bfloat16, **f), bias=torch.zeros(3, 100, dtype=torch.bfloat16, **f),
                blk=torch.zeros(1, 4, dtype=torch.int64, **f), temperature=torch.ones(3, **f),
                top_k=torch.zeros(3, dtype=torch.int32, **f), top_p=torch.ones(3, **f), min_p=torch.zeros(3, **f),
                u=torch.full((3,), 0.5, **f), prob=torch.zeros(3, **f))


def sample_wrong(name, device):
    """Tensors for this argument whose storage is long enough, but that are not what it takes."""
    f = dict(device=device)
    if name in ("base", "bias"):
        yield torch.zeros(3, 100, dtype=torch.float16, **f)
        yield torch.zeros(3, 100, **f)
        yield torch.zeros(100, 3, dtype=torch.bfloat16, **f).t()
        yield torch.zeros(3, 200, dtype=torch.bfloat16, **f)[:, ::2]
    elif name == "blk":
        yield torch.zeros(1, 8, dtype=torch.int32, **f)
        yield torch.zeros(1, 4, dtype=torch.float64, **f)
        yield torch.zeros(1, 8, dtype=torch.int64, **f)[:, ::2]
        yield torch.zeros(1, 8, dtype=torch.int64, **f)[:, :3]
    else:
        real = torch.int32 if name == "top_k" else torch.float32
        for other in (torch.int64, torch.float64, torch.int32, torch.float32):
            if other is not real:
                yield torch.zeros(6, dtype=other, **f)
        yield torch.zeros(3, 4, dtype=real, **f)[:, 0]      # a column of a table of settings
        yield torch.zeros(1, dtype=real, **f).expand(3)
        yield torch.zeros(8, dtype=real, **f)[:2]           # too few, in a longer storage


def refuses_sample(device):
    good = sample_inputs(device)
    for name in good:
        for bad in sample_wrong(name, device):
            args = dict(good, **{name: bad})
            with pytest.raises(ValueError, match="^%s:" % name):
                native.xpress_sample_to_blk(*[args[x] for x in ("base", "bias", "blk", "temperature", "top_k", "top_p",
                                                                "min_p", "u")], 1, 4, 100, 100, 100, prob=args["prob"])


def test_sample_refuses_other_types_and_strides():
    refuses_sample("cpu")


@pytest.mark.gpu
def test_sample_refuses_other_types_and_strides_on_the_gpu():
    refuses_sample("cuda")
    good = sample_inputs("cuda")
    for name in good:
        if name == "base":
            continue
        args = dict(good, **{name: good[name].cpu()})
        with pytest.raises(ValueError, match="^%s: expected a tensor on cuda:0" % name):
            native.xpress_sample_to_blk(*[args[x] for x in ("base", "bias", "blk", "temperature", "top_k", "top_p",
                                                            "min_p", "u")], 1, 4, 100, 100, 100, prob=args["prob"])
    assert (good["blk"] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [torch.int16, torch.uint16])
def test_sample_takes_bits_and_addresses(bits):
    good = sample_inputs("cuda")
    good["base"].copy_(torch.randn(3, 100))
    names = ("base", "bias", "blk", "temperature", "top_k", "top_p", "min_p", "u")
    native.xpress_sample_to_blk(*[good[x] for x in names], 1, 4, 100, 100, 100)
    want = good["blk"].clone()
    assert want[0, 1:].any()
    for other in (dict(good, base=good["base"].view(bits), bias=good["bias"].view(bits)),
                  {k: v.data_ptr() for k, v in good.items()}):
        good["blk"].zero_()
        native.xpress_sample_to_blk(*[other[x] for x in names], 1, 4, 100, 100, 100)
        assert torch.equal(good["blk"], want)


@pytest.mark.parametrize("shape", [
    (1, 4096, 32, 8, 128, 131072), (1, 32768, 32, 8, 128, 32768), (4, 8192, 32, 8, 128, 8192),
    (128, 16, 32, 8, 128, 131072), (4096, 1, 32, 8, 128, 131072), (1000, 2, 32, 2, 64, 2 ** 20),
    (1, 2 ** 20, 32, 8, 256, 2 ** 20), (2 ** 20, 1, 16, 16, 256, 2 ** 30), (64, 1, 8, 8, 64, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_parts_take_a_gib_at_most(shape):
    """Whatever the lengths' bound and the number of queries, the parts' sums stay within 1 GiB."""
    N, Q, Hq, heads, dim, max_len = shape[:6]
    p = native.xpress_paged_attention_plan(*shape)
    assert p["splits"] * p["chunk"] >= max_len and (p["splits"] - 1) * p["chunk"] < max_len
    assert p["chunk"] % 128 == 0 and p["chunk"] <= 2 ** 30
    if p["splits"] > 1 and max_len <= 2 ** 30:
        assert p["splits"] * N * Q * Hq * (dim + 2) * 4 <= 1 << 30


def test_groups_of_rows_that_fill_the_chip_are_not_split():
    for shape in ((1, 4096, 32, 8, 128, 131072), (1, 512, 256, 8, 64, 5000), (1, 32768, 32, 8, 128, 32768, 4096)):
        p = native.xpress_paged_attention_plan(*shape)
        assert p["splits"] == 1 and p["launches"] == 1


@no_gpu_only
@pytest.mark.parametrize("scale", [3.3e38, -3.3e38, 2.4e38, float("-inf")])
def test_attention_refuses_scales_that_pass_fp32_in_base_2(scale):
    """The kernel would hold infinity, and 0 times it is NaN."""
    assert attend(scale=scale) == native.XPRESS_EINVAL


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def test_append_takes_q_and_q_out_together(device):
    bf = dict(dtype=torch.bfloat16, device=device)
    kc, vc = torch.zeros(4, 2, 16, 64, **bf), torch.zeros(4, 2, 16, 64, **bf)
    table = torch.zeros(1, 4, dtype=torch.int32, device=device)
    q, k = torch.zeros(3, 4, 64, **bf), torch.zeros(3, 2, 64, **bf)
    pos = torch.zeros(3, dtype=torch.int32, device=device)
    for a, b in ((q, None), (None, q)):
        with pytest.raises(ValueError, match="^q, q_out:"):
            native.xpress_kv_append(a, k, k, b, kc, vc, table, pos, None)
