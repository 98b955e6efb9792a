"""The host module's functions for drafts that branch, pages and beams: the same calls as
the binding's Python code makes, and None for whatever that code refuses."""
import numpy as np
import pytest
import torch

import drafts_ref
import serving_ref
from test_marshal import Never
from vocab_wide_add_amd import native


def i32(*x, device="cpu"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def inputs(device):
    rng = np.random.default_rng(6)
    kc, vc, table = serving_ref.paged_pool(rng, [40, 17], 2, 64, 16, "e4m3", "token")
    d = dict(kc=kc, vc=vc, table=table, q=torch.from_numpy(rng.standard_normal((2, 3, 4, 64)).astype(np.float32)),
             k=torch.from_numpy(rng.standard_normal((6, 2, 64)).astype(np.float32)),
             tree=drafts_ref.words_of(drafts_ref.random_trees(rng, 2, 3)[1]), lens=i32(40, 17), start=i32(37, 14),
             pos=i32(37, 38, 38, 14, 15, 15), places=i32(37, 38, 39, 14, 15, 16),
             cs=torch.from_numpy(rng.standard_normal((50, 32)).astype(np.float32)), ks=torch.tensor([0.05, 0.04]),
             path=i32([0, 2], [0, 1]), count=i32(2, 1), refs=i32(*([1] * kc.shape[0] + [0] * 4)), src=i32(1, 0, 0),
             base=torch.from_numpy(rng.standard_normal((4, 100)).astype(np.float32)), scores=torch.zeros(4))
    d = {k: torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=device).copy_(x) for k, x in d.items()}
    for x in ("q", "k", "base"):
        d[x] = d[x].to(torch.bfloat16)
    return d


def step(device="cuda"):
    """One call of each function; everything they wrote."""
    d = inputs(device)
    kw = dict(device=device)
    native.xpress_kv_append_at(None, d["k"], d["k"], None, d["kc"], d["vc"], d["table"], d["places"], d["pos"],
                               d["cs"], k_scale=d["ks"], v_scale=d["ks"])
    out, lse = torch.empty_like(d["q"]), torch.empty(2, 3, 4, **kw)
    native.xpress_tree_attention(d["q"], d["kc"], d["vc"], d["table"], d["lens"], d["tree"], out, 40, lse=lse,
                                 scale=0.2, window=9, sinks=3, k_scale=d["ks"], v_scale=d["ks"])
    more = torch.empty_like(d["q"])
    native.xpress_sink_attention(d["q"], d["kc"], d["vc"], d["table"], d["lens"], more, 40, 9, 3)
    native.xpress_kv_compact(d["kc"], d["vc"], d["table"], d["start"], d["path"], d["count"])
    W = d["table"].shape[1]
    new_refs, new_table = torch.empty_like(d["refs"]), torch.empty(3, W, dtype=torch.int32, **kw)
    copies, missing = torch.empty(3, 3, dtype=torch.int32, **kw), torch.empty(1, dtype=torch.int32, **kw)
    native.xpress_kv_fork(d["refs"], d["table"], d["lens"], d["src"], new_refs, new_table, copies, 16, missing=missing)
    native.xpress_kv_fork(d["refs"], d["table"], d["lens"], d["src"], new_refs, new_table, copies, 16)
    native.xpress_kv_copy(d["kc"], d["vc"], copies % d["kc"].shape[0])
    grown, counts = new_table.clone(), new_refs.clone()
    native.xpress_kv_free(counts, grown, i32(5, 40, 0, **kw), 16, window=20, sinks=1)
    native.xpress_kv_grow(counts, grown, i32(5, 40, 0, **kw), i32(30, 41, 17, **kw), 16, missing=missing)
    best, rows = torch.empty(2, 3, **kw), torch.empty(2, 3, dtype=torch.int32, **kw)
    ids = torch.empty(2, 3, dtype=torch.int64, **kw)
    native.xpress_beam_select(d["base"], d["base"], d["scores"], best, rows, ids, 2, 2, 90, 3, 100, 100)
    states = torch.empty(6, 100, dtype=torch.bfloat16, **kw), torch.empty(6, **kw)
    native.xpress_beam_reorder([(d["base"], states[0]), (d["scores"], states[1])], rows)
    torch.cuda.synchronize()
    return [x.contiguous().view(torch.uint8).cpu() for x in (
        d["kc"], d["vc"], out, lse, more, new_refs, new_table, copies, missing, grown, counts, best, rows, ids, *states)]


@pytest.mark.gpu
def test_same_calls_as_the_python_code(monkeypatch):
    got = step()
    monkeypatch.setattr(native, "_marshal", Never())
    want = step()
    for i, (x, y) in enumerate(zip(got, want)):
        assert torch.equal(x, y), i


@pytest.mark.gpu
def test_it_takes_the_regular_case(monkeypatch):
    """None of the calls above falls back to the Python code."""
    def struct(*a):
        raise AssertionError("the Python code made the call")
    native._use_torch()
    for name in ("_kv_cache", "_pages_of", "_plain", "_numbers", "_logits"):
        monkeypatch.setattr(native, name, struct)
    step()


def test_irregular_arguments_are_left_alone():
    """No entry point is called (address 0 would end the process): None comes back."""
    native._use_torch()
    m, d = native._marshal, inputs("cpu")
    cache = [d["kc"], d["vc"], d["table"]]
    good = {
        "kv_append_at": [None, d["k"], d["k"], None, *cache, d["pos"], d["cs"], None, None, None, False, d["places"]],
        "sink_attention": [d["q"], *cache, d["lens"], d["q"], None, None, None, 40, 0, None, 4],
        "tree_attention": [d["q"], *cache, d["lens"], d["q"], None, None, None, 40, 0, None, 4, d["tree"]],
        "kv_fork": [d["refs"], d["table"], d["lens"], d["src"], d["refs"], d["table"], d["path"], None, 16],
        "kv_copy": [*cache[:2], d["path"]],
        "kv_grow": [d["refs"], d["table"], d["lens"], d["lens"], None, 16],
        "kv_free": [d["refs"], d["table"], d["lens"], 16, 0, 0],
        "kv_compact": [*cache, d["start"], d["path"], d["count"]],
        "beam_select": [d["base"], None, d["scores"], d["scores"], d["src"], d["src"], 2, 2, 90, 3, 100, 100],
        "beam_reorder": [[(d["base"], d["base"])], d["src"]],
    }
    assert set(good) == set(native.load().at)
    for name, args in good.items():
        f = getattr(m, name)
        assert f(0, 0, *args) is None, name                          # on the CPU
        for i in range(len(args)):
            for bad in (None, 7.5, "x", d["lens"].long()):
                assert f(0, 0, *args[:i], bad, *args[i + 1:]) is None, (name, i)
        with pytest.raises(TypeError):
            f(0, 0, *args[1:])
    assert m.beam_reorder(0, 0, [d["base"]], d["src"]) is None
    assert m.beam_reorder(0, 0, [(d["base"],)], d["src"]) is None
    for f, at in ((m.kv_free, 3), (m.beam_select, 6)):
        args = list(good[{m.kv_free: "kv_free", m.beam_select: "beam_select"}[f]])
        args[at] = 2 ** 70
        with pytest.raises(OverflowError):
            f(0, 0, *args)


@pytest.mark.gpu
def test_tensors_of_another_device_than_the_current_one(monkeypatch):
    """The current device's stream does not fit them: refused by each function's Python code."""
    monkeypatch.setattr(native, "_marshal", Never())
    d = inputs("cuda")
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    t = d["table"]
    for call in (
            lambda: native.xpress_kv_fork(d["refs"], t, d["lens"], d["lens"], d["refs"].clone(), t.clone(),
                                          d["path"], 16, stream=0),
            lambda: native.xpress_kv_copy(d["kc"], d["vc"], d["path"], stream=0),
            lambda: native.xpress_kv_grow(d["refs"], t, d["lens"], d["lens"], 16, stream=0),
            lambda: native.xpress_kv_free(d["refs"], t, d["lens"], 16, stream=0),
            lambda: native.xpress_kv_compact(d["kc"], d["vc"], t, d["start"], d["path"], d["count"], stream=0),
            lambda: native.xpress_sink_attention(d["q"], d["kc"], d["vc"], t, d["lens"], d["q"].clone(), 40, 9, 3,
                                                 stream=0),
            lambda: native.xpress_tree_attention(d["q"], d["kc"], d["vc"], t, d["lens"], d["tree"], d["q"].clone(), 40,
                                                 stream=0),
            lambda: native.xpress_kv_append_at(None, d["k"], d["k"], None, d["kc"], d["vc"], t, d["places"], d["pos"],
                                               None, stream=0),
            lambda: native.xpress_beam_select(d["base"], None, d["scores"], d["scores"].clone(), d["pos"],
                                              torch.zeros(4, dtype=torch.int64, device="cuda"), 2, 2, 90, 2, 100,
                                              stream=0),
            lambda: native.xpress_beam_reorder([(d["base"], d["base"].clone())], d["pos"], stream=0)):
        with pytest.raises(ValueError, match="current device is cuda:1"):
            call()
