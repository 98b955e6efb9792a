"""The host module that fills the serving operators' argument structs: the same calls as
the binding's Python code makes, and None for whatever that code refuses."""
import inspect
import sys

import numpy as np
import pytest
import torch

import serving_ref as ref
from vocab_wide_add_amd import native


class Never:
    """A host module that leaves every call to the Python code."""

    def __getattr__(self, name):
        return lambda *a: None


def inputs(device):
    rng = np.random.default_rng(5)
    kc, vc, table = ref.paged_pool(rng, [40, 17], 2, 64, 16, "e4m3", "token")
    rows = torch.from_numpy(rng.standard_normal((6, 8, 64)).astype(np.float32)).to(torch.bfloat16)
    d = dict(kc=kc, vc=vc, table=table, rows=rows, pos=torch.tensor([37, 38, 39, 14, 15, 16], dtype=torch.int32),
             cs=torch.from_numpy(rng.standard_normal((50, 32)).astype(np.float32)),
             seq=torch.tensor([0, 0, 0, 1, 1, 1], dtype=torch.int32), ks=torch.tensor([0.05, 0.04]),
             vs=torch.tensor([0.03, 0.06]), lens=torch.tensor([40, 17], dtype=torch.int32))
    return {k: torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=device).copy_(x)
            for k, x in d.items()}


def step():
    """One call of each operator; everything they wrote."""
    d = inputs("cuda")
    q, k, v = d["rows"][:, :4], d["rows"][:, 4:6], d["rows"][:, 6:]
    q_out = torch.empty(6, 4, 64, dtype=torch.bfloat16, device="cuda")
    native.xpress_kv_append(q, k, v, q_out, d["kc"], d["vc"], d["table"], d["pos"], d["cs"], seq_of=d["seq"],
                            k_scale=d["ks"], v_scale=d["vs"], interleaved=True)
    native.xpress_kv_append(None, k, v, None, d["kc"], d["vc"], d["table"], d["pos"], None, k_scale=d["ks"])
    out = torch.empty(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    lse = torch.empty(2, 3, 4, device="cuda")
    native.xpress_paged_attention(q_out.view(2, 3, 4, 64), d["kc"], d["vc"], d["table"], d["lens"], out, 40,
                                  lse=lse, window=20, scale=0.2, k_scale=d["ks"], v_scale=d["vs"])
    whole = torch.empty(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    native.xpress_paged_attention(q_out.view(2, 3, 4, 64), d["kc"], d["vc"], d["table"], d["lens"], whole, 40)
    blk, prob = torch.zeros(2, 4, dtype=torch.int64, device="cuda"), torch.empty(6, device="cuda")
    row = torch.full((6,), 0.7, device="cuda")
    base = q_out.reshape(6, 256)
    native.xpress_sample_to_blk(base, base, blk, row, torch.full((6,), 9, dtype=torch.int32, device="cuda"), row,
                                row / 100, row, 2, 4, 250, 256, 256, prob=prob)
    torch.cuda.synchronize()
    return [x.contiguous().view(torch.uint8).cpu() for x in (q_out, d["kc"], d["vc"], out, lse, whole, blk, prob)]


@pytest.mark.gpu
def test_same_calls_as_the_python_code(monkeypatch):
    got = step()
    monkeypatch.setattr(native, "_marshal", Never())
    want = step()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.gpu
def test_it_takes_the_regular_case(monkeypatch):
    """None of the calls above falls back to the Python code."""
    def struct(*a):
        raise AssertionError("the Python code made the call")
    native._use_torch()
    monkeypatch.setattr(native, "_kv_cache", struct)
    monkeypatch.setattr(native, "_span", struct)
    step()


def test_irregular_arguments_are_left_alone():
    """No entry point is called (address 0 would end the process): None comes back."""
    native._use_torch()
    m = native._marshal
    d = inputs("cpu")
    q, k, v = d["rows"][:, :4], d["rows"][:, 4:6], d["rows"][:, 6:]
    good = [0, 0, q, k, v, q, d["kc"], d["vc"], d["table"], d["pos"], d["cs"], d["seq"], d["ks"], d["vs"], False]
    assert m.kv_append(*good) is None                  # on the CPU
    for at, bad in ((2, None), (3, 7), (4, "v"), (6, None), (9, None), (8, d["table"].long())):
        assert m.kv_append(*(good[:at] + [bad] + good[at + 1:])) is None
    good = [0, 0, q.view(2, 3, 4, 64) if q.is_contiguous() else q.reshape(2, 3, 4, 64), d["kc"], d["vc"],
            d["table"], d["lens"], q.reshape(2, 3, 4, 64), None, d["ks"], d["vs"], 40, 0, None]
    assert m.paged_attention(*good) is None
    assert m.paged_attention(*(good[:11] + [40.0] + good[12:])) is None
    r = torch.zeros(1)
    good = [0, 0, r, None, r, None, r, r, r, r, r, 1, 2, 10, 10, 10]
    assert m.sample(*good) is None
    assert m.sample(*(good[:2] + [12345] + good[3:])) is None      # a bare address
    assert m.sample(*(good[:11] + [2 ** 62, 3] + good[13:])) is None
    for f, n in ((m.kv_append, 15), (m.paged_attention, 14), (m.sample, 16)):
        with pytest.raises(TypeError):
            f(*[None] * (n - 1))


def test_the_other_entry_points_do_without_it(monkeypatch):
    """A stream is looked up where the module is not built; a serving operator says so."""
    monkeypatch.setitem(sys.modules, "vocab_wide_add_amd._marshal", None)
    monkeypatch.delattr("vocab_wide_add_amd._marshal", raising=False)
    monkeypatch.setattr(native, "_marshal", None)
    monkeypatch.setattr(native, "_torch", None)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1234, raising=False)
    assert native._stream(None) == 1234
    d = inputs("cpu")
    q, k, v = d["rows"][:, :4], d["rows"][:, 4:6], d["rows"][:, 6:]
    with pytest.raises(ImportError, match="_marshal.so"):
        native.xpress_kv_append(q, k, v, q, d["kc"], d["vc"], d["table"], d["pos"], None)


@pytest.mark.parametrize("op", ["append", "attention", "sample"])
def test_first_calls_of_two_threads(monkeypatch, op):
    """Whatever another thread's first call has set so far, a call finds all that it needs."""
    native._use_torch()
    d = inputs("cpu")
    q, k, v = d["rows"][:, :4], d["rows"][:, 4:6], d["rows"][:, 6:]
    n = torch.zeros(3)

    def call():
        if op == "append":
            native.xpress_kv_append(q, k, v, q, d["kc"], d["vc"], d["table"], d["pos"], None)
        elif op == "attention":
            native.xpress_paged_attention(q.reshape(2, 3, 4, 64), d["kc"], d["vc"], d["table"], d["lens"],
                                          q.reshape(2, 3, 4, 64), 40)
        else:
            native.xpress_sample_to_blk(torch.zeros(3, 8, dtype=torch.bfloat16), None,
                                        torch.zeros(1, 4, dtype=torch.int64), n, n.int(), n, n, n, 1, 4, 8, 8)

    # what the names hold after each assignment of a first call, in its order
    states, names = [], ("_torch", "_marshal")
    real = {x: getattr(native, x) for x in names}

    order = [x.split(" = ")[0].strip() for x in inspect.getsource(native).splitlines()
             if x.startswith(("        _torch = ", "        _marshal = "))]
    assert sorted(order) == sorted(names)
    held = dict.fromkeys(names)
    states.append(dict(held))
    for x in order:
        held[x] = real[x]
        states.append(dict(held))
    for s in states:
        for x, y in s.items():
            monkeypatch.setattr(native, x, y)
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.gpu
def test_tensors_of_another_device_than_the_current_one(monkeypatch):
    """The current device's stream and workspace do not fit them: refused.  (The Python code, told
    of another current device; with one GPU the module cannot be.)"""
    d = inputs("cuda")
    q, k, v = d["rows"][:, :4], d["rows"][:, 4:6], d["rows"][:, 6:]
    n = torch.zeros(3, device="cuda")
    out = torch.empty(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty(6, 4, 64, dtype=torch.bfloat16, device="cuda")
    monkeypatch.setattr(native, "_marshal", Never())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        native.xpress_kv_append(q, k, v, q_out, d["kc"], d["vc"], d["table"], d["pos"], None, stream=0)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        native.xpress_paged_attention(q_out.view(2, 3, 4, 64), d["kc"], d["vc"], d["table"], d["lens"], out, 40,
                                      stream=0)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        native.xpress_sample_to_blk(torch.zeros(3, 8, dtype=torch.bfloat16, device="cuda"), None,
                                    torch.zeros(1, 4, dtype=torch.int64, device="cuda"), n, n.int(), n, n, n, 1, 4,
                                    8, 8, stream=0)
