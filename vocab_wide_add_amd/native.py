"""ctypes binding of ``libxpress_argmax.so`` (declared in include/xpress_argmax.h).

Argument marshalling only: every step of the readout runs in the library's
HIP kernels.  Entry points keep the C names.  Tensor arguments may be torch
tensors on a GPU (their ``data_ptr()`` is passed) or plain integer device
addresses; for a tensor the binding also checks that its storage covers the
bytes the call will touch, which a bare pointer cannot tell the library.  A
nonzero status raises :class:`XpressError`.  If the library has not been
built, the first call raises -- there is no fallback path.

The serving operators take their arguments from torch tensors in a small host
module, ``_marshal.so`` (4 us a call; asking the tensors in Python takes 10); the
Python code here makes the call where an argument is not a regular tensor, and
says what is wrong with it.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libxpress_argmax.so")

XPRESS_OK = 0
XPRESS_EINVAL = 1
XPRESS_EHIP = 2
XPRESS_ENOMEM = 3
XPRESS_ECAPTURE = 4
XPRESS_ESCRATCH = 5

XPRESS_COMBINE_AUTO = 0
XPRESS_COMBINE_SINGLE = 1
XPRESS_COMBINE_ATOMIC = 2
XPRESS_COMBINE_TWO_PASS = 3
XPRESS_COMBINE_BALANCED = 4

COMBINE_NAMES = {XPRESS_COMBINE_SINGLE: "single", XPRESS_COMBINE_ATOMIC: "atomic",
                 XPRESS_COMBINE_TWO_PASS: "two_pass", XPRESS_COMBINE_BALANCED: "balanced"}

XPRESS_BF16 = 0
XPRESS_FP16 = 1
XPRESS_E4M3 = 2

_lock = threading.Lock()
_lib = None


class XpressError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = "%s: %s" % (where, xpress_error_string(status))
        if status == XPRESS_EHIP:
            msg += " (hipError %d)" % xpress_last_hip_error()
        super().__init__(msg)


def load():
    """Load the library (once).  Raises ImportError when it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                "libxpress_argmax.so is not built; run `python -m vocab_wide_add_amd.build`")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        ip = ctypes.POINTER(ctypes.c_int)
        lib.xpress_add_argmax_to_blk.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, vp]
        lib.xpress_add_argmax_to_blk.restype = i32
        lib.xpress_add_argmax_to_blk_noalloc.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, vp]
        lib.xpress_add_argmax_to_blk_noalloc.restype = i32
        lib.xpress_topc_argmax_to_blk.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp]
        lib.xpress_topc_argmax_to_blk.restype = i32
        lib.xpress_readout_gemm_argmax_to_blk.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64,
                                                          i64, vp]
        lib.xpress_readout_gemm_argmax_to_blk.restype = i32
        lib.xpress_latent_pass.argtypes = [vp] * 10 + [i64] * 5 + [vp]
        lib.xpress_latent_pass.restype = i32
        lib.xpress_latent_set_tiles.argtypes = [i32, i32, i32]
        lib.xpress_latent_set_tiles.restype = i32
        lib.xpress_latent_reserve.argtypes = [i64, i64, i64, i64, vp]
        lib.xpress_latent_reserve.restype = i32
        lib.xpress_reserve.argtypes = [i64, i64, i64, vp]
        lib.xpress_reserve.restype = i32
        lib.xpress_release.argtypes = []
        lib.xpress_release.restype = i32
        lib.xpress_set_workspace_limit.argtypes = [i64]
        lib.xpress_set_workspace_limit.restype = i32
        lib.xpress_workspace_bytes.argtypes = [ctypes.POINTER(ctypes.c_int64)]
        lib.xpress_workspace_bytes.restype = i32
        lib.xpress_set_plan.argtypes = [i32, i32, i32]
        lib.xpress_set_plan.restype = i32
        lib.xpress_set_reverse_order.argtypes = [i32]
        lib.xpress_set_reverse_order.restype = i32
        lib.xpress_describe_plan.argtypes = [vp, vp, i64, i64, i64, i64, i64,
                                             ip, ip, ip, ip, ip]
        lib.xpress_describe_plan.restype = i32
        lib.xpress_describe_gemm_plan.argtypes = [i64, i64, i64, ip, ip, ip, ip]
        lib.xpress_describe_gemm_plan.restype = i32
        lib.xpress_bf16_add_round_table.argtypes = [vp, i64, vp, vp]
        lib.xpress_bf16_add_round_table.restype = i32
        lib.xpress_read_probe.argtypes = [vp, vp, i64, i64, i64, i32, vp, vp]
        lib.xpress_read_probe.restype = i32
        cp = ctypes.c_char_p
        lib.xpress_kv_append.argtypes = [cp, vp]
        lib.xpress_kv_append.restype = i32
        lib.xpress_paged_attention.argtypes = [cp, vp]
        lib.xpress_paged_attention.restype = i32
        lib.xpress_paged_attention_reserve.argtypes = [i64] * 7 + [vp]
        lib.xpress_paged_attention_reserve.restype = i32
        lib.xpress_paged_attention_plan.argtypes = [i64] * 7 + [ip, ip, ip, ip]
        lib.xpress_paged_attention_plan.restype = i32
        lib.xpress_sample_to_blk.argtypes = [vp] * 9 + [i64] * 5 + [vp]
        lib.xpress_sample_to_blk.restype = i32
        lib.xpress_sample_reserve.argtypes = [i64, i64, i64, vp]
        lib.xpress_sample_reserve.restype = i32
        lib.append_at, lib.attention_at, lib.sample_at = [
            ctypes.cast(f, vp).value for f in (lib.xpress_kv_append, lib.xpress_paged_attention,
                                               lib.xpress_sample_to_blk)]
        lib.xpress_last_hip_error.argtypes = []
        lib.xpress_last_hip_error.restype = i32
        lib.xpress_error_string.argtypes = [i32]
        lib.xpress_error_string.restype = ctypes.c_char_p
        lib.xpress_version.argtypes = []
        lib.xpress_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _ptr(x):
    """Device address of a torch tensor on a GPU, or an int address as is."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if not x.is_cuda:
            raise ValueError("expected a tensor on a GPU, got one on %s" % x.device)
        return x.data_ptr()
    raise TypeError("expected a GPU tensor or an integer address, got %r" % type(x))


def _span(t, nbytes: int, what: str):
    """Refuse a tensor whose storage ends before the ``nbytes`` the call
    will touch from its first element (integer addresses are the caller's
    responsibility, as in the C ABI)."""
    if nbytes <= 0 or t is None or isinstance(t, int) or not hasattr(t, "untyped_storage"):
        return
    avail = t.untyped_storage().nbytes() - t.storage_offset() * t.element_size()
    if nbytes > avail:
        raise ValueError("%s: the call reads or writes %d bytes from the tensor's first "
                         "element, its storage holds %d" % (what, nbytes, avail))


def _stream(stream):
    """HIP stream handle: None means torch's current stream on the current device."""
    if stream is None:
        torch = _torch or _import_torch()
        if not torch.cuda.is_initialized():
            return torch.cuda.current_stream().cuda_stream
        # the same handle, without building the Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _stream_of_tensors(stream):
    """The same for a call with tensors: before the GPU is in use there is none of
    them on it, and the handle goes nowhere."""
    if stream is None:
        if not _torch.cuda.is_initialized():
            return 0
        return _torch._C._cuda_getCurrentRawStream(_torch._C._cuda_getDevice())
    return _stream(stream)


def _check(status: int, where: str):
    if status != XPRESS_OK:
        raise XpressError(status, where)


def xpress_add_argmax_to_blk(base, bias, blk, N: int, B: int, V: int,
                             stride_base_r: int, stride_bias_r: int, stream=None) -> None:
    """blk[n, 1+b] = argmax_v bf16(base[r, v] + bias[r, v]), r = n*(B-1) + b.

    Queued on ``stream`` (default: torch's current stream).  See the header
    for the layout rules and error behaviour.
    """
    rows = int(N) * (int(B) - 1)
    if rows > 0:
        _span(base, ((rows - 1) * int(stride_base_r) + int(V)) * 2, "base")
        _span(bias, ((rows - 1) * int(stride_bias_r) + int(V)) * 2, "bias")
        _span(blk, int(N) * int(B) * 8, "blk")
    lib = load()
    _check(lib.xpress_add_argmax_to_blk(_ptr(base), _ptr(bias), _ptr(blk), int(N), int(B),
                                        int(V), int(stride_base_r), int(stride_bias_r),
                                        _stream(stream)),
           "xpress_add_argmax_to_blk")


def bind_add_argmax_to_blk(base, bias, blk, N: int, B: int, V: int, stride_base_r: int,
                           stride_bias_r: int, stream=None):
    """xpress_add_argmax_to_blk with its arguments marshalled once: checks
    the tensors' spans and resolves pointers and the stream now, and returns
    a callable that queues the readout (the library validates the arguments
    again on every call and the callable raises on a nonzero status).  The
    tensors must stay alive and in place while the callable is used."""
    rows = int(N) * (int(B) - 1)
    if rows > 0:
        _span(base, ((rows - 1) * int(stride_base_r) + int(V)) * 2, "base")
        _span(bias, ((rows - 1) * int(stride_bias_r) + int(V)) * 2, "bias")
        _span(blk, int(N) * int(B) * 8, "blk")
    fn = load().xpress_add_argmax_to_blk
    args = (_ptr(base), _ptr(bias), _ptr(blk), int(N), int(B), int(V), int(stride_base_r),
            int(stride_bias_r), _stream(stream))

    def call():
        st = fn(*args)
        if st != XPRESS_OK:
            raise XpressError(st, "xpress_add_argmax_to_blk")
    return call


def xpress_add_argmax_to_blk_noalloc(base, bias, blk, N: int, B: int, V: int,
                                     stride_base_r: int, stride_bias_r: int, stream=None) -> None:
    """The same readout without any device allocation (a fixed key table
    built into the library, shared by every call on the GPU)."""
    rows = int(N) * (int(B) - 1)
    if rows > 0:
        _span(base, ((rows - 1) * int(stride_base_r) + int(V)) * 2, "base")
        _span(bias, ((rows - 1) * int(stride_bias_r) + int(V)) * 2, "bias")
        _span(blk, int(N) * int(B) * 8, "blk")
    lib = load()
    _check(lib.xpress_add_argmax_to_blk_noalloc(_ptr(base), _ptr(bias), _ptr(blk), int(N),
                                                int(B), int(V), int(stride_base_r),
                                                int(stride_bias_r), _stream(stream)),
           "xpress_add_argmax_to_blk_noalloc")


def xpress_topc_argmax_to_blk(base_c, bias_c, cand, blk, N: int, B: int, C: int,
                              stream=None) -> None:
    """blk[n, 1+j] = cand[r, argmax_c bf16(base_c[r, c] + bias_c[r, c])],
    r = n*(B-1) + j; base_c, bias_c, cand are [N, B-1, C] contiguous."""
    rows = int(N) * (int(B) - 1)
    if rows > 0:
        _span(base_c, rows * int(C) * 2, "base_c")
        _span(bias_c, rows * int(C) * 2, "bias_c")
        _span(cand, rows * int(C) * 8, "cand")
        _span(blk, int(N) * int(B) * 8, "blk")
    lib = load()
    _check(lib.xpress_topc_argmax_to_blk(_ptr(base_c), _ptr(bias_c), _ptr(cand), _ptr(blk),
                                         int(N), int(B), int(C), _stream(stream)),
           "xpress_topc_argmax_to_blk")


def xpress_readout_gemm_argmax_to_blk(base, x, w, blk, N: int, B: int, V: int, R: int,
                                      stride_base_r: int, stream=None) -> None:
    """blk[n, 1+b] = argmax_v bf16(base[r, v] + bf16(x[r] . w[v])), r = n*(B-1) + b;
    x is [rows, R], w is [V, R], all bf16 on the GPU."""
    rows = int(N) * (int(B) - 1)
    if rows > 0:
        _span(base, ((rows - 1) * int(stride_base_r) + int(V)) * 2, "base")
        _span(x, rows * int(R) * 2, "x")
        _span(w, int(V) * int(R) * 2, "w")
        _span(blk, int(N) * int(B) * 8, "blk")
    lib = load()
    _check(lib.xpress_readout_gemm_argmax_to_blk(_ptr(base), _ptr(x), _ptr(w), _ptr(blk),
                                                 int(N), int(B), int(V), int(R),
                                                 int(stride_base_r), _stream(stream)),
           "xpress_readout_gemm_argmax_to_blk")


def xpress_latent_pass(blk, am1, xh, w1, wlat, mixl, wg, wu, wd, lat_out, N: int, B: int,
                       R: int, H: int, V: int, stream=None) -> None:
    """Latent stage of one pass: lat_out [N, B-1, R] from the block tokens
    blk [N, B], am1 [N] (int64), the hidden cache xh [N, B, R], the embedding
    w1 [V, R] and the out-major weights wlat [R, R], mixl [B, B, R],
    wg / wu [H, R], wd [R, H] (all bf16 on the GPU)."""
    n, b, r, h, v = int(N), int(B), int(R), int(H), int(V)
    if n > 0:
        for t, nb, what in ((blk, n * b * 8, "blk"), (am1, n * 8, "am1"),
                            (xh, n * b * r * 2, "xh"), (w1, v * r * 2, "w1"),
                            (wlat, r * r * 2, "wlat"), (mixl, b * b * r * 2, "mixl"),
                            (wg, h * r * 2, "wg"), (wu, h * r * 2, "wu"), (wd, r * h * 2, "wd"),
                            (lat_out, n * (b - 1) * r * 2, "lat_out")):
            _span(t, nb, what)
    lib = load()
    _check(lib.xpress_latent_pass(_ptr(blk), _ptr(am1), _ptr(xh), _ptr(w1), _ptr(wlat),
                                  _ptr(mixl), _ptr(wg), _ptr(wu), _ptr(wd), _ptr(lat_out),
                                  int(N), int(B), int(R), int(H), int(V), _stream(stream)),
           "xpress_latent_pass")


def xpress_latent_reserve(N: int, B: int, R: int, H: int, stream=None) -> None:
    _check(load().xpress_latent_reserve(int(N), int(B), int(R), int(H), _stream(stream)),
           "xpress_latent_reserve")


def xpress_latent_set_tiles(mix: int = 0, gate: int = 0, down: int = 0) -> None:
    """Row-slab counts of the three latent kernels: 1, 2 or 4 (direct kernels),
    8 (LDS-staged kernels), 0 = automatic."""
    _check(load().xpress_latent_set_tiles(int(mix), int(gate), int(down)),
           "xpress_latent_set_tiles")


def xpress_reserve(N: int, B: int, V: int, stream=None) -> None:
    _check(load().xpress_reserve(int(N), int(B), int(V), _stream(stream)), "xpress_reserve")


def xpress_release() -> None:
    _check(load().xpress_release(), "xpress_release")


def xpress_set_workspace_limit(nbytes: int) -> None:
    """Cap on the library's workspace per device (0 = none); past it a call
    returns XPRESS_ENOMEM (raised as XpressError)."""
    _check(load().xpress_set_workspace_limit(int(nbytes)), "xpress_set_workspace_limit")


def xpress_workspace_bytes() -> int:
    """Bytes of workspace (live and retired) held on the current device."""
    out = ctypes.c_int64(0)
    _check(load().xpress_workspace_bytes(ctypes.byref(out)), "xpress_workspace_bytes")
    return int(out.value)


def xpress_set_plan(combine: int = XPRESS_COMBINE_AUTO, splits: int = 0,
                    block_threads: int = 0) -> None:
    _check(load().xpress_set_plan(int(combine), int(splits), int(block_threads)),
           "xpress_set_plan")


def xpress_set_reverse_order(reversed_: bool) -> None:
    """Debug: later launches visit their work units from last to first."""
    _check(load().xpress_set_reverse_order(1 if reversed_ else 0), "xpress_set_reverse_order")


def xpress_describe_plan(base, bias, N: int, B: int, V: int, stride_base_r: int,
                         stride_bias_r: int) -> dict:
    """The plan a call would use, from sizes and pointer alignment (host only)."""
    out = [ctypes.c_int(0) for _ in range(5)]
    _check(load().xpress_describe_plan(
        _ptr(base), _ptr(bias), int(N), int(B), int(V), int(stride_base_r),
        int(stride_bias_r), *[ctypes.byref(o) for o in out]), "xpress_describe_plan")
    combine, splits, threads, vec, launches = [o.value for o in out]
    return {"combine": COMBINE_NAMES.get(combine, combine), "splits": splits,
            "block_threads": threads, "vector_path": bool(vec), "launches": launches}


def xpress_describe_gemm_plan(N: int, B: int, V: int) -> dict:
    """Launch shape of the readout with in-place bias for (N, B, V): waves
    per workgroup, vocabulary ranges, workgroups per range and 32-id tiles."""
    out = [ctypes.c_int(0) for _ in range(4)]
    _check(load().xpress_describe_gemm_plan(int(N), int(B), int(V),
                                            *[ctypes.byref(o) for o in out]),
           "xpress_describe_gemm_plan")
    waves, ranges, row_wgs, tiles = [o.value for o in out]
    return {"waves": waves, "ranges": ranges, "row_wgs": row_wgs, "tiles": tiles}


def xpress_bf16_add_round_table(a_vals, n_a: int, out, stream=None) -> None:
    """out[i*65536 + b] = bf16(a_vals[i] + b) on the GPU, for every pattern b."""
    _span(a_vals, int(n_a) * 2, "a_vals")
    _span(out, int(n_a) * 65536 * 2, "out")
    _check(load().xpress_bf16_add_round_table(_ptr(a_vals), int(n_a), _ptr(out),
                                              _stream(stream)),
           "xpress_bf16_add_round_table")


XPRESS_READ_ROWS = 0
XPRESS_READ_FLAT = 1


def xpress_read_probe(base, bias, rows: int, V: int, stride: int, mode: int, sink,
                      stream=None) -> None:
    """Plain streaming read of base and bias (no arithmetic): the read
    ceiling the readout is measured against.  mode XPRESS_READ_ROWS (one
    workgroup per row) or XPRESS_READ_FLAT (grid-stride sweep)."""
    if int(rows) > 0:
        _span(base, ((int(rows) - 1) * int(stride) + int(V)) * 2, "base")
        _span(bias, ((int(rows) - 1) * int(stride) + int(V)) * 2, "bias")
        _span(sink, 4, "sink")
    _check(load().xpress_read_probe(_ptr(base), _ptr(bias), int(rows), int(V), int(stride),
                                    int(mode), _ptr(sink), _stream(stream)),
           "xpress_read_probe")


# ---------------------------------------------------------------------------
# Serving operators.  The two over the paged cache take tensors only: sizes,
# strides and types come from them.  Tensors are on the current device.  Their C argument structs are 8-byte
# fields throughout, packed here in declaration order.
# ---------------------------------------------------------------------------

_KV_CACHE = "5Q11q"
_APPEND_ARGS = struct.Struct(_KV_CACHE + "7Q14q")
_ATTENTION_ARGS = struct.Struct(_KV_CACHE + "4Q5qd6q")
_torch = None
_marshal = None
_types = {}


def _import_torch():
    """torch, imported by the first call that takes tensors or a stream from it.
    (_torch is set last: another thread that sees it sees the rest.)"""
    global _torch
    if _torch is None:
        import torch
        _types.update({torch.bfloat16: XPRESS_BF16, torch.float16: XPRESS_FP16,
                       torch.float8_e4m3fn: XPRESS_E4M3})
        _torch = torch
    return _torch


def _use_torch():
    """torch, and the host module whose functions make a serving operator's call from
    tensors (None: the arguments are not what they should be, and the Python code
    after it says why).  The other entry points do without the module.  (_marshal is
    set after _torch, for other threads.)"""
    global _marshal
    torch = _import_torch()
    if _marshal is None:
        try:
            from . import _marshal as marshal
        except ImportError as e:
            raise ImportError("_marshal.so is not built for this torch; run `python -m "
                              "vocab_wide_add_amd.build`") from e
        _marshal = marshal
    return torch


def _dtype(t, what: str) -> int:
    try:
        return _types[t.dtype]
    except KeyError:
        raise ValueError("%s: bf16, fp16 or float8_e4m3fn expected, got %s" % (what, t.dtype)) from None


def _plain(t, what: str, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of the given type and shape on device
    dev (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s: a contiguous %s tensor of shape %s expected, got %s of shape %s"
                         % (what, dtype, tuple(shape), t.dtype, tuple(t.shape)))
    if t.get_device() != dev:
        _elsewhere(t, what, dev)
    return t.data_ptr()


def _elsewhere(t, what: str, dev: int):
    raise ValueError("%s: expected a tensor on %s, got one on %s"
                     % (what, "a GPU" if dev < 0 else "cuda:%d" % dev, t.device))


def _on_current(dev: int):
    """The library works on the current device, whose stream is taken too."""
    now = _torch._C._cuda_getDevice()
    if dev != now:
        raise ValueError("the tensors are on cuda:%d and the current device is cuda:%d; call this "
                         "under torch.cuda.device(%d)" % (dev, now, dev))


def _kv_cache(k_cache, v_cache, page_table, k_scale, v_scale, dev: int):
    """The fields of xpress_kv_cache from [pages, heads, page_size, dim] caches
    (any strides with unit stride along dim) on device dev and an int32
    [seqs, width] table."""
    shape, strides, dtype = k_cache.shape, k_cache.stride(), k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype is not dtype \
            or v_cache.stride() != strides:
        raise ValueError("k_cache, v_cache: [pages, heads, page_size, dim], one type, shape and "
                         "stride expected")
    pages, heads, size, dim = shape
    sp, sh, st, sd = strides
    if sd != 1 and dim > 1:
        raise ValueError("k_cache, v_cache: unit stride along dim expected")
    table, rows = page_table.shape, page_table.stride()
    if len(table) != 2 or page_table.dtype is not _torch.int32 or (table[1] > 1 and rows[1] != 1):
        raise ValueError("page_table: int32 [seqs, width] with unit stride along width expected")
    code = _dtype(k_cache, "k_cache")
    if dev < 0:
        _elsewhere(k_cache, "k_cache", dev)
    if v_cache.get_device() != dev:
        _elsewhere(v_cache, "v_cache", dev)
    if page_table.get_device() != dev:
        _elsewhere(page_table, "page_table", dev)
    _on_current(dev)
    f32 = _torch.float32
    return (k_cache.data_ptr(), v_cache.data_ptr(), _plain(k_scale, "k_scale", f32, (heads,), dev),
            _plain(v_scale, "v_scale", f32, (heads,), dev), page_table.data_ptr(), pages, size, heads,
            dim, sp, sh, st, code, table[0], table[1], rows[0])


def _rows(t, what: str, shape, dtype, dev: int):
    """(address, strides) of a tensor with unit stride along its last dimension
    and the given shape and type."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError("%s: shape %s and type %s expected, got %s of %s"
                         % (what, tuple(shape), dtype, tuple(t.shape), t.dtype))
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError("%s: unit stride along its last dimension expected" % what)
    if t.get_device() != dev:
        _elsewhere(t, what, dev)
    return t.data_ptr(), st


def xpress_kv_append(q, k, v, q_out, k_cache, v_cache, page_table, positions, cos_sin,
                     seq_of=None, k_scale=None, v_scale=None, interleaved: bool = False,
                     stream=None) -> None:
    """Rotate the keys of T new tokens to their positions and append them and
    their values to the paged cache; write the rotated queries to q_out.

    q, q_out [T, Hq, dim] (None, None: keys and values only), k, v [T, heads,
    dim] bf16 or fp16; k_cache, v_cache [pages, heads, page_size, dim] of that
    type or float8_e4m3fn (any strides, unit along dim); page_table int32
    [seqs, width]; positions int32 [T]; cos_sin fp32 [max_pos, rot_dim]
    (cosines, then sines; None: no rotation); seq_of int32 [T] (None: T / seqs
    tokens of each sequence in order); k_scale, v_scale fp32 [heads].  See the
    header for the definition.
    """
    lib = _lib or load()
    if _marshal is None:
        _use_torch()
    torch = _torch
    status = _marshal.kv_append(lib.append_at, _stream_of_tensors(stream), q, k, v, q_out, k_cache, v_cache, page_table,
                                positions, cos_sin, seq_of, k_scale, v_scale, interleaved)
    if status is not None:
        return _check(status, "xpress_kv_append")
    if (q is None) != (q_out is None):
        raise ValueError("q, q_out: both or neither expected")
    shape, dev = k.shape, k_cache.get_device()
    T, heads, dim = shape
    cache = _kv_cache(k_cache, v_cache, page_table, k_scale, v_scale, dev)
    if cache[7] != heads or cache[8] != dim:
        raise ValueError("k: [T, %d, %d] expected for this cache, got %s"
                         % (cache[7], cache[8], tuple(shape)))
    code, dtype, i32 = _dtype(k, "k"), k.dtype, torch.int32
    kp, (kt, kh, _) = _rows(k, "k", shape, dtype, dev)
    vp, (vt, vh, _) = _rows(v, "v", shape, dtype, dev)
    if q is None:
        hq, qp, qt, qh, op, ot, oh = 0, 0, 0, 0, 0, 0, 0
    else:
        hq = q.shape[1]
        qp, (qt, qh, _) = _rows(q, "q", (T, hq, dim), dtype, dev)
        op, (ot, oh, _) = _rows(q_out, "q_out", (T, hq, dim), dtype, dev)
    if cos_sin is None:
        cp, max_pos, rot = 0, 2 ** 31 - 1, 0
    else:
        max_pos, rot = cos_sin.shape
        cp = _plain(cos_sin, "cos_sin", torch.float32, (max_pos, rot), dev)
    args = _APPEND_ARGS.pack(
        *cache, qp, kp, vp, op, _plain(positions, "positions", i32, (T,), dev),
        _plain(seq_of, "seq_of", i32, (T,), dev), cp, T, hq, code, rot, max_pos,
        1 if interleaved else 0, qt, qh, kt, kh, vt, vh, ot, oh)
    _check(lib.xpress_kv_append(args, _stream(stream)), "xpress_kv_append")


def xpress_paged_attention(q, k_cache, v_cache, page_table, lens, out, max_len: int, lse=None,
                           scale: float = None, window: int = 0, k_scale=None, v_scale=None,
                           stream=None) -> None:
    """Attention of the Q newest tokens of each sequence over its paged cache.

    q, out [N, Q, Hq, dim] bf16 or fp16 (any strides, unit along dim); caches,
    page_table [N, width] and scales as for xpress_kv_append; lens int32 [N],
    the sequences' lengths with the new tokens; max_len, their upper bound;
    lse fp32 [N, Q, Hq] or None; scale, 1 / sqrt(dim) if None; window, the
    keys a query sees back from itself (0: all).  See the header for the
    definition.
    """
    lib = _lib or load()
    if _marshal is None:
        _use_torch()
    torch = _torch
    status = _marshal.paged_attention(lib.attention_at, _stream_of_tensors(stream), q, k_cache, v_cache, page_table, lens,
                                      out, lse, k_scale, v_scale, max_len, window, scale)
    if status is not None:
        return _check(status, "xpress_paged_attention")
    shape, dev = q.shape, k_cache.get_device()
    N, Q, hq, dim = shape
    cache = _kv_cache(k_cache, v_cache, page_table, k_scale, v_scale, dev)
    if cache[8] != dim or cache[13] != N:
        raise ValueError("q: [%d, Q, Hq, %d] expected for this cache and page table, got %s"
                         % (cache[13], cache[8], tuple(shape)))
    code, dtype = _dtype(q, "q"), q.dtype
    qp, (qn, qi, qh, _) = _rows(q, "q", shape, dtype, dev)
    op, (on, oi, oh, _) = _rows(out, "out", shape, dtype, dev)
    args = _ATTENTION_ARGS.pack(
        *cache, qp, op, _plain(lse, "lse", torch.float32, (N, Q, hq), dev),
        _plain(lens, "lens", torch.int32, (N,), dev), Q, hq, code, int(max_len), int(window),
        1.0 / math.sqrt(dim) if scale is None else float(scale), qn, qi, qh, on, oi, oh)
    _check(lib.xpress_paged_attention(args, _stream(stream)), "xpress_paged_attention")


def xpress_paged_attention_reserve(N: int, Q: int, Hq: int, heads: int, dim: int, max_len: int,
                                   window: int = 0, stream=None) -> None:
    _check(load().xpress_paged_attention_reserve(int(N), int(Q), int(Hq), int(heads), int(dim),
                                                 int(max_len), int(window), _stream(stream)),
           "xpress_paged_attention_reserve")


def xpress_paged_attention_plan(N: int, Q: int, Hq: int, heads: int, dim: int, max_len: int,
                                window: int = 0) -> dict:
    """The launch such a call would make (host only): keys of a part, parts of
    the longest sequence, rows of a workgroup, launches."""
    out = [ctypes.c_int(0) for _ in range(4)]
    _check(load().xpress_paged_attention_plan(int(N), int(Q), int(Hq), int(heads), int(dim),
                                              int(max_len), int(window),
                                              *[ctypes.byref(o) for o in out]),
           "xpress_paged_attention_plan")
    return dict(zip(("chunk", "splits", "rows", "launches"), [o.value for o in out]))


def _one_device(t, what: str, dev):
    if dev is not None and t.device != dev:
        raise ValueError("%s: expected a tensor on %s, as base is, got one on %s" % (what, dev, t.device))


def _logits(t, what: str, nbytes: int, dev):
    """Refuse a tensor that is not bf16 (or its bits in 16-bit integers) with unit
    stride along its last dimension, or that ends before nbytes (addresses are the
    caller's responsibility)."""
    if t is None or not hasattr(t, "data_ptr"):
        return
    if t.dtype not in (_torch.bfloat16, _torch.int16, _torch.uint16) \
            or (t.dim() > 0 and t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError("%s: bf16 with unit stride along its last dimension expected, got %s of strides %s"
                         % (what, t.dtype, t.stride()))
    _span(t, nbytes, what)
    _one_device(t, what, dev)


def _numbers(t, what: str, dtype, n: int, dev):
    """Refuse a tensor that is not n or more contiguous numbers of this type."""
    if t is None or not hasattr(t, "data_ptr"):
        return
    if t.dtype is not dtype or not t.is_contiguous() or t.numel() < n:
        raise ValueError("%s: a contiguous %s tensor of %d numbers expected, got %s of shape %s and strides %s"
                         % (what, dtype, n, t.dtype, tuple(t.shape), t.stride()))
    _one_device(t, what, dev)


def xpress_sample_to_blk(base, bias, blk, temperature, top_k, top_p, min_p, u, N: int, B: int,
                         V: int, stride_base_r: int, stride_bias_r: int = 0, prob=None,
                         stream=None) -> None:
    """blk[n, 1+b] = a token drawn from softmax(bf16(base + bias) / temperature)
    of row r = n*(B-1) + b, cut by top_k, top_p and min_p, with the uniform
    number u[r]; prob[r], its probability.  bias may be None.  base and bias
    bf16 (or its bits as 16-bit integers) with unit stride along a row, blk
    int64, top_k int32, temperature, top_p, min_p, u and prob fp32, one per row
    and contiguous, all on one device.  Integer addresses are taken as they are.
    """
    lib = _lib or load()
    if _marshal is None:
        _use_torch()
    status = _marshal.sample(lib.sample_at, _stream_of_tensors(stream), base, bias, blk, prob, temperature, top_k, top_p,
                             min_p, u, N, B, V, stride_base_r, stride_bias_r)
    if status is not None:
        return _check(status, "xpress_sample_to_blk")
    rows = int(N) * (int(B) - 1)
    if rows > 0:
        t, dev = _torch, base.device if hasattr(base, "data_ptr") else None
        _logits(base, "base", ((rows - 1) * int(stride_base_r) + int(V)) * 2, dev)
        if bias is not None:
            _logits(bias, "bias", ((rows - 1) * int(stride_bias_r) + int(V)) * 2, dev)
        _numbers(blk, "blk", t.int64, int(N) * int(B), dev)
        _numbers(top_k, "top_k", t.int32, rows, dev)
        for x, what in ((temperature, "temperature"), (top_p, "top_p"), (min_p, "min_p"), (u, "u"),
                        (prob, "prob")):
            _numbers(x, what, t.float32, rows, dev)
        if dev is not None and dev.type == "cuda":
            _on_current(dev.index)
    _check(load().xpress_sample_to_blk(_ptr(base), _ptr(bias), _ptr(blk), _ptr(prob),
                                       _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p),
                                       _ptr(u), int(N), int(B), int(V), int(stride_base_r),
                                       int(stride_bias_r), _stream(stream)),
           "xpress_sample_to_blk")


def xpress_sample_reserve(N: int, B: int, V: int, stream=None) -> None:
    """Grow the (device, stream) workspace to what xpress_sample_to_blk needs to
    spread few rows over the chip, as before a capture."""
    _check(load().xpress_sample_reserve(int(N), int(B), int(V), _stream(stream)),
           "xpress_sample_reserve")


def xpress_last_hip_error() -> int:
    return int(load().xpress_last_hip_error())


def xpress_error_string(status: int) -> str:
    return load().xpress_error_string(int(status)).decode()


def xpress_version() -> str:
    return load().xpress_version().decode()
