// kv_append.hip -- append of new keys and values to a paged cache, with the
// position rotation of keys and queries applied on the way (gfx950).
//
// For every token: rot(q) -> q_out, rot(k) / k_scale -> K page, v / v_scale ->
// V page, where rot turns the pairs (x[a_i], x[b_i]) by the angle whose cosine
// and sine stand in the token's row of cos_sin.  Each product and the sum is
// rounded in fp32 (no contraction into a fused multiply-add), so the value
// before the one rounding to the stored type is the same on every path.
//
// A pure stream: every element is read once and written once, a few flops
// each, so the bound is memory bandwidth for prompts and the chain of
// dependent loads (position -> table entry, cos_sin row -> store) for a
// handful of tokens.  A workgroup's threads belong to one token, so position,
// page and angles are loaded once per workgroup and come from the caches after.
// Measured (bf16, 32 query and 8 key-value heads of 128): 20011 tokens 98 us,
// 5.1 TB/s of reads and writes, the rate of a large copy (561 us with a thread
// per pair and 2-byte accesses); the same with rows that allow accesses of 4
// elements 113 us, of one 240, by the number of requests; 512 tokens into e4m3
// 5.6 us; one token 3.0 us.

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "device_common.h"
#include "host_common.h"
#include "kv_common.h"
#include "xpress_argmax.h"

namespace {

using namespace xpress;

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.0f;

struct AppendArgs {
    const uint16_t *q, *k, *v;
    uint16_t* q_out;
    void *kc, *vc;
    const float *k_scale, *v_scale;
    const int32_t *positions, *seq_of, *page_table;
    const float* cos_sin;
    int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;
    int64_t page, head, token, table;  // cache strides, page table row stride
    uint32_t T, Hq, Hk, D, half, rot;
    uint32_t pages, page_size, seqs, width, per_seq, pieces;
    int32_t max_pos;
};

// Where a token goes.
struct Place {
    int32_t pos;      // < 0: padding
    int64_t at;       // offset of its place in head 0 of the caches; < 0: not stored
};

__device__ __forceinline__ Place place_of(const AppendArgs& a, uint32_t t)
{
    Place p;
    p.pos = a.positions[t];
    p.at = -1;
    const uint32_t n = a.seq_of ? (uint32_t)a.seq_of[t] : t / a.per_seq;
    const uint32_t slot = (uint32_t)p.pos / a.page_size;  // a negative position is past any table
    if (p.pos < 0 || p.pos >= a.max_pos || n >= a.seqs || slot >= a.width) {
        p.pos = -1;
        return p;
    }
    const uint32_t page = (uint32_t)a.page_table[(int64_t)n * a.table + slot];
    if (page < a.pages) {
        p.at = (int64_t)page * a.page +
               (int64_t)((uint32_t)p.pos - slot * a.page_size) * a.token;
    }
    return p;
}

template <bool FP16>
__device__ __forceinline__ float widen(uint16_t h)
{
    if constexpr (FP16) return (float)__builtin_bit_cast(_Float16, h);
    return __uint_as_float((uint32_t)h << 16);
}

template <bool FP16>
__device__ __forceinline__ uint16_t narrow(float x)
{
    if constexpr (FP16) return __builtin_bit_cast(uint16_t, (_Float16)x);
    return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// Saturating conversion to the 8-bit type (NaN stays NaN).
__device__ __forceinline__ float saturate(float x)
{
    const float lo = x < -kE4m3Max ? -kE4m3Max : x;
    return lo > kE4m3Max ? kE4m3Max : lo;
}

__device__ __forceinline__ uint8_t narrow8(float x)
{
    return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(saturate(x), 0.0f, 0, false);
}

__device__ __forceinline__ void turn(float a, float b, float c, float s, float* ya, float* yb)
{
#pragma clang fp contract(off)
    const float ac = a * c, bs = b * s, bc = b * c, as = a * s;
    *ya = ac - bs;
    *yb = bc + as;
}

// One token's work is cut into pieces of 2 W elements of a head: for a rotated
// part W elements and their W partners, elsewhere 2 W elements in a row (a
// head's last piece may end after W).  Either way piece j of a head starts at
// element 2 W j, or W j where the partners lie rot / 2 away.  W is 8 where all
// rows start on 16 bytes, 4 on 8 bytes, else 1: a choice of the width of the
// loads and stores alone, the arithmetic is the same.
template <int W, typename E>
struct alignas(W * sizeof(E)) Row {
    E e[W];
};

template <bool FP16, bool E4M3, bool INTER, int W>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a)
{
    using Half = Row<W, uint16_t>;
    using Eight = Row<W, uint8_t>;
    using Real = Row<W < 4 ? W : 4, float>;
    const uint32_t items = (a.Hq + 2 * a.Hk) * a.pieces, step = gridDim.x * blockDim.x;
    const uint32_t i0 = blockIdx.x * blockDim.x + threadIdx.x;
    const uint32_t h0 = i0 / a.pieces, j0 = i0 - h0 * a.pieces;
    const uint32_t dh = step / a.pieces, dj = step - dh * a.pieces;
    for (uint32_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        const Place p = place_of(a, t);
        const float* cs = a.cos_sin + (int64_t)p.pos * a.rot;
        uint32_t h = h0, j = j0;
        for (uint32_t i = i0; i < items; i += step, h += dh, j += dj) {
            if (j >= a.pieces) {
                j -= a.pieces;
                ++h;
            }
            const int which = h < a.Hq ? 0 : h < a.Hq + a.Hk ? 1 : 2;  // query, key, value
            if (which != 0 && p.at < 0) continue;
            const uint32_t head = which == 0 ? h : which == 1 ? h - a.Hq : h - a.Hq - a.Hk;
            const uint16_t* src = which == 0   ? a.q + t * a.q_t + head * a.q_h
                                  : which == 1 ? a.k + t * a.k_t + head * a.k_h
                                               : a.v + t * a.v_t + head * a.v_h;
            const bool pairs = which != 2 && j * (2 * W) < a.rot;
            const uint32_t e0 = pairs && !INTER ? j * W : j * (2 * W);
            const uint32_t e1 = pairs && !INTER ? e0 + a.half : e0 + W;
            const bool two = e1 < a.D;
            const Half x0 = *reinterpret_cast<const Half*>(src + e0);
            const Half x1 = *reinterpret_cast<const Half*>(src + (two ? e1 : e0));
            float y[2 * W];
#pragma unroll
            for (int e = 0; e < W; ++e) {
                y[e] = widen<FP16>(x0.e[e]);
                y[W + e] = widen<FP16>(x1.e[e]);
            }
            if (pairs && p.pos >= 0) {
                constexpr int R = W < 4 ? W : 4;
#pragma unroll
                for (int f = 0; f < W / R; ++f) {
                    const Real c = *reinterpret_cast<const Real*>(cs + j * W + f * R);
                    const Real s = *reinterpret_cast<const Real*>(cs + a.half + j * W + f * R);
#pragma unroll
                    for (int e = 0; e < R; ++e) {
                        const int at = f * R + e;
                        if constexpr (INTER) {
                            turn(y[2 * at], y[2 * at + 1], c.e[e], s.e[e], &y[2 * at], &y[2 * at + 1]);
                        } else {
                            turn(y[at], y[W + at], c.e[e], s.e[e], &y[at], &y[W + at]);
                        }
                    }
                }
            }
            if (E4M3 && which != 0) {
                const float* sp = which == 1 ? a.k_scale : a.v_scale;
                const float sc = sp ? sp[head] : 1.0f;
                Eight z0, z1;
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    z0.e[e] = narrow8(y[e] / sc);
                    z1.e[e] = narrow8(y[W + e] / sc);
                }
                uint8_t* dst = (uint8_t*)(which == 1 ? a.kc : a.vc) + p.at + head * a.head;
                *reinterpret_cast<Eight*>(dst + e0) = z0;
                if (two) *reinterpret_cast<Eight*>(dst + e1) = z1;
                continue;
            }
            const bool blank = p.pos < 0;  // a query's: the others were left above
            Half z0, z1;
#pragma unroll
            for (int e = 0; e < W; ++e) {
                z0.e[e] = blank ? 0 : narrow<FP16>(y[e]);
                z1.e[e] = blank ? 0 : narrow<FP16>(y[W + e]);
            }
            uint16_t* dst = which == 0 ? a.q_out + t * a.o_t + head * a.o_h
                                       : (uint16_t*)(which == 1 ? a.kc : a.vc) + p.at + head * a.head;
            *reinterpret_cast<Half*>(dst + e0) = z0;
            if (two) *reinterpret_cast<Half*>(dst + e1) = z1;
        }
    }
}

// A thread per piece while that fills at most half of the chip's thread slots
// (512 tokens of 384 pieces into e4m3: 5.0 us, 5.8 with a workgroup a token);
// beyond, one workgroup a token, each thread taking items / kThreads pieces (1000
// such tokens: 7.5 us, 8.0 with a thread per piece; 8000: 44 and 52).
constexpr uint64_t kSlots = 1u << 18;  // of 256 compute units of 2048 threads

template <bool FP16, bool E4M3, bool INTER, int W>
hipError_t launch_pieces(const AppendArgs& a, hipStream_t stream)
{
    const uint32_t items = (a.Hq + 2 * a.Hk) * a.pieces;
    const uint32_t rounds = (items + kThreads - 1) / kThreads;
    const bool few = (uint64_t)a.T * items <= kSlots;
    const uint32_t threads = ((items + rounds - 1) / rounds + 63) / 64 * 64;
    const uint32_t gy = a.T < 65535u ? a.T : 65535u;
    hipLaunchKernelGGL((append_kernel<FP16, E4M3, INTER, W>), dim3(few ? rounds : 1, gy), dim3(threads),
                       0, stream, a);
    return hipGetLastError();
}

template <bool FP16, bool E4M3, bool INTER>
hipError_t launch_append(AppendArgs a, int width, hipStream_t stream)
{
    a.pieces = (a.D + 2 * width - 1) / (2 * width);
    if (width == 8) return launch_pieces<FP16, E4M3, INTER, 8>(a, stream);
    if (width == 4) return launch_pieces<FP16, E4M3, INTER, 4>(a, stream);
    return launch_pieces<FP16, E4M3, INTER, 1>(a, stream);
}

bool input_ok(const void* p, int64_t T, int64_t H, int64_t D, int64_t st, int64_t sh, size_t* bytes)
{
    if (!p || !is_aligned(p, 2) || st < 0 || sh < 0) return false;
    const Dim d[2] = {{T, st}, {H, sh}};
    const int64_t span = span_of(d, D);
    *bytes = (size_t)(span < 0 ? 0 : span) * 2u;
    return span > 0;
}

}  // namespace

extern "C" int xpress_kv_append(const xpress_kv_append_args* args, hipStream_t stream)
{
    if (!args) return XPRESS_EINVAL;
    const xpress_kv_append_args& x = *args;
    const xpress_kv_cache& c = x.cache;
    const int64_t most = 0x7FFFFFFFll;
    if (x.T < 0 || x.T > most || x.Hq < 0 || x.Hq > 65536) return XPRESS_EINVAL;
    if (x.dtype != XPRESS_BF16 && x.dtype != XPRESS_FP16) return XPRESS_EINVAL;
    if (x.T == 0) return XPRESS_OK;
    size_t cache_bytes = 0;
    if (!cache_ok(c, &cache_bytes)) return XPRESS_EINVAL;
    if (c.dtype != x.dtype && c.dtype != XPRESS_E4M3) return XPRESS_EINVAL;
    if (x.rot_dim < 0 || x.rot_dim > c.dim || x.rot_dim % 2 != 0) return XPRESS_EINVAL;
    if (x.max_pos < 1 || x.max_pos > most) return XPRESS_EINVAL;
    if (x.rot_dim > 0 && (!x.cos_sin || !is_aligned(x.cos_sin, 4))) return XPRESS_EINVAL;
    if (!x.positions || !is_aligned(x.positions, 4) || !is_aligned(x.seq_of, 4)) return XPRESS_EINVAL;
    if (!x.seq_of && (c.seqs < 1 || x.T % c.seqs != 0)) return XPRESS_EINVAL;
    // work items of one token in 32 bits
    if ((x.Hq + 2 * c.heads) * c.dim > most) return XPRESS_EINVAL;

    size_t nq = 0, nk = 0, nv = 0, no = 0;
    if (!input_ok(x.k, x.T, c.heads, c.dim, x.stride_k_t, x.stride_k_h, &nk) ||
        !input_ok(x.v, x.T, c.heads, c.dim, x.stride_v_t, x.stride_v_h, &nv)) {
        return XPRESS_EINVAL;
    }
    if (x.Hq > 0) {
        if (!input_ok(x.q, x.T, x.Hq, c.dim, x.stride_q_t, x.stride_q_h, &nq) ||
            !input_ok(x.q_out, x.T, x.Hq, c.dim, x.stride_o_t, x.stride_o_h, &no)) {
            return XPRESS_EINVAL;
        }
        Dim d[2] = {{x.T, x.stride_o_t}, {x.Hq, x.stride_o_h}};
        if (!is_disjoint(d, c.dim)) return XPRESS_EINVAL;
        // q_out on q is allowed as q itself only (one token's or one head's stride
        // addresses nothing)
        const bool same = x.q_out == x.q && (x.T == 1 || x.stride_o_t == x.stride_q_t) &&
                          (x.Hq == 1 || x.stride_o_h == x.stride_q_h);
        if (!same && ranges_overlap(x.q, nq, x.q_out, no)) return XPRESS_EINVAL;
    }
    if (!apart_from_cache(c, cache_bytes, x.k, nk) || !apart_from_cache(c, cache_bytes, x.v, nv) ||
        (x.Hq > 0 && (!apart_from_cache(c, cache_bytes, x.q, nq) ||
                      !apart_from_cache(c, cache_bytes, x.q_out, no))) ||
        !apart_from_cache(c, cache_bytes, x.positions, (size_t)x.T * 4u) ||
        !apart_from_cache(c, cache_bytes, x.seq_of, (size_t)x.T * 4u) ||
        !apart_from_cache(c, cache_bytes, c.page_table,
                          c.seqs ? (size_t)((c.seqs - 1) * c.stride_table + c.table_width) * 4u : 0)) {
        return XPRESS_EINVAL;
    }

    AppendArgs a;
    a.q = (const uint16_t*)x.q;
    a.k = (const uint16_t*)x.k;
    a.v = (const uint16_t*)x.v;
    a.q_out = (uint16_t*)x.q_out;
    a.kc = c.k;
    a.vc = c.v;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.positions = x.positions;
    a.seq_of = x.seq_of;
    a.page_table = c.page_table;
    a.cos_sin = x.cos_sin;
    a.q_t = x.stride_q_t;
    a.q_h = x.stride_q_h;
    a.k_t = x.stride_k_t;
    a.k_h = x.stride_k_h;
    a.v_t = x.stride_v_t;
    a.v_h = x.stride_v_h;
    a.o_t = x.stride_o_t;
    a.o_h = x.stride_o_h;
    a.page = c.stride_page;
    a.head = c.stride_head;
    a.token = c.stride_token;
    a.table = c.stride_table;
    a.T = (uint32_t)x.T;
    a.Hq = (uint32_t)x.Hq;
    a.Hk = (uint32_t)c.heads;
    a.D = (uint32_t)c.dim;
    a.rot = (uint32_t)x.rot_dim;
    a.half = a.rot / 2;
    a.pages = (uint32_t)c.pages;
    a.page_size = (uint32_t)c.page_size;
    a.seqs = (uint32_t)c.seqs;
    a.width = (uint32_t)c.table_width;
    a.per_seq = x.seq_of ? 1u : (uint32_t)(x.T / c.seqs);
    a.max_pos = (int32_t)x.max_pos;

    // the widest access that every row's start and the rotated part allow
    int width = 1;
    for (int w : {8, 4}) {
        const int64_t of_cache = c.stride_page | c.stride_head | c.stride_token;
        const int64_t of_rows = x.stride_k_t | x.stride_k_h | x.stride_v_t | x.stride_v_h |
                                (x.Hq ? x.stride_q_t | x.stride_q_h | x.stride_o_t | x.stride_o_h : 0);
        const size_t bytes = (size_t)w * 2u, cache_w = (size_t)(w * element_bytes(c.dtype));
        if (c.dim % w == 0 && x.rot_dim % (2 * w) == 0 && (of_cache | of_rows) % w == 0 &&
            is_aligned(x.k, bytes) && is_aligned(x.v, bytes) &&
            (!x.Hq || (is_aligned(x.q, bytes) && is_aligned(x.q_out, bytes))) &&
            is_aligned(c.k, cache_w) && is_aligned(c.v, cache_w) && is_aligned(x.cos_sin, 16)) {
            width = w;
            break;
        }
    }
    const bool f16 = x.dtype == XPRESS_FP16, e8 = c.dtype == XPRESS_E4M3, in = x.interleaved != 0;
    hipError_t e;
    if (f16) {
        e = e8 ? (in ? launch_append<true, true, true>(a, width, stream)
                     : launch_append<true, true, false>(a, width, stream))
               : (in ? launch_append<true, false, true>(a, width, stream)
                     : launch_append<true, false, false>(a, width, stream));
    } else {
        e = e8 ? (in ? launch_append<false, true, true>(a, width, stream)
                     : launch_append<false, true, false>(a, width, stream))
               : (in ? launch_append<false, false, true>(a, width, stream)
                     : launch_append<false, false, false>(a, width, stream));
    }
    return e == hipSuccess ? XPRESS_OK : hip_fail(e);
}
