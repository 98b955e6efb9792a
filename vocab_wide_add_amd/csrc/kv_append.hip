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
// handful of tokens.

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
    uint32_t pages, page_size, seqs, width, per_seq;
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

// Any layout: one thread per (token, head slot, pair or single element).
template <bool FP16, bool E4M3, bool INTER>
__global__ void __launch_bounds__(kThreads) append_scalar_kernel(AppendArgs a)
{
    const uint32_t turned = a.half + (a.D - a.rot);  // work items of a rotated head
    const uint32_t items = (a.Hq + a.Hk) * turned + a.Hk * a.D;
    for (uint32_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        const Place p = place_of(a, t);
        for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < items;
             i += gridDim.x * kThreads) {
            uint32_t h, e0, e1;
            int which;  // 0 query, 1 key, 2 value
            bool pair = false;
            if (i < (a.Hq + a.Hk) * turned) {
                h = i / turned;
                const uint32_t j = i - h * turned;
                which = h < a.Hq ? 0 : 1;
                if (which) h -= a.Hq;
                pair = j < a.half;
                e0 = !pair ? a.rot + (j - a.half) : INTER ? 2 * j : j;
                e1 = !pair ? e0 : INTER ? 2 * j + 1 : j + a.half;
            } else {
                const uint32_t j = i - (a.Hq + a.Hk) * turned;
                h = j / a.D;
                e0 = e1 = j - h * a.D;
                which = 2;
            }
            if (which != 0 && p.at < 0) continue;
            const uint16_t* src = which == 0   ? a.q + t * a.q_t + h * a.q_h
                                  : which == 1 ? a.k + t * a.k_t + h * a.k_h
                                               : a.v + t * a.v_t + h * a.v_h;
            float y0 = widen<FP16>(src[e0]), y1 = widen<FP16>(src[e1]);
            if (pair && p.pos >= 0) {
                const float* cs = a.cos_sin + (int64_t)p.pos * a.rot;
                const uint32_t j = INTER ? e0 / 2 : e0;
                turn(y0, y1, cs[j], cs[a.half + j], &y0, &y1);
            }
            if (which == 0) {
                uint16_t* dst = a.q_out + t * a.o_t + h * a.o_h;
                dst[e0] = p.pos < 0 ? 0 : narrow<FP16>(y0);
                if (pair) dst[e1] = p.pos < 0 ? 0 : narrow<FP16>(y1);
                continue;
            }
            const int64_t at = p.at + h * a.head;
            if constexpr (E4M3) {
                const float* sp = which == 1 ? a.k_scale : a.v_scale;
                const float sc = sp ? sp[h] : 1.0f;
                uint8_t* dst = (uint8_t*)(which == 1 ? a.kc : a.vc) + at;
                dst[e0] = narrow8(y0 / sc);
                if (pair) dst[e1] = narrow8(y1 / sc);
            } else {
                uint16_t* dst = (uint16_t*)(which == 1 ? a.kc : a.vc) + at;
                dst[e0] = narrow<FP16>(y0);
                if (pair) dst[e1] = narrow<FP16>(y1);
            }
        }
    }
}

template <bool FP16, bool E4M3, bool INTER>
hipError_t launch_append(const AppendArgs& a, hipStream_t stream)
{
    const uint64_t items = (uint64_t)(a.Hq + a.Hk) * (a.half + a.D - a.rot) + (uint64_t)a.Hk * a.D;
    const uint32_t gx = (uint32_t)((items + kThreads - 1) / kThreads);
    const uint32_t gy = a.T < 65535u ? a.T : 65535u;
    hipLaunchKernelGGL((append_scalar_kernel<FP16, E4M3, INTER>), dim3(gx, gy), dim3(kThreads), 0,
                       stream, a);
    return hipGetLastError();
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
        // q_out on q is allowed as q itself only
        const bool same = x.q_out == x.q && x.stride_o_t == x.stride_q_t && x.stride_o_h == x.stride_q_h;
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

    const bool f16 = x.dtype == XPRESS_FP16, e8 = c.dtype == XPRESS_E4M3, in = x.interleaved != 0;
    hipError_t e;
    if (f16) {
        e = e8 ? (in ? launch_append<true, true, true>(a, stream)
                     : launch_append<true, true, false>(a, stream))
               : (in ? launch_append<true, false, true>(a, stream)
                     : launch_append<true, false, false>(a, stream));
    } else {
        e = e8 ? (in ? launch_append<false, true, true>(a, stream)
                     : launch_append<false, true, false>(a, stream))
               : (in ? launch_append<false, false, true>(a, stream)
                     : launch_append<false, false, false>(a, stream));
    }
    return e == hipSuccess ? XPRESS_OK : hip_fail(e);
}
