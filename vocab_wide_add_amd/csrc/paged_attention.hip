// paged_attention.hip -- attention of the newest tokens of every sequence
// over a paged key-value cache (gfx950).
//
// Simple form: one workgroup per (sequence, query, head).  Keys go by in
// tiles of one per thread; the running maximum and sum of the softmax are
// carried in fp32 from tile to tile, and each thread accumulates one output
// element.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "device_common.h"
#include "host_common.h"
#include "kv_common.h"
#include "xpress_argmax.h"

namespace {

using namespace xpress;

constexpr int kThreads = 256;

struct AttnArgs {
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    const int32_t *lens, *page_table;
    const void *kc, *vc;
    const float *k_scale, *v_scale;
    int64_t q_n, q_i, q_h, o_n, o_i, o_h;
    int64_t page, head, token, table;
    uint32_t N, Q, Hq, Hk, G, D, pages, page_size;
    int32_t max_len, window;
    float scale;
};

template <bool FP16>
__device__ __forceinline__ float widen(uint16_t h)
{
    if constexpr (FP16) return (float)__builtin_bit_cast(_Float16, h);
    return __uint_as_float((uint32_t)h << 16);
}

template <bool FP16, bool E4M3>
__device__ __forceinline__ float element(const void* p, int64_t at)
{
    if constexpr (E4M3) return __builtin_amdgcn_cvt_f32_fp8(((const uint8_t*)p)[at], 0);
    return widen<FP16>(((const uint16_t*)p)[at]);
}

__device__ __forceinline__ float block_reduce(float v, bool sum, float* tmp)
{
    for (int m = 32; m; m >>= 1) {
        const float o = __shfl_xor(v, m);
        v = sum ? v + o : fmaxf(v, o);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x / 64] = v;
    __syncthreads();
    v = tmp[0];
    for (int w = 1; w < kThreads / 64; ++w) v = sum ? v + tmp[w] : fmaxf(v, tmp[w]);
    return v;
}

template <bool FP16, bool E4M3>
__global__ void __launch_bounds__(kThreads) attention_simple_kernel(AttnArgs a)
{
    __shared__ float sq[256], sp[kThreads], tmp[4];
    __shared__ int64_t so[kThreads];
    const uint32_t row = blockIdx.x;
    const uint32_t h = row % a.Hq, i = row / a.Hq % a.Q, n = row / a.Hq / a.Q;
    const uint32_t hk = h / a.G, tid = threadIdx.x;
    int32_t len = a.lens[n];
    len = len < 0 ? 0 : len > a.max_len ? a.max_len : len;
    const int32_t pos = len - (int32_t)a.Q + (int32_t)i;
    const int32_t lo = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
    if (tid < a.D) sq[tid] = widen<FP16>(a.q[n * a.q_n + i * a.q_i + h * a.q_h + tid]);
    const float ks = a.scale * (a.k_scale ? a.k_scale[hk] : 1.0f);
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int32_t j0 = lo; j0 <= pos; j0 += kThreads) {
        __syncthreads();
        const int32_t j = j0 + (int32_t)tid;
        int64_t at = -1;
        if (j <= pos) {
            const uint32_t slot = (uint32_t)j / a.page_size;
            const uint32_t page = (uint32_t)a.page_table[(int64_t)n * a.table + slot];
            if (page < a.pages) {
                at = (int64_t)page * a.page + (int64_t)((uint32_t)j - slot * a.page_size) * a.token +
                     (int64_t)hk * a.head;
            }
        }
        float s = -INFINITY;
        if (at >= 0) {
            s = 0.0f;
            for (uint32_t d = 0; d < a.D; ++d) s += sq[d] * element<FP16, E4M3>(a.kc, at + d);
            s *= ks;
        }
        const float mt = fmaxf(m, block_reduce(s, false, tmp));
        const float base = mt == -INFINITY ? 0.0f : mt;
        const float p = at >= 0 ? expf(s - base) : 0.0f;
        sp[tid] = p;
        so[tid] = at;
        const float f = m == -INFINITY ? 0.0f : expf(m - base);
        l = l * f + block_reduce(p, true, tmp);
        m = mt;
        if (tid < a.D) {
            o *= f;
            for (int32_t t = 0; t < kThreads && j0 + t <= pos; ++t) {
                if (so[t] >= 0) o += sp[t] * element<FP16, E4M3>(a.vc, so[t] + tid);
            }
        }
    }
    if (tid < a.D) {
        float y = l == 0.0f ? 0.0f : o / l * (a.v_scale ? a.v_scale[hk] : 1.0f);
        a.out[n * a.o_n + i * a.o_i + h * a.o_h + tid] =
            FP16 ? __builtin_bit_cast(uint16_t, (_Float16)y) : __builtin_bit_cast(uint16_t, (__bf16)y);
    }
    if (tid == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : m + logf(l);
}

struct Shape {
    int64_t N, Q, Hq, heads, dim, max_len, window;
};

bool shape_ok(const Shape& s)
{
    const int64_t most = 0x7FFFFFFFll;
    return s.N >= 0 && s.N <= most && s.Q >= 0 && s.Q <= most && s.heads >= 1 && s.Hq >= 1 &&
           s.Hq <= 65536 && s.Hq % s.heads == 0 && s.dim >= 8 && s.dim <= 256 && s.dim % 8 == 0 &&
           s.max_len >= 1 && s.max_len <= most && s.window >= 0 && s.window <= most &&
           (s.N == 0 || s.Q == 0 || s.Q <= most / s.Hq / s.N);
}

}  // namespace

extern "C" {

int xpress_paged_attention(const xpress_paged_attention_args* args, hipStream_t stream)
{
    if (!args) return XPRESS_EINVAL;
    const xpress_paged_attention_args& x = *args;
    const xpress_kv_cache& c = x.cache;
    const Shape s = {c.seqs, x.Q, x.Hq, c.heads, c.dim, x.max_len, x.window};
    if (!shape_ok(s)) return XPRESS_EINVAL;
    if (x.dtype != XPRESS_BF16 && x.dtype != XPRESS_FP16) return XPRESS_EINVAL;
    if (s.N == 0 || s.Q == 0) return XPRESS_OK;
    size_t cache_bytes = 0;
    if (!cache_ok(c, &cache_bytes)) return XPRESS_EINVAL;
    if (c.dtype != x.dtype && c.dtype != XPRESS_E4M3) return XPRESS_EINVAL;
    const int64_t e = element_bytes(c.dtype);
    if (c.dim * e % 16 != 0 || !is_aligned16(c.k) || !is_aligned16(c.v) ||
        c.stride_page * e % 16 != 0 || c.stride_head * e % 16 != 0 || c.stride_token * e % 16 != 0) {
        return XPRESS_EINVAL;
    }
    if (x.max_len > c.table_width * c.page_size || !isfinite(x.scale) || !isfinite((float)x.scale)) {
        return XPRESS_EINVAL;
    }
    if (!x.q || !x.out || !x.lens || !is_aligned(x.q, 2) || !is_aligned(x.out, 2) ||
        !is_aligned(x.lens, 4) || !is_aligned(x.lse, 4)) {
        return XPRESS_EINVAL;
    }
    if (x.stride_q_n < 0 || x.stride_q_i < 0 || x.stride_q_h < 0 || x.stride_o_n < 0 ||
        x.stride_o_i < 0 || x.stride_o_h < 0) {
        return XPRESS_EINVAL;
    }
    const Dim dq[3] = {{s.N, x.stride_q_n}, {s.Q, x.stride_q_i}, {s.Hq, x.stride_q_h}};
    Dim d_o[3] = {{s.N, x.stride_o_n}, {s.Q, x.stride_o_i}, {s.Hq, x.stride_o_h}};
    const int64_t nq = span_of(dq, s.dim), no = span_of(d_o, s.dim);
    if (nq < 0 || no < 0 || !is_disjoint(d_o, s.dim)) return XPRESS_EINVAL;
    const size_t bq = (size_t)nq * 2u, bo = (size_t)no * 2u;
    const size_t bl = (size_t)(s.N * s.Q * s.Hq) * 4u, bn = (size_t)s.N * 4u;
    const size_t bt = (size_t)((s.N - 1) * c.stride_table + c.table_width) * 4u;
    const struct { const void* p; size_t n; } reads[] = {{x.q, bq}, {x.lens, bn}, {c.page_table, bt}};
    for (const auto& r : reads) {
        if (ranges_overlap(x.out, bo, r.p, r.n) || (x.lse && ranges_overlap(x.lse, bl, r.p, r.n))) {
            return XPRESS_EINVAL;
        }
    }
    if (!apart_from_cache(c, cache_bytes, x.out, bo) || !apart_from_cache(c, cache_bytes, x.lse, bl) ||
        (x.lse && ranges_overlap(x.lse, bl, x.out, bo))) {
        return XPRESS_EINVAL;
    }

    AttnArgs a;
    a.q = (const uint16_t*)x.q;
    a.out = (uint16_t*)x.out;
    a.lse = x.lse;
    a.lens = x.lens;
    a.page_table = c.page_table;
    a.kc = c.k;
    a.vc = c.v;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.q_n = x.stride_q_n;
    a.q_i = x.stride_q_i;
    a.q_h = x.stride_q_h;
    a.o_n = x.stride_o_n;
    a.o_i = x.stride_o_i;
    a.o_h = x.stride_o_h;
    a.page = c.stride_page;
    a.head = c.stride_head;
    a.token = c.stride_token;
    a.table = c.stride_table;
    a.N = (uint32_t)s.N;
    a.Q = (uint32_t)s.Q;
    a.Hq = (uint32_t)s.Hq;
    a.Hk = (uint32_t)s.heads;
    a.G = (uint32_t)(s.Hq / s.heads);
    a.D = (uint32_t)s.dim;
    a.pages = (uint32_t)c.pages;
    a.page_size = (uint32_t)c.page_size;
    a.max_len = (int32_t)x.max_len;
    a.window = (int32_t)x.window;
    a.scale = (float)x.scale;
    const dim3 grid((uint32_t)(s.N * s.Q * s.Hq));
    const bool f16 = x.dtype == XPRESS_FP16, e8 = c.dtype == XPRESS_E4M3;
    if (f16 && e8) {
        hipLaunchKernelGGL((attention_simple_kernel<true, true>), grid, dim3(kThreads), 0, stream, a);
    } else if (f16) {
        hipLaunchKernelGGL((attention_simple_kernel<true, false>), grid, dim3(kThreads), 0, stream, a);
    } else if (e8) {
        hipLaunchKernelGGL((attention_simple_kernel<false, true>), grid, dim3(kThreads), 0, stream, a);
    } else {
        hipLaunchKernelGGL((attention_simple_kernel<false, false>), grid, dim3(kThreads), 0, stream, a);
    }
    const hipError_t err = hipGetLastError();
    return err == hipSuccess ? XPRESS_OK : hip_fail(err);
}

int xpress_paged_attention_reserve(int64_t N, int64_t Q, int64_t Hq, int64_t heads, int64_t dim,
                                   int64_t max_len, int64_t window, hipStream_t stream)
{
    const Shape s = {N, Q, Hq, heads, dim, max_len, window};
    (void)stream;
    return shape_ok(s) ? XPRESS_OK : XPRESS_EINVAL;
}

int xpress_paged_attention_plan(int64_t N, int64_t Q, int64_t Hq, int64_t heads, int64_t dim,
                                int64_t max_len, int64_t window, int* chunk, int* splits, int* rows,
                                int* launches)
{
    const Shape s = {N, Q, Hq, heads, dim, max_len, window};
    if (!shape_ok(s)) return XPRESS_EINVAL;
    if (chunk) *chunk = (int)max_len;
    if (splits) *splits = 1;
    if (rows) *rows = 1;
    if (launches) *launches = (N == 0 || Q == 0) ? 0 : 1;
    return XPRESS_OK;
}

}  // extern "C"
