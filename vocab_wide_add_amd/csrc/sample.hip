// sample.hip -- the sampled readout (gfx950): one token per draft row, drawn
// with a given uniform number from softmax(bf16(base + bias) / temperature)
// cut by top-k, top-p and min-p.
//
// A logit is a bf16 value, so a row holds at most 65536 distinct ones, and
// everything the draw needs follows from how often each value occurs: the
// order is by value (then id), all three rules keep a prefix of it, and the
// masses are sums of count * exp((value - max) / temperature).  One pass over
// the row counts the values in LDS (exact, whatever the order of the atomics);
// the exponentials are then taken once per distinct value, in 64 bits; and
// the drawn token is the j-th id holding one known value, found by a second
// look at the row.  No sort, no prefix sum over the vocabulary.
//
// Bins.  Value bits h = (sign, 15 magnitude bits): the counts of +m and -m
// share LDS word m, the positive one in the low 16 bits.  128 KiB of LDS hold
// all 32768 words.  A 16-bit count overflows when more than 65535 logits of
// a row are equal; the words' total then falls short of the number counted,
// and the row is done again in two half-passes (positive, negative) of 32-bit
// counts.  Logits below -2^101 (-inf and the type's lowest value, the usual
// masks) are not counted at first: next to a maximum above -2^100, at a
// temperature below 2^90, their weight exp(-1024) is 0 in 64 bits; otherwise
// the half-passes run instead.
//
// The order's walk goes by 1024 segments of 64 values: positive magnitudes
// downwards, then negative ones upwards.  A wave takes a segment at a time,
// one value per lane.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "device_common.h"
#include "host_common.h"
#include "xpress_argmax.h"

namespace {

using namespace xpress;

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr uint32_t kWords = 32768;           // magnitudes
constexpr uint32_t kSegs = 1024;             // segments of 64 values, both signs
constexpr uint32_t kInf = 0x7F80u;           // magnitude bits of infinity
constexpr uint32_t kLow = 0x8000u | (0x7F80u - 27u * 128u);     // bits of -2^101
constexpr uint32_t kTopLow = 0x8000u | (0x7F80u - 28u * 128u);  // bits of -2^100

struct SampleArgs {
    const uint16_t *base, *bias;
    int64_t* blk;
    float* prob;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t* top_k;
    int64_t stride_base, stride_bias;
    uint32_t rows, bm1, V;
};

struct Shared {
    uint32_t bins[kWords];
    uint32_t count[kSegs];   // logits of a segment; then: of all segments before it
    double mass[kSegs];      // their mass; then: of all segments before it
    double mass_min[kWaves];
    double wave_mass[kWaves];
    uint32_t wave_count[kWaves];
    uint32_t wave_total[kWaves];
    uint32_t top;            // order position of the largest value counted
    uint32_t found;
    double f64;
    uint32_t counted;
};

__device__ __forceinline__ float value_of(uint32_t h) { return __uint_as_float(h << 16); }

// Value bits at position i of the descending order (i = 0: the largest
// positive magnitude 0x7FFF; 32767: +0; 32768: -0; 65535: magnitude 0x7FFF).
__device__ __forceinline__ uint32_t bits_at(uint32_t i) { return i < kWords ? kWords - 1 - i : i; }
__device__ __forceinline__ uint32_t order_of(uint32_t h) { return h < kWords ? kWords - 1 - h : h; }

// Eight summed logits of a row from element e on; bits past the row are NaN.
template <bool VEC, bool BIAS>
__device__ __forceinline__ u32x4 logits8(const uint16_t* base, const uint16_t* bias, uint32_t e,
                                         uint32_t V)
{
    u32x4 z;
    if (VEC && e + 8 <= V) {
        z = *reinterpret_cast<const u32x4*>(base + e);
        if constexpr (BIAS) {
            const u32x4 b = *reinterpret_cast<const u32x4*>(bias + e);
            for (int w = 0; w < 4; ++w) z[w] = add_round2(z[w], b[w]);
        }
        return z;
    }
    for (int w = 0; w < 4; ++w) {
        uint32_t two = 0;
        for (int s = 0; s < 2; ++s) {
            const uint32_t i = e + 2 * w + s;
            uint32_t h = 0xFFFFu;
            if (i < V) {
                h = base[i];
                if constexpr (BIAS) h = add_round2(h, bias[i]) & 0xFFFFu;
            }
            two |= h << (16 * s);
        }
        z[w] = two;
    }
    return z;
}

// What is counted: 0 both signs in 16-bit halves; 1 / 2 the positive / the
// negative logits in 32-bit words.
template <bool VEC, bool BIAS>
__device__ void count_row(Shared& s, const uint16_t* base, const uint16_t* bias, uint32_t V, int what)
{
    for (uint32_t i = threadIdx.x; i < kWords; i += kThreads) s.bins[i] = 0;
    __syncthreads();
    uint32_t mine = 0;
    for (uint32_t e = threadIdx.x * 8; e < V; e += kThreads * 8) {
        const u32x4 z = logits8<VEC, BIAS>(base, bias, e, V);
        for (int w = 0; w < 8; ++w) {
            const uint32_t h = w & 1 ? z[w / 2] >> 16 : z[w / 2] & 0xFFFFu;
            const uint32_t sign = h >> 15;
            if (what == 0) {
                if (h <= kLow) {
                    atomicAdd(&s.bins[h & 0x7FFFu], 1u + sign * 65535u);
                    ++mine;
                }
            } else if (sign == (uint32_t)(what - 1)) {
                atomicAdd(&s.bins[h & 0x7FFFu], 1u);
            }
        }
    }
    if (what == 0) {
        for (int m = 32; m; m >>= 1) mine += __shfl_xor(mine, m);
        if ((threadIdx.x & 63) == 0) s.wave_total[threadIdx.x / 64] = mine;
    }
    __syncthreads();
    // -0 counts as +0 (in the half-passes the two words are in different
    // passes; count_at puts them together)
    if (what == 0 && threadIdx.x == 0) s.bins[0] = (s.bins[0] & 0xFFFFu) + (s.bins[0] >> 16);
    __syncthreads();
}

// The draw of one row.
template <bool VEC, bool BIAS>
struct Row {
    Shared& s;
    const uint16_t *base, *bias;
    uint32_t V;
    int state;          // what the bins hold now (see count_row)
    bool halves;        // 32-bit half-passes
    uint32_t zeros;     // half-passes: the number of -0 and +0 logits
    uint32_t top;       // order position of the largest value
    double zmax, t;

    // Number of logits at order position i, whose sign's bins are loaded.
    __device__ uint32_t count_at(uint32_t i) const
    {
        const uint32_t h = bits_at(i), w = s.bins[h & 0x7FFFu];
        if (!halves) {
            if (h == 0) return w;
            if (h == 0x8000u) return 0;
            return i < kWords ? w & 0xFFFFu : w >> 16;
        }
        if (h == 0) return zeros;
        if (h == 0x8000u) return 0;
        return w;
    }

    __device__ void load_half(uint32_t i)
    {
        const int want = i < kWords ? 1 : 2;
        if (!halves || state == want) return;
        __syncthreads();
        count_row<VEC, BIAS>(s, base, bias, V, want);
        state = want;
    }

    __device__ double weight_at(uint32_t i) const
    {
        if (i == top) return 1.0;
        return exp(((double)value_of(bits_at(i)) - zmax) / t);
    }

    // Whether order position i may be drawn: a value below or at the top, not
    // NaN, not -inf.
    __device__ bool real(uint32_t i) const
    {
        const uint32_t h = bits_at(i);
        return i >= top && (h & 0x7FFFu) <= kInf && h != (0x8000u | kInf);
    }

    // The wave's lanes look at one segment: its count and mass, in order,
    // inclusive up to each lane.
    __device__ void segment(uint32_t seg, uint32_t* n, double* w, uint32_t* n_to, double* m_to) const
    {
        const uint32_t i = seg * 64 + (threadIdx.x & 63);
        *n = real(i) ? count_at(i) : 0;
        *w = *n ? weight_at(i) : 0.0;
        uint32_t c = *n;
        double m = (double)*n * *w;
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t c2 = __shfl_up(c, d);
            const double m2 = __shfl_up(m, d);
            if ((int)(threadIdx.x & 63) >= d) {
                c += c2;
                m += m2;
            }
        }
        *n_to = c;
        *m_to = m;
    }
};

__device__ __forceinline__ double wave_sum(double v)
{
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

template <bool VEC, bool BIAS>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a)
{
    __shared__ Shared s;
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid / 64;

    for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float temp = a.temperature[r];
        const bool greedy = !(temp > 0.0f);
        Row<VEC, BIAS> row{s, a.base + (int64_t)r * a.stride_base,
                           BIAS ? a.bias + (int64_t)r * a.stride_bias : nullptr, a.V, 0, false, 0, 0,
                           0.0, greedy ? 1.0 : (double)temp};

        // 1. count, and find the largest value
        count_row<VEC, BIAS>(s, row.base, row.bias, a.V, 0);
        uint32_t total = 0, top = 65536u, sum = 0;
        for (uint32_t w = 0; w < kWaves; ++w) total += s.wave_total[w];
        for (uint32_t i = tid; i < kWords; i += kThreads) {
            const uint32_t b = s.bins[i];
            sum += (b & 0xFFFFu) + (b >> 16);
            if (i <= kInf) {
                if (i == 0 ? b != 0 : (b & 0xFFFFu) != 0) top = min(top, order_of(i));
                if (i != 0 && i != kInf && (b >> 16)) top = min(top, order_of(0x8000u | i));
            }
        }
        for (int m = 32; m; m >>= 1) {
            sum += __shfl_xor(sum, m);
            top = min(top, __shfl_xor(top, m));
        }
        if (lane == 0) {
            s.wave_count[wave] = sum;
            s.count[wave] = top;
        }
        __syncthreads();
        sum = 0;
        top = 65536u;
        for (uint32_t w = 0; w < kWaves; ++w) {
            sum += s.wave_count[w];
            top = min(top, s.count[w]);
        }
        __syncthreads();
        const bool again = sum != total || top >= order_of(kTopLow) || !(row.t < 0x1p90);
        if (again) {
            row.halves = true;
            uint32_t best = 65536u;
            for (int half = 1; half <= 2; ++half) {
                count_row<VEC, BIAS>(s, row.base, row.bias, a.V, half);
                row.zeros += s.bins[0];
                for (uint32_t i = tid; i < kWords; i += kThreads) {
                    if (s.bins[i] == 0) continue;
                    const uint32_t h = half == 1 ? i : 0x8000u | i;
                    if (i == 0) best = min(best, order_of(0));
                    else if (i < kInf || (i == kInf && half == 1)) best = min(best, order_of(h));
                }
                __syncthreads();
            }
            row.state = 2;
            for (int m = 32; m; m >>= 1) best = min(best, __shfl_xor(best, m));
            if (lane == 0) s.count[wave] = best;
            __syncthreads();
            top = 65536u;
            for (uint32_t w = 0; w < kWaves; ++w) top = min(top, s.count[w]);
            __syncthreads();
        }
        const uint32_t n_blk = r / a.bm1;
        int64_t* dst = a.blk + (r + n_blk + 1);
        if (top >= 65536u) {  // nothing but NaN and -inf
            if (tid == 0) {
                *dst = 0;
                if (a.prob) a.prob[r] = 0.0f;
            }
            __syncthreads();
            continue;
        }
        row.top = top;
        row.zmax = (double)value_of(bits_at(top));

        uint32_t key = top, nth = 0;  // the drawn value, and which of its ids
        double p_drawn = 1.0;
        if (!greedy) {
            // 2. counts and masses of the segments, and the mass that min-p keeps
            const float min_p = a.min_p[r], top_p = a.top_p[r];
            const bool by_min = min_p > 0.0f;
            double kept_min = 0.0;
            for (uint32_t seg0 = 0; seg0 < kSegs; seg0 += kWaves) {
                if (row.halves && (seg0 == 0 || seg0 == kSegs / 2)) row.load_half(seg0 * 64);
                const uint32_t seg = seg0 + wave, i = seg * 64 + lane;
                const uint32_t n = row.real(i) ? row.count_at(i) : 0;
                uint32_t c = 0;
                double m = 0.0;
                if (__any(n != 0)) {
                    const double w = n ? row.weight_at(i) : 0.0;
                    m = (double)n * w;
                    if (w >= (double)min_p) kept_min += m;
                    m = wave_sum(m);
                    c = n;
                    for (int d = 32; d; d >>= 1) c += __shfl_xor(c, d);
                }
                if (lane == 0) {
                    s.count[seg] = c;
                    s.mass[seg] = m;
                }
            }
            kept_min = wave_sum(kept_min);
            if (lane == 0) s.mass_min[wave] = kept_min;
            __syncthreads();
            // 3. exclusive prefix over the segments, one per thread
            const uint32_t c_own = s.count[tid];
            const double m_own = s.mass[tid];
            uint32_t c = c_own;
            double m = m_own;
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t c2 = __shfl_up(c, d);
                const double m2 = __shfl_up(m, d);
                if ((int)lane >= d) {
                    c += c2;
                    m += m2;
                }
            }
            if (lane == 63) {
                s.wave_count[wave] = c;
                s.wave_mass[wave] = m;
            }
            __syncthreads();
            uint32_t c_before = 0, c_all = 0;
            double m_before = 0.0, m_all = 0.0, m_min = 0.0;
            for (uint32_t w = 0; w < kWaves; ++w) {
                if (w == wave) {
                    c_before = c_all;
                    m_before = m_all;
                }
                c_all += s.wave_count[w];
                m_all += s.wave_mass[w];
                m_min += s.mass_min[w];
            }
            c_before += c - c_own;
            m_before += m - m_own;
            s.count[tid] = c_before;
            s.mass[tid] = m_before;
            __syncthreads();
            // 4. the kept mass: the least of the rules' (each keeps a prefix)
            const int32_t k = a.top_k[r];
            double z_mass = m_all;
            if (k > 0 && (uint32_t)k < c_all) {
                // the segment in which the k-th id lies
                if (c_own && c_before < (uint32_t)k && (uint32_t)k <= c_before + c_own) s.found = tid;
                __syncthreads();
                const uint32_t seg = s.found;
                row.load_half(seg * 64);
                if (wave == 0) {
                    uint32_t n, n_to;
                    double w, m_to;
                    row.segment(seg, &n, &w, &n_to, &m_to);
                    const uint32_t need = (uint32_t)k - s.count[seg];  // ids of this segment kept
                    if (n && n_to - n < need && need <= n_to) {
                        s.f64 = s.mass[seg] + (m_to - (double)n * w) + (double)(need - (n_to - n)) * w;
                    }
                }
                __syncthreads();
                z_mass = s.f64;
                __syncthreads();
            }
            double kept = z_mass;
            if (top_p < 1.0f) {
                const double goal = (double)top_p * z_mass;
                // the segment holding the last id before which less than goal has gathered
                if (tid == 0) s.found = top / 64;
                __syncthreads();
                if (c_own && m_before < goal) atomicMax(&s.found, tid);
                __syncthreads();
                const uint32_t seg = s.found;
                row.load_half(seg * 64);
                if (wave == 0) {
                    uint32_t n, n_to;
                    double w, m_to;
                    row.segment(seg, &n, &w, &n_to, &m_to);
                    const double before = s.mass[seg] + (m_to - (double)n * w);
                    double got = 0.0;
                    if (n && before < goal) {
                        double j = w > 0.0 ? ceil((goal - before) / w) : (double)n;
                        j = j < 1.0 ? 1.0 : j > (double)n ? (double)n : j;
                        got = before + j * w;
                    }
                    for (int d = 32; d; d >>= 1) got = fmax(got, __shfl_xor(got, d));
                    if (lane == 0) s.f64 = got;
                }
                __syncthreads();
                kept = fmin(kept, s.f64);
                __syncthreads();
            }
            if (by_min) kept = fmin(kept, m_min);
            kept = fmax(kept, 1.0);  // the first id's weight
            // 5. the first id at which the mass passes u * kept
            float u = a.u[r];
            u = u > 0.0f ? u : 0.0f;
            u = u < 1.0f ? u : 0x1.fffffep-1f;
            const double goal = (double)u * kept;
            if (tid == 0) s.found = top / 64;
            __syncthreads();
            if (c_own && m_own > 0.0 && m_before <= goal) atomicMax(&s.found, tid);
            __syncthreads();
            const uint32_t seg = s.found;
            row.load_half(seg * 64);
            if (wave == 0) {
                uint32_t n, n_to;
                double w, m_to;
                row.segment(seg, &n, &w, &n_to, &m_to);
                const double before = s.mass[seg] + (m_to - (double)n * w);
                const uint64_t may = __ballot(n && w > 0.0 && before <= goal);
                // the segment's first value where rounding leaves none
                const uint64_t any = __ballot(n && w > 0.0);
                const int at = may ? 63 - __clzll(may) : __ffsll((unsigned long long)any) - 1;
                if ((int)lane == at) {
                    double j = floor((goal - before) / w);
                    j = j < 0.0 ? 0.0 : j > (double)(n - 1) ? (double)(n - 1) : j;
                    s.found = seg * 64 + lane;
                    s.counted = (uint32_t)j;
                    s.f64 = w / kept;
                }
            }
            __syncthreads();
            key = s.found;
            nth = s.counted;
            p_drawn = s.f64;
            __syncthreads();
        }

        // 6. the nth id (in id order) that holds the drawn value: each wave
        //    counts its share of the row, then the share with the id is walked
        const uint32_t want = bits_at(key);
        const bool zero = want == 0;
        const uint32_t steps = (a.V + kWaves * 512 - 1) / (kWaves * 512);  // of 512 logits per wave
        auto matches = [&](u32x4 z) {
            uint32_t m = 0;
            for (int w = 0; w < 8; ++w) {
                const uint32_t h = w & 1 ? z[w / 2] >> 16 : z[w / 2] & 0xFFFFu;
                m |= (uint32_t)(h == want || (zero && h == 0x8000u)) << w;
            }
            return m;
        };
        uint32_t mine = 0;
        for (uint32_t i = 0; i < steps; ++i) {
            const uint32_t e = (wave * steps + i) * 512 + lane * 8;
            if (e < a.V) mine += __popc(matches(logits8<VEC, BIAS>(row.base, row.bias, e, a.V)));
        }
        for (int m = 32; m; m >>= 1) mine += __shfl_xor(mine, m);
        if (lane == 0) s.wave_count[wave] = mine;
        __syncthreads();
        uint32_t before = 0;
        for (uint32_t w = 0; w < wave; ++w) before += s.wave_count[w];
        if (before <= nth && nth < before + mine) {
            uint32_t left = nth - before;
            for (uint32_t i = 0; i < steps; ++i) {
                const uint32_t e = (wave * steps + i) * 512 + lane * 8;
                const uint32_t m = e < a.V ? matches(logits8<VEC, BIAS>(row.base, row.bias, e, a.V)) : 0;
                const uint32_t n = __popc(m);
                uint32_t to = n;
                for (int d = 1; d < 64; d <<= 1) {
                    const uint32_t o = __shfl_up(to, d);
                    if ((int)lane >= d) to += o;
                }
                const uint32_t all = __shfl(to, 63);
                if (left < all) {
                    if (to - n <= left && left < to) {
                        uint32_t bits = m;
                        for (uint32_t k = left - (to - n); k; --k) bits &= bits - 1;
                        *dst = (int64_t)(e + (uint32_t)__ffs(bits) - 1u);
                        if (a.prob) a.prob[r] = (float)p_drawn;
                    }
                    break;
                }
                left -= all;
            }
        }
        __syncthreads();
    }
}

template <bool VEC, bool BIAS>
hipError_t launch_sample(const SampleArgs& a, hipStream_t stream)
{
    const uint32_t grid = a.rows < 65536u ? a.rows : 65536u;
    hipLaunchKernelGGL((sample_kernel<VEC, BIAS>), dim3(grid), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

extern "C" int xpress_sample_to_blk(const uint16_t* base, const uint16_t* bias, int64_t* blk,
                                    float* prob, const float* temperature, const int32_t* top_k,
                                    const float* top_p, const float* min_p, const float* u,
                                    int64_t N, int64_t B, int64_t V, int64_t stride_base_r,
                                    int64_t stride_bias_r, hipStream_t stream)
{
    if (N < 0 || B < 1 || V < 1 || V > 0x7FFFFFFFll || stride_base_r < V ||
        (bias && stride_bias_r < V)) {
        return XPRESS_EINVAL;
    }
    if (B - 1 > 0 && N > INT64_MAX / (B - 1)) return XPRESS_EINVAL;
    const int64_t rows = N * (B - 1);
    if (rows == 0) return XPRESS_OK;
    if (rows > 0x7FFFFFFFll || N > 0x7FFFFFFFll / B) return XPRESS_EINVAL;
    if (!base || !blk || !temperature || !top_k || !top_p || !min_p || !u) return XPRESS_EINVAL;
    const struct { const void* p; uintptr_t n; } aligned[] = {
        {base, 2}, {bias, 2}, {blk, 8}, {prob, 4}, {temperature, 4}, {top_k, 4}, {top_p, 4},
        {min_p, 4}, {u, 4}};
    for (const auto& x : aligned) {
        if (reinterpret_cast<uintptr_t>(x.p) % x.n != 0) return XPRESS_EINVAL;
    }
    if ((rows - 1) > (INT64_MAX / 8 - V) / stride_base_r ||
        (bias && (rows - 1) > (INT64_MAX / 8 - V) / stride_bias_r)) {
        return XPRESS_EINVAL;
    }
    const size_t base_bytes = (size_t)((rows - 1) * stride_base_r + V) * 2u;
    const size_t bias_bytes = bias ? (size_t)((rows - 1) * stride_bias_r + V) * 2u : 0;
    const size_t blk_bytes = (size_t)(N * B) * 8u, row_bytes = (size_t)rows * 4u;
    const struct { const void* p; size_t n; } reads[] = {
        {base, base_bytes}, {bias, bias_bytes}, {temperature, row_bytes}, {top_k, row_bytes},
        {top_p, row_bytes}, {min_p, row_bytes}, {u, row_bytes}};
    for (const auto& x : reads) {
        if (x.p && (xpress::ranges_overlap(blk, blk_bytes, x.p, x.n) ||
                    (prob && xpress::ranges_overlap(prob, row_bytes, x.p, x.n)))) {
            return XPRESS_EINVAL;
        }
    }
    if (prob && xpress::ranges_overlap(prob, row_bytes, blk, blk_bytes)) return XPRESS_EINVAL;

    SampleArgs a;
    a.base = base;
    a.bias = bias;
    a.blk = blk;
    a.prob = prob;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.u = u;
    a.stride_base = stride_base_r;
    a.stride_bias = bias ? stride_bias_r : 0;
    a.rows = (uint32_t)rows;
    a.bm1 = (uint32_t)(B - 1);
    a.V = (uint32_t)V;
    const bool vec = xpress::is_aligned16(base) && (rows == 1 || stride_base_r % 8 == 0) &&
                     (!bias || (xpress::is_aligned16(bias) && (rows == 1 || stride_bias_r % 8 == 0)));
    hipError_t e;
    if (vec) {
        e = bias ? launch_sample<true, true>(a, stream) : launch_sample<true, false>(a, stream);
    } else {
        e = bias ? launch_sample<false, true>(a, stream) : launch_sample<false, false>(a, stream);
    }
    return e == hipSuccess ? XPRESS_OK : xpress::hip_fail(e);
}
