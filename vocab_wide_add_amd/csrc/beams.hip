// beams.hip -- beam search's selection (gfx950): of all continuations of a sequence's
// beams, the K with the largest score, and the gather of the chosen beams' states.
//
//     z_v = bf16(base[r, v] + bias[r, v])
//     score(r, v) = scores[r] + z_v - log sum_v' exp(z_v')
//
// One pass over a row gives both its sum of exponentials and its K largest logits; a
// second launch joins the rows of a sequence.  Rows are cut into parts where there
// are too few of them for the chip, and where a part's list of runs would not fit LDS.
//
// The sum.  exp(z - m) = 2^(z L - r) with L = log2(e), r an integer near the thread's
// largest z L.  L = Lh + Ll, Lh of 15 bits: z is a bf16 of 8 bits, so z Lh is exact in
// fp32, and the rest is a factor 1 + (z - m) Ll ln 2, summed beside: sum y and sum y z, of
// which the second enters once, in 64 bits.  The eight terms of a vector are added in fp32,
// pair by pair, and the eights in 64 bits (all of a thread's 256 in fp32: 4e-6 off for
// rows of equal logits, 1.3e-5 for a long tail behind one large logit; each term in 64
// bits and every argument exact: 76 us for 480 rows where this takes 68).  A sum is off, relatively, by
// less than 6e-7, usually 3e-8: 2^-23 by the hardware's 2^x; 2^-22 by the rounding of z Lh - r,
// which is below 8 in magnitude but for logits that together are .6 of the thread's sum at most,
// and there below 16; 3 2^-24 by the pairs; 2^-25 by the rest.  Threads' sums meet
// as 64-bit numbers, with powers of two as factors.  Where a part's largest |z| is
// 2^13 or more, neighbouring bf16 values are 32 or more apart, and the sum is the count
// of the largest.
//
// The K largest.  The largest of every eight logits, a run, goes to LDS as the row goes
// by.  The K-th largest of the threads' maxima, T0, is below K logits; runs above it
// are few, and where they are K or more the K-th largest of theirs is T.  The runs
// above T, and the first K in order that reach T, are read again; their logits not
// below T are ranked by counting.  Ties cost no more than anything else.
//
// Bound by the bytes for many rows; by the two launches and the chain of one workgroup
// for few.  Measured (V = 152064, K = 8): 480 rows of 60 sequences with a bias 57 us for
// the parts, 5.1 TB/s, and 10 for the join, most of it the logs and the lists' loads, each
// waited for; 4 rows of one 8.3 and 7.6.  Their states (256 tokens and 4096 hidden values
// a row) 5 and 3.0.  Whole calls for the 480 rows without a bias 52, by instructions a logit,
// and in rows that are not on 16 bytes, whose logits are loaded one by one, 189 with a bias
// and 128 without.  Two vectors of a thread on their way in place of four: 71 us for the
// 68 of the whole; six 72; shorter parts 69.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <memory>
#include <new>

#include "device_common.h"
#include "host_common.h"
#include "kv_common.h"
#include "xpress_argmax.h"

namespace {

using namespace xpress;

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kThreads = 512;
constexpr uint32_t kWaves = kThreads / 64;
constexpr uint32_t kRuns = 16384;          // of a part: 131072 logits
constexpr uint32_t kMostK = 128;
constexpr uint32_t kAbove = 4096;          // runs above T0: fewer than K threads', 32 each
constexpr uint32_t kFound = 2304;          // logits that are ranked
constexpr uint32_t kFew = 512;             // runs of the common case
constexpr uint32_t kAhead = 4;             // vectors that a thread has on their way
constexpr float kLh = 0x1.7154p+0f;        // log2(e) to 15 bits
constexpr double kRest = 1.4426950408889634074 - 0x1.7154p+0;
constexpr double kLn2 = 0.69314718055994530942;
constexpr float kFarMost = 1048576.0f;
constexpr float kLarge = 8192.0f;

struct BeamArgs {
    const uint16_t *base, *bias;
    const float* scores;
    float* best;
    int32_t* rows_out;
    int64_t* ids;
    int64_t stride_base, stride_bias;
    uint32_t V, K, beams, rows, parts, part_vecs;   // vectors of 8 logits
    uint32_t first;      // of the launch's units
    uint64_t* lists;     // [rows, parts, K]: keys in descending order, 0 where there is none
    double* sums;        // [rows, parts]: sum of exp(z - m), m the list's first
};

// A logit's place in the order, 16 bits: larger is better, 0 none.  (-0 is +0.)
__device__ __forceinline__ uint32_t order_of(float z)
{
    uint32_t h = __float_as_uint(z) >> 16;
    h = h == 0x8000u ? 0 : h;
    const uint32_t o = h & 0x8000u ? ~h & 0xFFFFu : h | 0x8000u;
    return z > -INFINITY ? o : 0;   // NaN and -inf: none
}

__device__ __forceinline__ float value_at(uint32_t o)
{
    return __uint_as_float((o & 0x8000u ? o & 0x7FFFu : ~o & 0xFFFFu) << 16);
}

template <bool VEC, bool BIAS>
struct Row {
    const uint16_t *base, *bias;
    uint32_t V;

    // Logits e .. e + 7 in pairs; bits past the row are NaN.
    __device__ __forceinline__ u32x4 at(uint32_t e) const
    {
        u32x4 z;
        if (VEC && e + 8 <= V) {
            z = *reinterpret_cast<const u32x4*>(base + e);
            if constexpr (BIAS) {
                const u32x4 b = *reinterpret_cast<const u32x4*>(bias + e);
#pragma unroll
                for (int w = 0; w < 4; ++w) z[w] = add_round2(z[w], b[w]);
            }
            return z;
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t two = 0;
#pragma unroll
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
};

// A thread's sum: sum 2^(z Lh - r) and the same times z.
struct Sum {
    double y = 0.0, yz = 0.0;
    float r = -kFarMost;

    __device__ __forceinline__ void add(const float* z, float top)
    {
        if (top * kLh > r + 8.0f) {   // (not for +inf past the first time: r is bounded)
            const float to = fminf(rintf(top * kLh), kFarMost);
            if (to > r) {
                y = ldexp(y, (int)(r - to));
                yz = ldexp(yz, (int)(r - to));
                r = to;
            }
        }
        float e[8], ez = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // no infinity: 0 times it would be NaN (a NaN logit becomes -3e38 too)
            const float x = fmaxf(z[i], -3e38f);
            e[i] = __builtin_amdgcn_exp2f(fmaf(x, kLh, -r));
            ez = fmaf(e[i], x, ez);
        }
        y += (double)(((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7])));
        yz += (double)ez;
    }
};

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    return v;
}

struct PartShared {
    __align__(16) uint16_t runs[kRuns];
    uint16_t above[kAbove];
    __align__(16) uint64_t found[kFound];
    uint32_t maxima[kThreads];
    uint32_t firsts[kMostK];
    uint32_t counts[kWaves];
    double part[kWaves];
    uint32_t n_above, n_found, threshold, n_runs, counted;
};

// Sum of v over the threads before this one; *total over all.
__device__ __forceinline__ uint32_t ranks(uint32_t v, uint32_t* sums, uint32_t* total)
{
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    uint32_t x = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t y = __shfl_up(x, d);
        if (lane >= (uint32_t)d) x += y;
    }
    __syncthreads();
    if (lane == 63) sums[wave] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) {
        const uint32_t s = sums[w];
        before += w < wave ? s : 0;
        all += s;
    }
    *total = all;
    return before + x - v;
}

__device__ __forceinline__ uint32_t wave_most(uint32_t v)
{
    v = max(v, dpp_u32<0xB1>(v));   // lane ^ 1, ^ 2, the other quad of 8, the other 8 of 16
    v = max(v, dpp_u32<0x4E>(v));
    v = max(v, dpp_u32<0x141>(v));
    v = max(v, dpp_u32<0x140>(v));
    v = max(v, (uint32_t)__shfl_xor(v, 16));
    return max(v, (uint32_t)__shfl_xor(v, 32));
}

// Adds the logits of a run that are not below `low` to the found ones.
template <typename R>
__device__ __forceinline__ void take_run(PartShared& s, const R& z, uint32_t e, uint32_t low)
{
    const u32x4 v = z.at(e);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        const uint32_t o = order_of(x & 1 ? bf16_hi(v[x / 2]) : bf16_lo(v[x / 2]));
        if (o > 0 && o >= low) {
            const uint32_t to = atomicAdd(&s.n_found, 1u);
            if (to < kFound) s.found[to] = (uint64_t)o << 32 | (kNoIndex - (e + x));
        }
    }
}

// The K largest logits of a part, by the largest of its runs: see the top of the file.
// Whatever the values are; the common case does without most of it.
template <typename R>
__device__ void find_any(PartShared& s, const R& z, uint32_t vec0, uint32_t vecs, uint32_t K, uint32_t best)
{
    const uint32_t tid = threadIdx.x;
    __syncthreads();
    s.maxima[tid] = best;
    if (tid == 0) s.n_above = s.n_found = s.threshold = 0;
    __syncthreads();
    // T0: the largest value that fewer than K of the threads' maxima pass, but K or
    // more reach
    uint32_t better = 0, equal = 0;
    for (uint32_t i = 0; i < kThreads; ++i) {
        better += s.maxima[i] > best;
        equal += s.maxima[i] == best;
    }
    if (better < K && better + equal >= K) s.threshold = best;
    __syncthreads();
    uint32_t low = s.threshold;   // 0: fewer than K threads have a logit
    const uint32_t span = (vecs + kThreads - 1) / kThreads;   // runs of a thread, one after the other
    const uint32_t run0 = min(tid * span, vecs), run1 = min(run0 + span, vecs);
    for (uint32_t i = run0; i < run1; ++i) {
        // fewer than K threads' runs: fewer than kAbove
        if (s.runs[i] > low) s.above[atomicAdd(&s.n_above, 1u) % kAbove] = (uint16_t)i;
    }
    __syncthreads();
    const uint32_t n0 = s.n_above;
    __syncthreads();
    if (n0 >= K) {
        // T: the K-th largest of these runs
        for (uint32_t i = tid; i < n0; i += kThreads) {
            const uint32_t o = s.runs[s.above[i]];
            uint32_t more = 0, same = 0;
            for (uint32_t j = 0; j < n0; ++j) {
                const uint32_t p = s.runs[s.above[j]];
                more += p > o;
                same += p == o;
            }
            if (more < K && more + same >= K) s.threshold = o;
        }
        __syncthreads();
        low = s.threshold;
    }
    // the first K runs, in order, whose largest is T
    uint32_t reach = 0;
    for (uint32_t i = run0; i < run1; ++i) reach += low > 0 && s.runs[i] == low;
    uint32_t reached;
    uint32_t at = ranks(reach, s.counts, &reached);
    for (uint32_t i = run0; i < run1 && at < K; ++i) {
        if (low > 0 && s.runs[i] == low) s.firsts[at++] = i;
    }
    __syncthreads();
    reached = min(reached, K);
    for (uint32_t i = tid; i < n0 + reached; i += kThreads) {
        const uint32_t run = i < n0 ? s.above[i] : s.firsts[i - n0];
        if (i >= n0 || s.runs[run] > low) take_run(s, z, (vec0 + run) * 8, low);
    }
    __syncthreads();
}

// The same where few runs come into question (false: they do not, nothing is done).
// T0 from the waves instead of the threads: the least of the waves' q-th largest, q =
// K / waves, is below K runs too, and costs q rounds over a wave.
template <typename R>
__device__ bool find_few(PartShared& s, const R& z, uint32_t vec0, uint32_t vecs, uint32_t K, uint32_t best)
{
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
    const uint32_t waves = min(kWaves, (vecs + 63) / 64), q = (K + waves - 1) / waves;
    uint32_t key = best << 6 | lane, least = 0;
    for (uint32_t i = 0; i < min(q, 64u); ++i) {
        const uint32_t m = wave_most(key);
        key = key == m ? 0 : key;
        least = m >> 6;
    }
    if (lane == 0) s.counts[wave] = q > 64 ? 0 : least;
    __syncthreads();   // and the runs are all there
    uint32_t low = s.counts[0];
    for (uint32_t w = 1; w < waves; ++w) low = min(low, s.counts[w]);
    low = max(low, 1u);
    const uint32_t words = (vecs + 7) / 8;
    for (uint32_t i = tid; i < words; i += kThreads) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(&s.runs[i * 8]);
        u16x2 top = {0, 0};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t two = v[w];   // (a bit cast of a vector's element takes its first one)
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, two));
        }
        if (max((uint32_t)top.x, (uint32_t)top.y) < low) continue;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            if ((x & 1 ? v[x / 2] >> 16 : v[x / 2] & 0xFFFFu) >= low) {
                const uint32_t at = atomicAdd(&s.n_above, 1u);
                if (at < kFew) s.above[at] = (uint16_t)(i * 8 + x);
            }
        }
    }
    __syncthreads();
    const uint32_t n0 = s.n_above;
    if (n0 > kFew) return false;
    uint32_t runs = n0;
    if (n0 > K) {
        for (uint32_t i = tid; i < n0; i += kThreads) {
            const uint32_t o = s.runs[s.above[i]];
            uint32_t more = 0, same = 0;
            for (uint32_t j = 0; j < n0; ++j) {
                const uint32_t p = s.runs[s.above[j]];
                more += p > o;
                same += p == o;
            }
            if (more < K && more + same >= K) {
                s.threshold = o;
                s.n_runs = more + same;
            }
        }
        __syncthreads();
        low = s.threshold;
        runs = s.n_runs;
    }
    if (runs > kFound / 8) return false;
    for (uint32_t i = tid; i < n0; i += kThreads) {
        const uint32_t run = s.above[i];
        if (s.runs[run] >= low) take_run(s, z, (vec0 + run) * 8, low);
    }
    __syncthreads();
    return true;
}

template <bool VEC, bool BIAS>
__global__ void __launch_bounds__(kThreads, 4) part_kernel(BeamArgs a)
{
    __shared__ PartShared s;
    const uint32_t unit = a.first + blockIdx.x, tid = threadIdx.x;
    const uint32_t row = unit / a.parts, part = unit - row * a.parts;
    const Row<VEC, BIAS> z = {a.base + row * a.stride_base, BIAS ? a.bias + row * a.stride_bias : nullptr, a.V};
    const uint32_t all_vecs = (a.V + 7) / 8, vec0 = part * a.part_vecs;
    const uint32_t vecs = min(a.part_vecs, all_vecs - vec0);
    if (tid == 0) s.n_above = s.n_found = s.counted = 0;
    if (tid < 8) s.runs[min(vecs + tid, kRuns - 1)] = 0;   // the last word of runs; a run there comes after
    __syncthreads();

    Sum sum;
    uint32_t best = 0;   // the thread's largest, in the order
    auto go = [&](const u32x4& v, uint32_t i) {
        float x[8], top = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            x[2 * w] = bf16_lo(v[w]);
            x[2 * w + 1] = bf16_hi(v[w]);
            top = fmaxf(top, fmaxf(x[2 * w], x[2 * w + 1]));
        }
        sum.add(x, top);
        const uint32_t o = order_of(top);
        s.runs[i] = (uint16_t)o;
        best = max(best, o);
    };
    if constexpr (VEC) {
        // whole vectors, kAhead of a thread at once and as many on their way
        const uint32_t whole = min(vecs, a.V / 8 - min(a.V / 8, vec0));
        u32x4 b[kAhead], c[kAhead];
        auto load = [&](uint32_t i0) {
#pragma unroll
            for (uint32_t u = 0; u < kAhead; ++u) {
                const uint32_t i = min(i0 + u * kThreads + tid, whole - 1);
                b[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(z.base + (vec0 + i) * 8));
                if constexpr (BIAS) {
                    c[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(z.bias + (vec0 + i) * 8));
                }
            }
        };
        if (whole > 0) {
            load(0);
            for (uint32_t i0 = 0; i0 < whole; i0 += kAhead * kThreads) {
                u32x4 v[kAhead];
#pragma unroll
                for (uint32_t u = 0; u < kAhead; ++u) {
                    v[u] = b[u];
                    if constexpr (BIAS) {
#pragma unroll
                        for (int w = 0; w < 4; ++w) v[u][w] = add_round2(v[u][w], c[u][w]);
                    }
                }
                if (i0 + kAhead * kThreads < whole) load(i0 + kAhead * kThreads);
#pragma unroll
                for (uint32_t u = 0; u < kAhead; ++u) {
                    const uint32_t i = i0 + u * kThreads + tid;
                    if (i < whole) go(v[u], i);
                }
            }
        }
        if (whole < vecs && tid == 0) go(z.at((vec0 + whole) * 8), whole);   // the row's end
    } else {
        for (uint32_t i = tid; i < vecs; i += kThreads) go(z.at((vec0 + i) * 8), i);
    }

    uint32_t most = wave_most(best);
    if ((tid & 63) == 0) s.maxima[tid / 64] = most;
    if (!find_few(s, z, vec0, vecs, a.K, best)) {
        for (uint32_t w = 0; w < kWaves; ++w) most = max(most, s.maxima[w]);
        find_any(s, z, vec0, vecs, a.K, best);
    } else {
        for (uint32_t w = 0; w < kWaves; ++w) most = max(most, s.maxima[w]);
    }
    const uint32_t n = min(s.n_found, kFound);
    uint64_t* list = a.lists + (int64_t)unit * a.K;
    for (uint32_t i = tid; i < n; i += kThreads) {
        const uint64_t key = s.found[i];
        uint32_t rank = 0;
        for (uint32_t j = 0; j < n; ++j) rank += s.found[j] > key;
        if (rank < a.K) list[rank] = key;
    }
    for (uint32_t i = n + tid; i < a.K; i += kThreads) list[i] = 0;

    // the sum, from the part's largest
    const float m = most ? value_at(most) : 0.0f;
    double total;
    if (most == 0) {
        total = 0.0;
    } else if (fabsf(m) >= kLarge) {
        uint32_t count = 0;
        for (uint32_t i = tid; i < vecs; i += kThreads) {
            if (s.runs[i] != most) continue;
            const u32x4 v = z.at((vec0 + i) * 8);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                count += (x & 1 ? bf16_hi(v[x / 2]) : bf16_lo(v[x / 2])) == m;
            }
        }
        atomicAdd(&s.counted, count);
        __syncthreads();
        total = (double)s.counted;
    } else {
        // 2^(z Lh - r) against 2^(m Lh - R): R the integer next to m Lh
        const double R = rint((double)m * (double)kLh);
        double v = sum.y + kRest * kLn2 * (sum.yz - (double)m * sum.y);
        v = best ? ldexp(v, (int)((double)sum.r - R)) : 0.0;
        v = wave_sum(v);
        if ((tid & 63) == 0) s.part[tid / 64] = v;
        __syncthreads();
        total = 0.0;
        for (uint32_t w = 0; w < kWaves; ++w) total += s.part[w];
        // sum 2^(z Lh - R) (1 + (z - m) Ll ln 2) to sum exp(z - m)
        total *= exp2(R - (double)m * (double)kLh);
    }
    if (tid == 0) a.sums[unit] = total;
}

constexpr uint32_t kJoinThreads = 256;
constexpr uint32_t kRanked = 512;    // candidates, and lists, that are ranked by counting
constexpr uint32_t kDirect = 32;     // candidates that are all ranked

// A candidate of the join: larger first.  rest: the beam, reversed, in 16 bits, over the
// 48 of the list's key; 0: none.
struct Candidate {
    double score;
    uint64_t rest;

    __device__ __forceinline__ bool before(const Candidate& o) const
    {
        return score > o.score || (score == o.score && rest > o.rest);
    }
};

struct Beams {
    const BeamArgs& a;
    const double *shift, *top;   // of a beam: its score less the log of its sum, and its largest
    uint32_t n;

    __device__ __forceinline__ Candidate of(uint32_t list, uint64_t key) const
    {
        const uint32_t b = list / a.parts;
        const double z = (double)value_at((uint32_t)(key >> 32)), d = z == top[b] ? 0.0 : z - top[b];
        // shift -inf: not in use; d -inf: beside +inf
        if (key == 0 || shift[b] == -INFINITY || d == -INFINITY) return Candidate{-INFINITY, 0};
        return Candidate{shift[b] + d, (uint64_t)(65535u - b) << 48 | key};
    }

    __device__ __forceinline__ uint64_t key(uint32_t list, uint32_t at) const
    {
        return a.lists[((int64_t)n * (a.beams * a.parts) + list) * a.K + at];
    }

    __device__ __forceinline__ void put(uint32_t k, const Candidate& c) const
    {
        const int64_t to = (int64_t)n * a.K + k;
        a.best[to] = c.rest ? (float)c.score : -INFINITY;
        a.rows_out[to] = c.rest ? (int32_t)(n * a.beams + 65535u - (uint32_t)(c.rest >> 48)) : -1;
        a.ids[to] = c.rest ? key_index(c.rest) : -1;
    }
};

// Every list's first candidate that is not taken yet meets the others', K times.
__device__ void join_by_turns(const Beams& beams, uint32_t* taken)
{
    __shared__ Candidate won[kJoinThreads / 64];
    const BeamArgs& a = beams.a;
    const uint32_t tid = threadIdx.x, lists = a.beams * a.parts;
    for (uint32_t i = tid; i < lists; i += kJoinThreads) taken[i] = 0;
    for (uint32_t k = 0; k < a.K; ++k) {
        Candidate mine = {-INFINITY, 0};
        uint32_t list = 0;
        for (uint32_t l = tid; l < lists; l += kJoinThreads) {
            if (taken[l] >= a.K) continue;
            const Candidate c = beams.of(l, beams.key(l, taken[l]));
            if (c.before(mine)) {
                mine = c;
                list = l;
            }
        }
        Candidate w = mine;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const Candidate o = {__shfl_xor(w.score, d), (uint64_t)__shfl_xor((unsigned long long)w.rest, d)};
            if (o.before(w)) w = o;
        }
        if ((tid & 63) == 0) won[tid / 64] = w;
        __syncthreads();
        w = won[0];
        for (uint32_t i = 1; i < kJoinThreads / 64; ++i) {
            if (won[i].before(w)) w = won[i];
        }
        if (tid == 0) beams.put(k, w);
        if (w.rest != 0 && mine.rest == w.rest) taken[list] += 1;
        __syncthreads();
    }
}

// A workgroup takes a sequence.  Of its lists' candidates those that can be among the K
// best are ranked by counting.  With d = K / lists rounded up, the K / d-th largest of
// the lists' d-th candidates is below K candidates or equal to some, and few others
// pass it.
__global__ void __launch_bounds__(kJoinThreads) join_kernel(BeamArgs a, uint32_t group)
{
    extern __shared__ double shift[];
    __shared__ __align__(16) Candidate few[kRanked];
    __shared__ uint32_t count;
    __shared__ double least;
    const uint32_t n = a.first + blockIdx.x, tid = threadIdx.x;
    const uint32_t lists = a.beams * a.parts;
    double* top = shift + a.beams;
    uint32_t* taken = reinterpret_cast<uint32_t*>(top + a.beams);   // of each list
    if (tid == 0) {
        count = 0;
        least = -INFINITY;
    }
    // `group` lanes a beam, a power of two
    const uint32_t lane = tid % group;
    for (uint32_t b0 = 0; b0 < a.beams; b0 += kJoinThreads / group) {
        const uint32_t b = b0 + tid / group;
        const bool on = b < a.beams;
        const int64_t unit = (int64_t)(n * a.beams + (on ? b : 0)) * a.parts;
        uint32_t o = 0;
        for (uint32_t p = lane; p < a.parts; p += group) o = max(o, (uint32_t)(a.lists[(unit + p) * a.K] >> 32));
        for (uint32_t d = 1; d < group; d *= 2) o = max(o, (uint32_t)__shfl_xor(o, d));
        const double m = (double)value_at(o);
        double total = 0.0;
        for (uint32_t p = lane; p < a.parts; p += group) {
            const uint32_t q = (uint32_t)(a.lists[(unit + p) * a.K] >> 32);
            if (q) total += a.sums[unit + p] * (q == o ? 1.0 : exp((double)value_at(q) - m));
        }
        for (uint32_t d = 1; d < group; d *= 2) total += __shfl_xor(total, d);
        if (on && lane == 0) {
            const double score = (double)a.scores[n * a.beams + b];
            shift[b] = o && fabs(score) < INFINITY ? score - log(total) : -INFINITY;
            top[b] = m;
        }
    }
    __syncthreads();
    const Beams beams = {a, shift, top, n};
    const uint32_t all = lists * a.K;
    if (lists > kRanked) return join_by_turns(beams, taken);
    if (all > kDirect) {
        const uint32_t deep = (a.K + lists - 1) / lists, need = (a.K + deep - 1) / deep;
        for (uint32_t l = tid; l < lists; l += kJoinThreads) few[l] = beams.of(l, beams.key(l, deep - 1));
        __syncthreads();
        for (uint32_t l = tid; l < lists; l += kJoinThreads) {
            const double mine = few[l].score;
            uint32_t more = 0, same = 0;
            for (uint32_t i = 0; i < lists; ++i) {
                more += few[i].score > mine;
                same += few[i].score == mine;
            }
            if (more < need && more + same >= need) least = mine;
        }
        __syncthreads();
    }
    const double from = least;
    for (uint32_t i = tid; i < all; i += kJoinThreads) {
        const uint32_t l = i / a.K;
        const Candidate c = beams.of(l, beams.key(l, i - l * a.K));
        if (c.rest && c.score >= from) {
            const uint32_t at = atomicAdd(&count, 1u);
            if (at < kRanked) few[at] = c;
        }
    }
    __syncthreads();
    const uint32_t found = count;
    if (found > kRanked) return join_by_turns(beams, taken);
    for (uint32_t i = tid; i < found; i += kJoinThreads) {
        const Candidate c = few[i];
        uint32_t rank = 0;
        for (uint32_t j = 0; j < found; ++j) rank += few[j].before(c);
        if (rank < a.K) beams.put(rank, c);
    }
    for (uint32_t k = found + tid; k < a.K; k += kJoinThreads) beams.put(k, Candidate{-INFINITY, 0});
}

constexpr int kMostStates = 8;   // of one launch

struct State {
    const char* from;
    char* to;
    int64_t step_from, step_to;   // bytes
    uint64_t bytes;               // of a row
    uint32_t piece;
};

struct ReorderArgs {
    State s[kMostStates];
    const int32_t* src;
    uint32_t N, M;
};

template <typename W>
__device__ __forceinline__ void move_row(const State& s, const char* from, char* to, bool on)
{
    const uint64_t n = s.bytes / sizeof(W);
    for (uint64_t i = blockIdx.x * (uint64_t)blockDim.x + threadIdx.x; i < n; i += (uint64_t)gridDim.x * blockDim.x) {
        W x = {};
        if (on) x = reinterpret_cast<const W*>(from)[i];
        reinterpret_cast<W*>(to)[i] = x;
    }
}

__global__ void __launch_bounds__(256) reorder_kernel(ReorderArgs a)
{
    const State s = a.s[blockIdx.z];
    for (uint32_t m = blockIdx.y; m < a.M; m += gridDim.y) {
        const uint32_t n = (uint32_t)a.src[m];
        const bool on = n < a.N;
        const char* from = s.from + (on ? n * s.step_from : 0);
        char* to = s.to + m * s.step_to;
        if (s.piece == 16) move_row<u32x4>(s, from, to, on);
        else if (s.piece == 4) move_row<uint32_t>(s, from, to, on);
        else move_row<uint8_t>(s, from, to, on);
    }
}

// Bytes that a call writes or reads.
struct Span {
    uintptr_t begin, end;
    bool write;
};

constexpr int64_t kMost = 0x7FFFFFFFll;

struct Shape {
    int64_t N, beams, V, K;
};

struct Plan {
    int64_t parts, part_vecs;
};

bool shape_ok(const Shape& s)
{
    return s.N >= 0 && s.N <= kMost && s.beams >= 1 && s.beams <= 4096 && s.V >= 1 && s.V <= kMost - 8 &&
           s.K >= 1 && s.K <= kMostK && s.N <= (kMost / s.beams);
}

// Parts: up to two workgroups a compute unit where the rows alone are fewer, but no part of
// fewer vectors than a workgroup has threads, nor of more than kRuns.  Parts of more are whole
// rounds of the threads, and so fewer: 4 rows of 152064 in 37 parts would have 514 vectors
// each, and are 19 of 1024.
Plan plan_of(const Shape& s)
{
    const int64_t vecs = (s.V + 7) / 8, rows = s.N * s.beams;
    int64_t parts = (vecs + kRuns - 1) / kRuns;
    const int64_t fill = (2 * 256 + rows - 1) / rows, fits = vecs / kThreads;
    const int64_t more = fill < fits ? fill : fits;
    if (more > parts) parts = more;
    Plan p;
    // whole rounds of a workgroup's threads, if a part has more than one
    p.part_vecs = (vecs + parts - 1) / parts;
    if (p.part_vecs > kThreads) p.part_vecs = (p.part_vecs + kThreads - 1) / kThreads * kThreads;
    p.parts = (vecs + p.part_vecs - 1) / p.part_vecs;
    return p;
}

int64_t words_of(const Shape& s, const Plan& p) { return s.N * s.beams * p.parts * (s.K + 1); }

// LDS of a sequence's beams and lists in the join.
int64_t join_bytes(const Shape& s, const Plan& p) { return s.beams * 16 + s.beams * p.parts * 4; }

bool plan_ok(const Shape& s, const Plan& p)
{
    return s.N * s.beams <= kMost / p.parts && join_bytes(s, p) <= 48 * 1024;
}

constexpr int64_t kMostUnits = 1 << 22;   // a grid has fewer than 2^32 threads

}  // namespace

extern "C" {

int xpress_beam_select(const uint16_t* base, const uint16_t* bias, const float* scores, float* best,
                       int32_t* rows, int64_t* ids, int64_t N, int64_t beams, int64_t V, int64_t K,
                       int64_t stride_base_r, int64_t stride_bias_r, hipStream_t stream)
{
    const Shape s = {N, beams, V, K};
    if (!shape_ok(s)) return XPRESS_EINVAL;
    if (N == 0) return XPRESS_OK;
    if (stride_base_r < V || stride_base_r > (kMost << 16) ||
        (bias && (stride_bias_r < V || stride_bias_r > (kMost << 16)))) {
        return XPRESS_EINVAL;
    }
    if (!base || !scores || !best || !rows || !ids || !is_aligned(base, 2) || !is_aligned(bias, 2) ||
        !is_aligned(scores, 4) || !is_aligned(best, 4) || !is_aligned(rows, 4) || !is_aligned(ids, 8)) {
        return XPRESS_EINVAL;
    }
    const int64_t R = N * beams;
    const size_t nb = ((size_t)(R - 1) * (size_t)stride_base_r + (size_t)V) * 2u;
    const size_t ni = bias ? ((size_t)(R - 1) * (size_t)stride_bias_r + (size_t)V) * 2u : 0;
    const size_t out = (size_t)(N * K);
    const struct { const void* p; size_t n; } w[] = {{best, out * 4u}, {rows, out * 4u}, {ids, out * 8u}},
                                              r[] = {{base, nb}, {bias, ni}, {scores, (size_t)R * 4u}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < i; ++j) {
            if (ranges_overlap(w[i].p, w[i].n, w[j].p, w[j].n)) return XPRESS_EINVAL;
        }
        for (const auto& x : r) {
            if (x.p && ranges_overlap(w[i].p, w[i].n, x.p, x.n)) return XPRESS_EINVAL;
        }
    }
    const Plan p = plan_of(s);
    if (!plan_ok(s, p)) return XPRESS_EINVAL;
    uint64_t* table = nullptr;
    const int rc = workspace_table(stream, words_of(s, p), &table);
    if (rc != XPRESS_OK) return rc;
    BeamArgs a = {base, bias, scores, best, rows, ids, stride_base_r, stride_bias_r, (uint32_t)V, (uint32_t)K,
                  (uint32_t)beams, (uint32_t)R, (uint32_t)p.parts, (uint32_t)p.part_vecs, 0, table,
                  reinterpret_cast<double*>(table + R * p.parts * K)};
    const bool vec = is_aligned16(base) && is_aligned16(bias) && stride_base_r % 8 == 0 &&
                     (!bias || stride_bias_r % 8 == 0);
    for (int64_t first = 0, units = R * p.parts; first < units; first += kMostUnits) {
        a.first = (uint32_t)first;
        const dim3 grid((uint32_t)(units - first < kMostUnits ? units - first : kMostUnits)), block(kThreads);
        if (vec && bias) hipLaunchKernelGGL((part_kernel<true, true>), grid, block, 0, stream, a);
        else if (vec) hipLaunchKernelGGL((part_kernel<true, false>), grid, block, 0, stream, a);
        else if (bias) hipLaunchKernelGGL((part_kernel<false, true>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((part_kernel<false, false>), grid, block, 0, stream, a);
    }
    for (int64_t first = 0; first < N; first += kMostUnits) {
        a.first = (uint32_t)first;
        const dim3 grid((uint32_t)(N - first < kMostUnits ? N - first : kMostUnits)), block(kJoinThreads);
        uint32_t group = 1;   // lanes for a beam's parts
        while (group < 64 && group < p.parts) group *= 2;
        hipLaunchKernelGGL(join_kernel, grid, block, (size_t)join_bytes(s, p), stream, a, group);
    }
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? XPRESS_OK : hip_fail(e);
}

int xpress_beam_select_reserve(int64_t N, int64_t beams, int64_t V, int64_t K, hipStream_t stream)
{
    const Shape s = {N, beams, V, K};
    if (!shape_ok(s)) return XPRESS_EINVAL;
    if (N == 0) return XPRESS_OK;
    const Plan p = plan_of(s);
    if (!plan_ok(s, p)) return XPRESS_EINVAL;
    uint64_t* table = nullptr;
    return workspace_table(stream, words_of(s, p), &table);
}

int xpress_beam_reorder(const xpress_beam_state* states, int64_t count, const int32_t* src, int64_t N,
                        int64_t M, hipStream_t stream)
{
    if (count < 0 || count > 4096 || N < 0 || N > kMost || M < 0 || M > kMost) return XPRESS_EINVAL;
    if (count == 0 || M == 0) return XPRESS_OK;
    if (!states || !src || !is_aligned(src, 4)) return XPRESS_EINVAL;
    const int64_t far = (int64_t)1 << 60;
    auto span = [&](int64_t rows, int64_t step, int64_t bytes) -> size_t {
        return rows > 0 ? (size_t)((rows - 1) * step + bytes) : 0;
    };
    for (int64_t i = 0; i < count; ++i) {
        const xpress_beam_state& x = states[i];
        if (x.bytes < 0 || x.bytes > far || x.step_from < 0 || x.step_to < 0) return XPRESS_EINVAL;
        if (x.bytes == 0) continue;
        if ((N > 0 && !x.from) || !x.to || x.step_from > far / (N > 0 ? N : 1) || x.step_to > far / M) {
            return XPRESS_EINVAL;
        }
        if (M > 1 && x.step_to < x.bytes) return XPRESS_EINVAL;
        if (ranges_overlap(x.to, span(M, x.step_to, x.bytes), src, (size_t)M * 4u)) return XPRESS_EINVAL;
    }
    // what is written lies apart from what any of them reads or writes: in the order of
    // their starts (pair by pair 160 states took 100 us)
    Span few_spans[64], *spans = few_spans;
    std::unique_ptr<Span[]> many;
    if (2 * count > 64) {
        many.reset(new (std::nothrow) Span[2 * count]);
        spans = many.get();
        if (!spans) return XPRESS_ENOMEM;
    }
    int64_t n_spans = 0;
    for (int64_t i = 0; i < count; ++i) {
        const xpress_beam_state& x = states[i];
        if (x.bytes == 0) continue;
        const uintptr_t to = reinterpret_cast<uintptr_t>(x.to), from = reinterpret_cast<uintptr_t>(x.from);
        spans[n_spans++] = Span{to, to + span(M, x.step_to, x.bytes), true};
        if (x.from && N > 0) spans[n_spans++] = Span{from, from + span(N, x.step_from, x.bytes), false};
    }
    std::sort(spans, spans + n_spans, [](const Span& x, const Span& y) { return x.begin < y.begin; });
    uintptr_t read = 0, written = 0;   // their ends so far
    for (int64_t i = 0; i < n_spans; ++i) {
        const Span& x = spans[i];
        if (x.begin < written || (x.write && x.begin < read)) return XPRESS_EINVAL;
        uintptr_t& end = x.write ? written : read;
        end = x.end > end ? x.end : end;
    }
    for (int64_t i = 0; i < count;) {
        ReorderArgs a = {};
        a.src = src;
        a.N = (uint32_t)N;
        a.M = (uint32_t)M;
        uint32_t n = 0;
        uint64_t most = 0;
        for (; i < count && n < (uint32_t)kMostStates; ++i) {
            const xpress_beam_state& x = states[i];
            if (x.bytes == 0) continue;
            State& s = a.s[n++];
            s = State{(const char*)x.from, (char*)x.to, x.step_from, x.step_to, (uint64_t)x.bytes, 1};
            for (uint32_t w : {16u, 4u}) {
                if (x.bytes % w == 0 && is_aligned(x.from, w) && is_aligned(x.to, w) &&
                    (N <= 1 || x.step_from % w == 0) && (M <= 1 || x.step_to % w == 0)) {
                    s.piece = w;
                    break;
                }
            }
            const uint64_t pieces = (uint64_t)x.bytes / s.piece;
            most = pieces > most ? pieces : most;
        }
        if (n == 0) break;
        uint64_t gx = (most + 1023) / 1024;   // a thread takes four pieces of the longest rows
        const uint32_t gy = (uint32_t)(M < 16384 ? M : 16384);
        if (gx > 64) gx = 64;
        hipLaunchKernelGGL(reorder_kernel, dim3((uint32_t)gx, gy, n), dim3(256), 0, stream, a);
    }
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? XPRESS_OK : hip_fail(e);
}

}  // extern "C"
