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
// the drawn token is the j-th id holding one known value.  No sort, no prefix
// sum over the vocabulary.  A workgroup of 512 threads, or 1024 where it has a
// compute unit for itself, takes a row; few long rows are counted in parts.
//
// Bins.  Magnitudes of 2^-26 to 2^16 have a 32-bit count each, for either sign:
// 43 KB, so that two workgroups share a compute unit and one streams its row
// while the other draws.  Values of -2^16 and below (masks) go to words that
// are not looked at, one for each lane: next to a maximum above -2^15, at a
// temperature of 2^15 / 746 or less, their weight is at most exp(-746), 0 in 64
// bits.  A row with anything else (a tinier value that is not 0, 2^16 or more, a
// lower maximum, a higher temperature) is counted again over all 65536 values,
// in seven windows of the order, a pass over the row for each, and another for a
// search whose window has gone: 480 rows with bias 629 us at a temperature of 44
// where 43 takes 146, one row 181 and 37; a +NaN in a row is as dear (596 and 180).
//
// The j-th id.  While the row goes by, the largest of each 16 logits is kept
// (in 16 bits; a run doubles with every doubling of the row past 163840): only
// runs that reach the drawn value are read again, for a likely token a few
// hundredths of the row.
//
// The order's walk goes by segments of 64 values, largest first.  A wave takes
// a segment at a time, one value per lane.
//
// Bound: many rows by their bytes, by the vector instructions (some 12 a logit in
// all, half of the time) and by how little of a row's draw overlaps with the two
// rows' counting, none of them alone; few rows by the chain of one workgroup.
// Measured at V = 152064: 480 rows with bias 67 (top-p alone) to 79 us, 3.7 to
// 4.4 TB/s, without bias 48 us, 3.1 TB/s (half the bytes, the same instructions); 15
// rows with bias 28 us, 9 of them the counting in parts, the rest the exponentials
// and searches of one workgroup; one row without bias 23 to 27 us.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "device_common.h"
#include "host_common.h"
#include "xpress_argmax.h"

namespace {

using namespace xpress;

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kDrawThreads = 1024;               // where a row has a compute unit for itself
constexpr uint32_t kUnits = 256;                 // compute units of the chip
constexpr int kMostWaves = kDrawThreads / 64;
constexpr uint32_t kInf = 0x7F80u;               // magnitude bits of infinity
constexpr uint32_t kOne = 0x3F80u;               // of 1
constexpr uint32_t kLeast = kOne - 26u * 128u;   // of 2^-26
constexpr uint32_t kRels = 42u * 128u;           // magnitudes up to 2^16: 1 .. kRels; 0 is zero
constexpr uint32_t kHuge = kRels + 1;            // all from 2^16 on: this and 62 more
constexpr uint32_t kTwo16 = kOne + 16u * 128u;   // magnitude bits of 2^16
constexpr double kHottest = 32768.0 / 746.0;
constexpr uint32_t kSide = 5440;                 // bins of a sign, whole segments
constexpr uint32_t kWindow = 10240;              // of the 65536 values, whole segments
constexpr uint32_t kKeys = 10240;
constexpr uint32_t kWidest = 5;                  // runs are of a wave's vectors at most
constexpr uint32_t kMaxParts = 8;
constexpr uint32_t kSegs = 1024;
static_assert(kSide % 64 == 0 && kHuge + 63 == kSide && kWindow <= 2 * kSide && kWindow % 64 == 0, "bins");

struct SampleArgs {
    const uint16_t *base, *bias;
    int64_t* blk;
    float* prob;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t* top_k;
    int64_t stride_base, stride_bias;
    uint32_t rows, bm1, V;
    uint32_t first;    // of the launch's rows
    // a row in parts
    uint32_t parts, part_vecs, list_room;
    uint32_t* lists;   // [rows, parts, list_room]
    uint4* infos;      // [rows, parts]: entries of the list, and what the counting saw
};

struct Shared {
    __align__(16) uint32_t bins[2 * kSide];
    uint16_t keys[kKeys];    // largest logit of a run, as int16 bits
    double mass[kSegs];      // mass of a segment; then: of all segments before it
    uint32_t count[kSegs];   // the same for logits
    double wave_mass[kMostWaves];
    double wave_min[kMostWaves];
    uint32_t wave_count[kMostWaves];
    uint32_t wave_low[kMostWaves];
    int32_t wave_high[kMostWaves];
    uint16_t turns[kMostWaves][kKeys / 64 / kWaves + 1];
    double f64;
    uint32_t found, counted;
    uint32_t chosen;         // apart from `found`, which waves still read when it is set
};

__device__ __forceinline__ float value_of(uint32_t h) { return __uint_as_float(h << 16); }

// Value bits at position i of the descending order of all values (i = 0: the
// largest positive magnitude 0x7FFF; 32767: +0; 32768: -0; 65535: magnitude
// 0x7FFF), and the reverse.
__device__ __forceinline__ uint32_t all_bits_at(uint32_t i) { return i < 32768u ? 32767u - i : i; }
__device__ __forceinline__ uint32_t all_order_of(uint32_t h) { return h < 32768u ? 32767u - h : h; }

template <bool VEC, bool BIAS>
struct Logits {
    const uint16_t *base, *bias;
    uint32_t V;

    // Eight summed logits of a row from element e on; bits past the row are NaN.
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

__device__ __forceinline__ uint32_t half_of(const u32x4& z, int i)
{
    return i & 1 ? z[i / 2] >> 16 : z[i / 2] & 0xFFFFu;
}

// Whether a vector's eight halves are one value.
__device__ __forceinline__ bool all_alike(const u32x4& z)
{
    return z[0] == z[1] && z[0] == z[2] && z[0] == z[3] && z[0] >> 16 == (z[0] & 0xFFFFu);
}

// Counts one vector into the bins.  No branch a logit, the arithmetic on pairs.
// Returns the vector's largest logit as an int16 (right where it is not
// negative); *least: the smallest magnitude less 1 (so that zero does not count).
__device__ __forceinline__ int32_t tally(Shared& s, const u32x4& z, u16x2* least)
{
    const u16x2 last = (u16x2)(uint16_t)(kHuge + threadIdx.x % 63);
    u32x4 at;   // byte offsets
    i16x2 top = {INT16_MIN, INT16_MIN};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint32_t two = z[w];
        const u16x2 mag = __builtin_bit_cast(u16x2, two & 0x7FFF7FFFu);
        *least = __builtin_elementwise_min(*least, (u16x2)(mag - (u16x2)1));
        const i16x2 h = __builtin_bit_cast(i16x2, two);
        top = __builtin_elementwise_max(top, h);
        u16x2 r = __builtin_elementwise_sub_sat(mag, (u16x2)(uint16_t)(kLeast - 1));
        r = __builtin_elementwise_min(r, last);
        const u16x2 side = __builtin_bit_cast(u16x2, (i16x2)(h >> (i16x2)15)) & (u16x2)(uint16_t)kSide;
        at[w] = __builtin_bit_cast(uint32_t, (u16x2)((r + side) << (u16x2)2));
    }
    char* bins = reinterpret_cast<char*>(s.bins);
    if (all_alike(z)) {
        atomicAdd(reinterpret_cast<uint32_t*>(bins + (at[0] & 0xFFFFu)), 8u);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) atomicAdd(reinterpret_cast<uint32_t*>(bins + half_of(at, i)), 1u);
    }
    return max((int32_t)top.x, (int32_t)top.y);
}

// Sums over the wave, the same in every lane.
__device__ __forceinline__ uint32_t wave_add(uint32_t v)
{
    v += dpp_u32<0xB1>(v);   // lane ^ 1, ^ 2, the other quad of 8, the other 8 of 16
    v += dpp_u32<0x4E>(v);
    v += dpp_u32<0x141>(v);
    v += dpp_u32<0x140>(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)dpp_u32<CTRL>((uint32_t)(b >> 32)) << 32 |
                                          dpp_u32<CTRL>((uint32_t)b));
}

__device__ __forceinline__ double wave_add(double v)
{
    v += dpp_f64<0xB1>(v);
    v += dpp_f64<0x4E>(v);
    v += dpp_f64<0x141>(v);
    v += dpp_f64<0x140>(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// exp((z - max) / t) in 64 bits, for d = z - max <= 0 and inv = 1 / t.  The
// quotient with one correction step; then x = k ln 2 + f, |f| <= ln(2) / 2, and
// the Taylor series of e^f to f^13 (its rest is below 2^-57).
__device__ __forceinline__ double weight_of(double d, double t, double inv)
{
    double x = d * inv;
    if (t < INFINITY) x = fma(fma(-x, t, d), inv, x);
    x = d > -INFINITY ? fmax(x, -800.0) : -800.0;   // 0 from exp(-746) on
    const double k = rint(x * 1.4426950408889634);
    double f = fma(-k, 0x1.62e42fefa39efp-1, x);    // ln 2 in two parts
    f = fma(-k, 0x1.abc9e3b39803fp-56, f);
    double y = 1.0 / 6227020800.0;
    y = fma(y, f, 1.0 / 479001600.0);
    y = fma(y, f, 1.0 / 39916800.0);
    y = fma(y, f, 1.0 / 3628800.0);
    y = fma(y, f, 1.0 / 362880.0);
    y = fma(y, f, 1.0 / 40320.0);
    y = fma(y, f, 1.0 / 5040.0);
    y = fma(y, f, 1.0 / 720.0);
    y = fma(y, f, 1.0 / 120.0);
    y = fma(y, f, 1.0 / 24.0);
    y = fma(y, f, 1.0 / 6.0);
    y = fma(y, f, 0.5);
    y = fma(y, f, 1.0);
    y = fma(y, f, 1.0);
    return ldexp(y, (int)k);
}

// The draw of one row.  FULL: over all values, a window of whose counts the bins
// hold; else the bins hold the counts of all values that can be drawn.
template <bool VEC, bool BIAS, bool FULL, int THREADS>
struct Row {
    static constexpr uint32_t kThreads = THREADS, kWaves = THREADS / 64;

    Shared& s;
    const Logits<VEC, BIAS>& z;
    uint32_t window;    // FULL: whose counts the bins hold
    uint32_t top;       // order position of the largest value
    double zmax, t, inv;

    static constexpr uint32_t kOrder = FULL ? 65536u : 2 * kSide;   // positions

    __device__ __forceinline__ uint32_t bits_at(uint32_t i) const
    {
        if constexpr (FULL) return all_bits_at(i);
        const uint32_t rel = i < kSide ? kSide - 1 - i : i - kSide;
        return (rel ? kLeast - 1 + rel : 0) | (i < kSide ? 0 : 0x8000u);
    }

    // Number of logits at order position i (FULL: of the window); both zeros
    // count at +0.
    __device__ __forceinline__ uint32_t count_at(uint32_t i) const
    {
        if constexpr (FULL) return s.bins[i - window * kWindow];
        if (i == kSide - 1) return s.bins[0] + s.bins[kSide];
        if (i == kSide) return 0;
        return i < kSide ? s.bins[kSide - 1 - i] : s.bins[i];
    }

    // Whether order position i may be drawn: a value at or below the top, not
    // NaN, not -inf.
    __device__ __forceinline__ bool real(uint32_t i) const
    {
        if (i < top) return false;
        if constexpr (FULL) {
            const uint32_t h = all_bits_at(i);
            return (h & 0x7FFFu) <= kInf && h != (0x8000u | kInf);
        }
        return (i < kSide ? kSide - 1 - i : i - kSide) <= kRels;
    }

    // FULL: counts the window of segment seg.
    __device__ void load(uint32_t seg)
    {
        if constexpr (FULL) {
            const uint32_t want = seg / (kWindow / 64);
            if (window == want) return;
            __syncthreads();
            window = want;
            for (uint32_t i = threadIdx.x; i < kWindow; i += kThreads) s.bins[i] = 0;
            __syncthreads();
            for (uint32_t e = threadIdx.x * 8; e < z.V; e += kThreads * 8) {
                const u32x4 v = z.at(e);
                const bool alike = all_alike(v);
                for (int i = 0; i < 8; ++i) {
                    const uint32_t h = half_of(v, i);
                    const uint32_t at = (h == 0x8000u ? 32767u : all_order_of(h)) - want * kWindow;
                    if (at < kWindow && (!alike || i == 0)) atomicAdd(&s.bins[at], alike ? 8u : 1u);
                }
            }
            __syncthreads();
        }
    }

    // The first position of the order that holds a value, or kOrder.
    __device__ uint32_t find_top()
    {
        const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x / 64;
        uint32_t best = kOrder;
        top = 0;
        constexpr uint32_t kSpan = FULL ? kWindow : kOrder;
        for (uint32_t from = 0; from < kOrder && best == kOrder; from += kSpan) {
            load(from / 64);
            for (uint32_t i = from + threadIdx.x; i < min(from + kSpan, kOrder); i += kThreads) {
                if (real(i) && count_at(i) != 0) {
                    best = i;
                    break;
                }
            }
            for (int m = 32; m; m >>= 1) best = min(best, __shfl_xor(best, m));
            if (lane == 0) s.wave_count[wave] = best;
            __syncthreads();
            for (uint32_t w = 0; w < kWaves; ++w) best = min(best, s.wave_count[w]);
            __syncthreads();
        }
        return best;
    }

    __device__ __forceinline__ double weight_at(uint32_t i) const
    {
        if (i == top) return 1.0;
        return weight_of((double)value_of(bits_at(i)) - zmax, t, inv);
    }

    // The wave's lanes look at one segment: its counts and masses, in order,
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

    // Chooses the value: its bits in *want, which of its ids in *nth; returns the
    // probability.
    __device__ double choose(const SampleArgs& a, uint32_t r, bool greedy, uint32_t* want, uint32_t* nth)
    {
        const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
        if (greedy) {
            *want = bits_at(top);
            *nth = 0;
            return 1.0;
        }
        // counts and masses of the segments, and the mass that min-p keeps
        constexpr uint32_t kUsed = kOrder / 64;
        const float min_p = a.min_p[r], top_p = a.top_p[r];
        const bool by_min = min_p > 0.0f;
        double kept_min = 0.0;
        // three segments of a wave at a time, for their latencies to overlap
        constexpr uint32_t kTurn = FULL ? 1 : 3;
        for (uint32_t seg0 = 0; seg0 < kUsed; seg0 += kTurn * kWaves) {
            if (FULL && seg0 % (kWindow / 64) == 0) load(seg0);
            uint32_t n[kTurn];
            bool some = false;
#pragma unroll
            for (uint32_t x = 0; x < kTurn; ++x) {
                const uint32_t seg = seg0 + x * kWaves + wave, i = seg * 64 + lane;
                n[x] = seg < kUsed && real(i) ? count_at(i) : 0;
                some |= n[x] != 0;
            }
            if (!__any(some)) {
#pragma unroll
                for (uint32_t x = 0; x < kTurn; ++x) {
                    const uint32_t seg = seg0 + x * kWaves + wave;
                    if (lane == 0 && seg < kUsed) {
                        s.count[seg] = 0;
                        s.mass[seg] = 0.0;
                    }
                }
                continue;
            }
            uint32_t c[kTurn];
            double m[kTurn];
#pragma unroll
            for (uint32_t x = 0; x < kTurn; ++x) {
                const uint32_t i = (seg0 + x * kWaves + wave) * 64 + lane;
                const double w = n[x] ? weight_at(i) : 0.0;
                m[x] = (double)n[x] * w;
                if (w >= (double)min_p) kept_min += m[x];
            }
#pragma unroll
            for (uint32_t x = 0; x < kTurn; ++x) {
                m[x] = wave_add(m[x]);
                c[x] = wave_add(n[x]);
            }
#pragma unroll
            for (uint32_t x = 0; x < kTurn; ++x) {
                const uint32_t seg = seg0 + x * kWaves + wave;
                if (lane == 0 && seg < kUsed) {
                    s.count[seg] = c[x];
                    s.mass[seg] = m[x];
                }
            }
        }
        if (by_min) {
            kept_min = wave_add(kept_min);
            if (lane == 0) s.wave_min[wave] = kept_min;
        }
        __syncthreads();
        // exclusive prefix over the segments, kEach to a thread
        constexpr uint32_t kEach = (kUsed + kThreads - 1) / kThreads;
        constexpr uint32_t kHold = (kUsed + 64 * kEach - 1) / (64 * kEach);  // waves that have segments
        uint32_t c_own[kEach], c_before[kEach], c = 0, c_all = 0;
        double m_own[kEach], m_before[kEach], m = 0.0, m_all = 0.0, m_min = 0.0;
#pragma unroll
        for (uint32_t x = 0; x < kEach; ++x) {
            const uint32_t seg = tid * kEach + x;
            c_own[x] = seg < kUsed ? s.count[seg] : 0;
            m_own[x] = seg < kUsed ? s.mass[seg] : 0.0;
            c += c_own[x];
            m += m_own[x];
        }
        const uint32_t c_thread = c;
        const double m_thread = m;
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
        c -= c_thread;
        m -= m_thread;
        for (uint32_t w = 0; w < kHold; ++w) {
            if (w < wave) {
                c += s.wave_count[w];
                m += s.wave_mass[w];
            }
            c_all += s.wave_count[w];
            m_all += s.wave_mass[w];
        }
        if (by_min) {
            for (uint32_t w = 0; w < kWaves; ++w) m_min += s.wave_min[w];
        }
#pragma unroll
        for (uint32_t x = 0; x < kEach; ++x) {
            const uint32_t seg = tid * kEach + x;
            c_before[x] = c;
            m_before[x] = m;
            if (seg < kUsed) {
                s.count[seg] = c;
                s.mass[seg] = m;
            }
            c += c_own[x];
            m += m_own[x];
        }
        __syncthreads();
        // the kept mass: the least of the rules' (each keeps a prefix)
        const int32_t k = a.top_k[r];
        double z_mass = m_all;
        if (k > 0 && (uint32_t)k < c_all) {
            // the segment in which the k-th id lies
#pragma unroll
            for (uint32_t x = 0; x < kEach; ++x) {
                if (c_own[x] && c_before[x] < (uint32_t)k && (uint32_t)k <= c_before[x] + c_own[x]) {
                    s.found = tid * kEach + x;
                }
            }
            __syncthreads();
            const uint32_t seg = s.found;
            load(seg);
            if (wave == 0) {
                uint32_t n, n_to;
                double w, m_to;
                segment(seg, &n, &w, &n_to, &m_to);
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
#pragma unroll
            for (uint32_t x = 0; x < kEach; ++x) {
                if (c_own[x] && m_before[x] < goal) atomicMax(&s.found, tid * kEach + x);
            }
            __syncthreads();
            const uint32_t seg = s.found;
            load(seg);
            if (wave == 0) {
                uint32_t n, n_to;
                double w, m_to;
                segment(seg, &n, &w, &n_to, &m_to);
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
        // the first id at which the mass passes u * kept
        float u = a.u[r];
        u = u > 0.0f ? u : 0.0f;
        u = u < 1.0f ? u : 0x1.fffffep-1f;
        const double goal = (double)u * kept;
        if (tid == 0) s.found = top / 64;
        __syncthreads();
#pragma unroll
        for (uint32_t x = 0; x < kEach; ++x) {
            if (c_own[x] && m_own[x] > 0.0 && m_before[x] <= goal) atomicMax(&s.found, tid * kEach + x);
        }
        __syncthreads();
        const uint32_t seg = s.found;
        load(seg);
        if (wave == 0) {
            uint32_t n, n_to;
            double w, m_to;
            segment(seg, &n, &w, &n_to, &m_to);
            const double before = s.mass[seg] + (m_to - (double)n * w);
            const uint64_t may = __ballot(n && w > 0.0 && before <= goal);
            // the segment's first value where rounding leaves none
            const uint64_t any = __ballot(n && w > 0.0);
            const int at = may ? 63 - __clzll(may) : __ffsll((unsigned long long)any) - 1;
            if ((int)lane == at) {
                double j = floor((goal - before) / w);
                j = j < 0.0 ? 0.0 : j > (double)(n - 1) ? (double)(n - 1) : j;
                s.chosen = seg * 64 + lane;
                s.counted = (uint32_t)j;
                s.f64 = w / kept;
            }
        }
        __syncthreads();
        *want = bits_at(s.chosen);
        *nth = s.counted;
        return s.f64;
    }
};

// Which of a vector's logits hold the value `want` (either zero for +0).
__device__ __forceinline__ uint32_t matches(const u32x4& z, uint32_t want)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = half_of(z, i);
        m |= (uint32_t)(h == want || (want == 0 && h == 0x8000u)) << i;
    }
    return m;
}

__device__ __forceinline__ uint32_t nth_bit(uint32_t bits, uint32_t nth)
{
    for (; nth; --nth) bits &= bits - 1;
    return (uint32_t)__ffs(bits) - 1u;
}

// What the counting learns beside the counts: the largest logit (right where it is
// not negative) and the smallest magnitude less 1.
struct Seen {
    int32_t high;
    uint32_t tiny;
};

// Counts the vectors [v0, v1) of a row into the bins, which it clears.  KEYS: also
// keeps the runs' largest logits, of 16 << wide each.
template <int THREADS, bool VEC, bool BIAS, bool KEYS>
__device__ __forceinline__ Seen count_range(Shared& s, const Logits<VEC, BIAS>& z, uint32_t v0, uint32_t v1,
                                            uint32_t wide)
{
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
    constexpr int kAhead = BIAS || !KEYS ? 4 : 8;  // vectors of a thread in flight
    u32x4 got[kAhead], add[kAhead];
    const uint32_t whole = VEC ? min(v1, z.V / 8) : 0;  // the vectors below it are loaded whole
    // loads are queued always (past the range, its last vector again)
    auto fetch = [&](int x, uint32_t v) {
        const uint32_t e = min(v, whole - 1) * 8;
        got[x] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(z.base + e));
        if constexpr (BIAS) add[x] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(z.bias + e));
    };
    Seen seen = {INT16_MIN, 0};
    u16x2 least = {0xFFFFu, 0xFFFFu};
    auto take = [&](const u32x4& y, uint32_t v) {
        int32_t key = tally(s, y, &least);
        seen.high = max(seen.high, key);
        if constexpr (KEYS) {
            if (wide <= kWidest) {
                key = max(key, (int32_t)dpp_u32<0xB1>((uint32_t)key));   // lane ^ 1
                for (uint32_t d = 2; d < 2u << wide; d <<= 1) key = max(key, __shfl_xor(key, d));
                if ((v & ((2u << wide) - 1)) == 0 && v < v1) s.keys[v >> (wide + 1)] = (uint16_t)key;
            }
        }
    };
    const bool some = VEC && whole > v0;
    if (some) {
#pragma unroll
        for (int x = 0; x < kAhead; ++x) fetch(x, v0 + tid + x * THREADS);
    }
    for (uint32_t i = tid * 4; i < 2 * kSide; i += THREADS * 4) {
        *reinterpret_cast<u32x4*>(&s.bins[i]) = u32x4{0, 0, 0, 0};
    }
    __syncthreads();
    // Every lane takes part in every vector (as NaN past the range), for the runs.
    auto arrived = [&](int x) {
        u32x4 y = got[x];
        if constexpr (BIAS) {
#pragma unroll
            for (int w = 0; w < 4; ++w) y[w] = add_round2(y[w], add[x][w]);
        }
        return y;
    };
    auto slow = [&](uint32_t v) { return z.at(v < v1 ? v * 8 : z.V); };
    uint32_t at = v0;  // of all threads
    if (VEC) {
        for (; at + kAhead * THREADS <= whole; at += kAhead * THREADS) {
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const u32x4 y = arrived(x);
                const uint32_t v = at + x * THREADS + tid;
                fetch(x, v + kAhead * THREADS);
                take(y, v);
            }
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            if (some && at < whole) {
                const uint32_t v = at + tid;
                take(v < whole ? arrived(x) : slow(v), v);
                at += THREADS;
            }
        }
    }
    for (; at < v1; at += THREADS) take(slow(at + tid), at + tid);
    seen.tiny = min((uint32_t)least.x, (uint32_t)least.y);
    for (int m = 32; m; m >>= 1) {
        seen.tiny = min(seen.tiny, __shfl_xor(seen.tiny, m));
        seen.high = max(seen.high, __shfl_xor(seen.high, m));
    }
    if (lane == 0) {
        s.wave_low[wave] = seen.tiny;
        s.wave_high[wave] = seen.high;
    }
    __syncthreads();
    for (uint32_t w = 0; w < THREADS / 64; ++w) {
        seen.tiny = min(seen.tiny, s.wave_low[w]);
        seen.high = max(seen.high, s.wave_high[w]);
    }
    return seen;
}

struct Drawn {
    uint32_t want, nth;   // value bits, and which of its ids
    double p;
    bool usual, none;     // from the bins of all drawable values; nothing to draw
};

// Draws a value from the counts in the bins, or from the row counted again.
template <int THREADS, bool VEC, bool BIAS>
__device__ __forceinline__ Drawn draw(Shared& s, const SampleArgs& a, const Logits<VEC, BIAS>& z, uint32_t r,
                                      const Seen& seen, bool greedy, double t)
{
    const double inv = 1.0 / t;
    Drawn d = {0, 0, 0.0, false, false};
    d.usual = seen.tiny >= kLeast - 1 && seen.high < (int32_t)kTwo16 && t <= kHottest;
    if (d.usual) {
        Row<VEC, BIAS, false, THREADS> row{s, z, 0, 0, 0.0, t, inv};
        // a positive maximum is known already
        const uint32_t top = seen.high > 0 ? kSide - 1 - ((uint32_t)seen.high - (kLeast - 1)) : row.find_top();
        const uint32_t h = row.bits_at(top);
        d.usual = top < row.kOrder && (h < 0x8000u || (h & 0x7FFFu) < kTwo16 - 128u);
        if (d.usual) {
            row.top = top;
            row.zmax = (double)value_of(h);
            d.p = row.choose(a, r, greedy, &d.want, &d.nth);
        }
    }
    if (!d.usual) {
        Row<VEC, BIAS, true, THREADS> row{s, z, 0xFFFFu, 0, 0.0, t, inv};
        const uint32_t top = row.find_top();
        d.none = top >= row.kOrder;  // nothing but NaN and -inf
        if (!d.none) {
            row.top = top;
            row.zmax = (double)value_of(all_bits_at(top));
            d.p = row.choose(a, r, greedy, &d.want, &d.nth);
        }
    }
    __syncthreads();
    return d;
}

// The nth id (in id order) of vectors [v0, v1) that holds the value: each wave
// counts its share, then the share with the id is walked.
template <int THREADS, bool VEC, bool BIAS>
__device__ __forceinline__ void walk(Shared& s, const Logits<VEC, BIAS>& z, uint32_t v0, uint32_t v1, uint32_t want,
                                     uint32_t nth, int64_t* dst)
{
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const uint32_t steps = (v1 - v0 + THREADS - 1) / THREADS;  // of 64 vectors per wave
    auto look = [&](uint32_t i) {
        const uint32_t v = v0 + (wave * steps + i) * 64 + lane;
        return z.at(i < steps && v < v1 ? v * 8 : z.V);
    };
    uint32_t mine = 0;
    for (uint32_t i = 0; i < steps; i += 4) {
        u32x4 y[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) y[x] = look(i + x);
#pragma unroll
        for (int x = 0; x < 4; ++x) mine += __popc(matches(y[x], want));
    }
    mine = wave_add(mine);
    if (lane == 0) s.wave_count[wave] = mine;
    __syncthreads();
    uint32_t before = 0;
    for (uint32_t w = 0; w < wave; ++w) before += s.wave_count[w];
    if (before <= nth && nth < before + mine) {
        uint32_t left = nth - before;
        for (uint32_t i = 0; i < steps; ++i) {
            const uint32_t m = matches(look(i), want), n = __popc(m);
            uint32_t to = n;
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t o = __shfl_up(to, d);
                if ((int)lane >= d) to += o;
            }
            const uint32_t all = __shfl(to, 63);
            if (left < all) {
                if (to - n <= left && left < to) {
                    const uint32_t v = v0 + (wave * steps + i) * 64 + lane;
                    *dst = (int64_t)(v * 8 + nth_bit(m, left - (to - n)));
                }
                break;
            }
            left -= all;
        }
    }
}

template <bool VEC, bool BIAS>
__device__ __forceinline__ Logits<VEC, BIAS> logits_of(const SampleArgs& a, uint32_t r)
{
    return {a.base + (int64_t)r * a.stride_base, BIAS ? a.bias + (int64_t)r * a.stride_bias : nullptr, a.V};
}

// A workgroup a row.
template <int THREADS, bool VEC, bool BIAS>
__global__ void __launch_bounds__(THREADS, 4) sample_kernel(SampleArgs a)
{
    __shared__ Shared s;
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid / 64, r = a.first + blockIdx.x;
    const uint32_t V = a.V, vecs = (V + 7) / 8;
    uint32_t wide = 0;
    while ((vecs + (2u << wide) - 1) >> (wide + 1) > kKeys) ++wide;
    const float temp = a.temperature[r];
    const bool greedy = !(temp > 0.0f);
    const double t = greedy ? 1.0 : (double)temp;
    const Logits<VEC, BIAS> z = logits_of<VEC, BIAS>(a, r);
    int64_t* dst = a.blk + (r + r / a.bm1 + 1);

    const Seen seen = count_range<THREADS, VEC, BIAS, true>(s, z, 0, vecs, wide);
    const Drawn d = draw<THREADS>(s, a, z, r, seen, greedy, t);
    if (tid == 0 && a.prob) a.prob[r] = (float)d.p;
    if (d.none) {
        if (tid == 0) *dst = 0;
        return;
    }
    const uint32_t want = d.want, nth = d.nth;
    // The nth id (in id order) that holds the value, among the runs that reach
    // it: a wave lists those of its share in order, counts their matches 64 runs
    // at a time, and the one with the id looks at its 64 again.
    if (d.usual && wide <= kWidest && want > 0 && want < 0x8000u) {
        const uint32_t runs = (vecs + (2u << wide) - 1) >> (wide + 1);
        const uint32_t share = (runs + (THREADS / 64) * 64 - 1) / ((THREADS / 64) * 64) * 64, first = wave * share;
        uint32_t* list = s.bins + first;   // the bins are not needed any more
        uint32_t n = 0;
        for (uint32_t g0 = first; g0 < min(first + share, runs); g0 += 256) {
            int32_t key[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t g = g0 + x * 64 + lane;
                key[x] = g < min(first + share, runs) ? (int32_t)(int16_t)s.keys[g] : -1;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const bool on = key[x] >= (int32_t)want;
                const uint64_t all = __ballot(on);
                if (on) list[n + __popcll(all & ((1ull << lane) - 1))] = g0 + x * 64 + lane;
                n += (uint32_t)__popcll(all);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        auto held = [&](uint32_t at) {
            uint32_t count = 0;
            if (at < n) {
                const uint32_t x0 = list[at] << (wide + 1);
                for (uint32_t x = x0; x < x0 + (2u << wide) && x < vecs; x += 2) {
                    const u32x4 p0 = z.at(x * 8), p1 = z.at(min(x * 8 + 8, V));
                    count += __popc(matches(p0, want)) + __popc(matches(p1, want));
                }
            }
            return count;
        };
        uint32_t sum = 0, first64 = 0;
        for (uint32_t at = 0; at < n; at += 128) {
            const uint32_t h0 = held(at + lane), h1 = n > at + 64 ? held(at + 64 + lane) : 0;
            const uint32_t c0 = wave_add(h0), c1 = wave_add(h1);
            if (at == 0) first64 = h0;
            if (lane == 0) {
                s.turns[wave][at / 64] = (uint16_t)min(c0, 65535u);
                s.turns[wave][at / 64 + 1] = (uint16_t)min(c1, 65535u);
            }
            sum += c0 + c1;
        }
        if (lane == 0) s.wave_count[wave] = sum;
        __syncthreads();
        uint32_t before = 0;
        for (uint32_t w = 0; w < wave; ++w) before += s.wave_count[w];
        if (before <= nth && nth < before + sum) {
            uint32_t left = nth - before, at = 0;
            while (left >= s.turns[wave][at]) left -= s.turns[wave][at++];
            const uint32_t in = at == 0 ? first64 : held(at * 64 + lane);
            uint32_t to = in;
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t o = __shfl_up(to, d);
                if ((int)lane >= d) to += o;
            }
            if (to - in <= left && left < to) {
                left -= to - in;
                for (uint32_t x = list[at * 64 + lane] << (wide + 1);; ++x) {
                    const uint32_t m = matches(z.at(x * 8), want), k = __popc(m);
                    if (left < k) {
                        *dst = (int64_t)(x * 8 + nth_bit(m, left));
                        break;
                    }
                    left -= k;
                }
            }
        }
        return;
    }
    walk<THREADS>(s, z, 0, vecs, want, nth, dst);
}

// Few rows: a.parts workgroups count a row's parts, and list the bins that are
// not 0, as bin << 18 | count; one workgroup a row then adds the lists up and
// draws, and looks for the id in the one part that has it.
template <bool VEC, bool BIAS>
__global__ void __launch_bounds__(kThreads, 4) count_kernel(SampleArgs a)
{
    __shared__ Shared s;
    const uint32_t tid = threadIdx.x, lane = tid & 63, r = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    const uint32_t vecs = (a.V + 7) / 8, v0 = min(part * a.part_vecs, vecs), v1 = min(v0 + a.part_vecs, vecs);
    const Seen seen = count_range<kThreads, VEC, BIAS, false>(s, logits_of<VEC, BIAS>(a, r), v0, v1, 0);
    if (tid == 0) s.found = 0;
    __syncthreads();
    uint32_t* list = a.lists + (int64_t)blockIdx.x * a.list_room;
    for (uint32_t i0 = 0; i0 < 2 * kSide; i0 += kThreads) {
        const uint32_t i = i0 + tid, n = i < 2 * kSide ? s.bins[i] : 0;
        const uint64_t on = __ballot(n != 0);
        uint32_t at = 0;
        if (lane == 0 && on) at = atomicAdd(&s.found, (uint32_t)__popcll(on));
        at = __shfl(at, 0) + (uint32_t)__popcll(on & ((1ull << lane) - 1));
        if (n != 0) list[at] = i << 18 | n;
    }
    __syncthreads();
    // whole quadruples
    if (tid < 4 && (s.found + tid) / 4 == s.found / 4 && s.found % 4 != 0) list[s.found + tid] = 0;
    if (tid == 0) {
        a.infos[blockIdx.x] = uint4{s.found, seen.tiny, (uint32_t)seen.high, 0};
    }
}

template <bool VEC, bool BIAS>
__global__ void __launch_bounds__(kDrawThreads, 4) draw_kernel(SampleArgs a)
{
    __shared__ Shared s;
    __shared__ uint32_t held[kMaxParts];
    const uint32_t tid = threadIdx.x, lane = tid & 63, r = blockIdx.x;
    const uint32_t vecs = (a.V + 7) / 8;
    const float temp = a.temperature[r];
    const bool greedy = !(temp > 0.0f);
    const double t = greedy ? 1.0 : (double)temp;
    const Logits<VEC, BIAS> z = logits_of<VEC, BIAS>(a, r);
    int64_t* dst = a.blk + (r + r / a.bm1 + 1);
    for (uint32_t i = tid * 4; i < 2 * kSide; i += kDrawThreads * 4) {
        *reinterpret_cast<u32x4*>(&s.bins[i]) = u32x4{0, 0, 0, 0};
    }
    if (tid < kMaxParts) held[tid] = 0;
    __syncthreads();
    // a wave's list: two waves a part, four entries a lane
    static_assert(kMaxParts * 2 * 64 == kDrawThreads, "waves of a part");
    const uint32_t part = tid / 128;
    const u32x4* list = reinterpret_cast<const u32x4*>(a.lists + (int64_t)(r * a.parts + part) * a.list_room);
    const uint32_t quads = (a.infos[r * a.parts + part].x + 3) / 4;
    auto each = [&](auto use) {
        for (uint32_t i = tid % 128; i < quads; i += 4 * 128) {
            u32x4 e[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) e[x] = i + x * 128 < quads ? list[i + x * 128] : u32x4{0, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) use(e[x][y] >> 18, e[x][y] & 0x3FFFFu);
        }
    };
    each([&](uint32_t bin, uint32_t n) {
        if (n) atomicAdd(&s.bins[bin], n);
    });
    Seen seen = {INT16_MIN, 0xFFFFu};
    for (uint32_t p = 0; p < a.parts; ++p) {
        const uint4 info = a.infos[r * a.parts + p];
        seen.tiny = min(seen.tiny, info.y);
        seen.high = max(seen.high, (int32_t)info.z);
    }
    __syncthreads();
    const Drawn d = draw<kDrawThreads>(s, a, z, r, seen, greedy, t);
    if (tid == 0 && a.prob) a.prob[r] = (float)d.p;
    if (d.none) {
        if (tid == 0) *dst = 0;
        return;
    }
    uint32_t v0 = 0, v1 = vecs, nth = d.nth;
    if (d.usual) {
        // the parts' numbers of the value (either zero for +0)
        const uint32_t mag = d.want & 0x7FFFu, rel = mag ? mag - (kLeast - 1) : 0;
        const uint32_t bin = rel + (d.want >> 15) * kSide;
        uint32_t count = 0;
        each([&](uint32_t at, uint32_t n) {
            if (at == bin || (rel == 0 && at == kSide)) count += n;
        });
        count = wave_add(count);
        if (lane == 0 && count) atomicAdd(&held[part], count);
        __syncthreads();
        uint32_t p = 0;
        while (p + 1 < a.parts && nth >= held[p]) nth -= held[p++];
        v0 = min(p * a.part_vecs, vecs);
        v1 = min(v0 + a.part_vecs, vecs);
    }
    walk<kDrawThreads>(s, z, v0, v1, d.want, nth, dst);
}

// Long rows with a bias go in parts while their number leaves most compute units
// idle: a row of 152064 in 26 us where one workgroup takes 28, 16 rows 28 and 30;
// at 64 rows one workgroup each is faster (33 and 31), at 50000 logits too (24
// and 19), and without a bias, which is half the bytes (26 and 25).
void plan_parts(SampleArgs* a, bool bias)
{
    a->part_vecs = ((a->V + 7) / 8 + kMaxParts - 1) / kMaxParts;
    a->parts = bias && a->V >= 98304u && a->part_vecs < (1u << 15) && a->rows <= 32 ? kMaxParts : 1;  // counts in 18 bits
    a->list_room = a->part_vecs * 8 < 2 * kSide ? a->part_vecs * 8 : 2 * kSide;   // quadruples
}

// Workspace words (8 bytes) of rows in parts.
int64_t part_words(const SampleArgs& a)
{
    return a.parts > 1 ? (int64_t)a.rows * a.parts * (2 + (a.list_room + 1) / 2) : 0;
}

// Rows of one launch: a grid has fewer than 2^32 threads.
constexpr uint32_t kMostRows = 1u << 21;

template <int THREADS, bool VEC, bool BIAS>
hipError_t launch_rows(SampleArgs a, hipStream_t stream)
{
    for (a.first = 0; a.first < a.rows; a.first += kMostRows) {
        const uint32_t n = a.rows - a.first < kMostRows ? a.rows - a.first : kMostRows;
        hipLaunchKernelGGL((sample_kernel<THREADS, VEC, BIAS>), dim3(n), dim3(THREADS), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool VEC, bool BIAS>
hipError_t launch_sample(const SampleArgs& a, hipStream_t stream)
{
    if (a.parts > 1) {
        hipLaunchKernelGGL((count_kernel<VEC, BIAS>), dim3(a.rows * a.parts), dim3(kThreads), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((draw_kernel<VEC, BIAS>), dim3(a.rows), dim3(kDrawThreads), 0, stream, a);
        return hipGetLastError();
    }
    // 512 threads: two rows to a compute unit (480 rows of 152064: 73 us, 112 with
    // 1024), or short ones (2000 logits: 12 us and 14).  1024 else (200 rows of
    // 152064: 41 us, 50 with 512).
    if (a.rows > kUnits || a.V <= 32768u) return launch_rows<kThreads, VEC, BIAS>(a, stream);
    return launch_rows<kDrawThreads, VEC, BIAS>(a, stream);
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
    a.first = 0;
    plan_parts(&a, bias != nullptr);
    if (a.parts > 1) {
        // Without the memory, or in a capture that would have to allocate it, the
        // rows go in one part each: the same draws, later.
        uint64_t* table = nullptr;
        const int rc = xpress::workspace_table(stream, part_words(a), &table);
        if (rc == XPRESS_OK) {
            a.infos = reinterpret_cast<uint4*>(table);
            a.lists = reinterpret_cast<uint32_t*>(a.infos + (int64_t)a.rows * a.parts);
        } else if (rc == XPRESS_ENOMEM || rc == XPRESS_ECAPTURE) {
            a.parts = 1;
        } else {
            return rc;
        }
    }
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

extern "C" int xpress_sample_reserve(int64_t N, int64_t B, int64_t V, hipStream_t stream)
{
    if (N < 0 || B < 1 || V < 1 || V > 0x7FFFFFFFll) return XPRESS_EINVAL;
    if (B - 1 > 0 && N > 0x7FFFFFFFll / (B - 1)) return XPRESS_EINVAL;
    SampleArgs a = {};
    a.rows = (uint32_t)(N * (B - 1));
    a.V = (uint32_t)V;
    if (a.rows == 0) return XPRESS_OK;
    plan_parts(&a, true);
    if (a.parts == 1) return XPRESS_OK;
    uint64_t* table = nullptr;
    return xpress::workspace_table(stream, part_words(a), &table);
}
