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
// sum over the vocabulary.  A workgroup of 512 threads takes a row.
//
// Bins.  Magnitudes of 2^-26 to 2^16 have a 32-bit count each, for either sign:
// 43 KB, so that two workgroups share a compute unit and one streams its row
// while the other draws.  Values below -c are not counted, c = 2^12 or more by
// the temperature: next to a maximum above -c / 2 their weight is at most
// exp(-746), 0 in 64 bits (masks are such values, and counting them would send
// every lane to one word).  A row with anything else (a tinier value that is
// not 0, 2^16 or more, a maximum too low, a temperature above 43) is counted
// again over all 65536 values, in seven windows of the order, a pass for each.
//
// The j-th id.  While the row goes by, the largest of each 16 logits is kept
// (in 16 bits; a run doubles with every doubling of the row past 163840): only
// runs that reach the drawn value are read again, for a likely token a few
// hundredths of the row.
//
// The order's walk goes by segments of 64 values, largest first.  A wave takes
// a segment at a time, one value per lane.
//
// Measured (V = 152064): 480 rows with bias 88 us, 3.3 TB/s; 15 rows 57 us; one row
// without bias 37 us, the time of one workgroup from load to draw.

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
constexpr uint32_t kInf = 0x7F80u;               // magnitude bits of infinity
constexpr uint32_t kOne = 0x3F80u;               // of 1
constexpr uint32_t kLeast = kOne - 26u * 128u;   // of 2^-26
constexpr uint32_t kRels = 42u * 128u;           // magnitudes up to 2^16: 1 .. kRels; 0 is zero
constexpr uint32_t kHuge = kRels + 1;            // all from 2^16 on
constexpr uint32_t kSide = 5440;                 // bins of a sign, whole segments
constexpr uint32_t kWindow = 10240;              // of the 65536 values, whole segments
constexpr uint32_t kKeys = 10240;
constexpr uint32_t kSegs = 1024;
static_assert(kSide % 64 == 0 && kSide > kHuge && kWindow <= 2 * kSide && kWindow % 64 == 0, "bins");

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
    __align__(16) uint32_t bins[2 * kSide + 64];   // then a word a lane for what is not counted
    uint16_t keys[kKeys];    // largest logit of a run, as int16 bits
    double mass[kSegs];      // mass of a segment; then: of all segments before it
    uint32_t count[kSegs];   // the same for logits
    double wave_mass[kWaves];
    double wave_min[kWaves];
    uint32_t wave_count[kWaves];
    uint32_t wave_low[kWaves];
    int32_t wave_high[kWaves];
    uint16_t turns[kWaves][kKeys / 64 / kWaves + 1];
    double f64;
    uint32_t found, counted;
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

// Counts one vector into the bins; logits with bits from cut on go to a word of
// the lane's own instead.  No branch a logit, the arithmetic on pairs: the LDS
// takes an add of a wave in 15 cycles or so, and this keeps up with it.  Returns
// the vector's largest logit as an int16 (right where it is not negative);
// *least: the smallest magnitude less 1 (so that zero does not count).
__device__ __forceinline__ int32_t tally(Shared& s, const u32x4& z, uint32_t cut, u16x2* least)
{
    const u16x2 dump = (u16x2)(uint16_t)((2 * kSide + (threadIdx.x & 63)) * 4);
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
        r = __builtin_elementwise_min(r, (u16x2)(uint16_t)kHuge);
        const u16x2 side = __builtin_bit_cast(u16x2, (i16x2)(h >> (i16x2)15)) & (u16x2)(uint16_t)kSide;
        r = (r + side) << (u16x2)2;
        u16x2 over = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, two), (u16x2)(uint16_t)(cut - 1));
        over = (u16x2)0 - __builtin_elementwise_min(over, (u16x2)1);
        at[w] = __builtin_bit_cast(uint32_t, (u16x2)((r & ~over) | (dump & over)));
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
template <bool VEC, bool BIAS, bool FULL>
struct Row {
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
                s.found = seg * 64 + lane;
                s.counted = (uint32_t)j;
                s.f64 = w / kept;
            }
        }
        __syncthreads();
        *want = bits_at(s.found);
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

template <bool VEC, bool BIAS>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(SampleArgs a)
{
    __shared__ Shared s;
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid / 64;
    const uint32_t V = a.V, vecs = (V + 7) / 8;
    // logits of a run: 16 << wide; none where even a wave's vectors are too few
    uint32_t wide = 0;
    while ((vecs + (2u << wide) - 1) >> (wide + 1) > kKeys) ++wide;
    const bool keyed = wide <= 5;

    const uint32_t r = blockIdx.x;
    const float temp = a.temperature[r];
    const bool greedy = !(temp > 0.0f);
    const double t = greedy ? 1.0 : (double)temp, inv = 1.0 / t;
    const Logits<VEC, BIAS> z{a.base + (int64_t)r * a.stride_base,
                              BIAS ? a.bias + (int64_t)r * a.stride_bias : nullptr, V};
    int64_t* dst = a.blk + (r + r / a.bm1 + 1);

    // 1. count.  The cut c is 2^12 .. 2^16, at least 1492 temperatures.
    uint32_t c = kOne + 12u * 128u;
    while (c < kOne + 16u * 128u && (double)value_of(c) < 1492.0 * t) c += 128u;
    const uint32_t cut = 0x8000u | c;
    for (uint32_t i = tid * 4; i < 2 * kSide; i += kThreads * 4) {
        *reinterpret_cast<u32x4*>(&s.bins[i]) = u32x4{0, 0, 0, 0};
    }
    constexpr int kAhead = BIAS ? 4 : 8;     // vectors of a thread in flight
    u32x4 got[kAhead], add[kAhead];
    const uint32_t whole = VEC ? V / 8 : 0;  // vectors that are loaded whole
    // loads are queued always (past the row, its last vector again)
    auto fetch = [&](int x, uint32_t v) {
        const uint32_t e = min(v, whole - 1) * 8;
        got[x] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(z.base + e));
        if constexpr (BIAS) add[x] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(z.bias + e));
    };
    u16x2 least = {0xFFFFu, 0xFFFFu};
    int32_t high = INT16_MIN;
    auto take = [&](const u32x4& y, uint32_t v) {
        int32_t key = tally(s, y, cut, &least);
        high = max(high, key);
        if (keyed) {
            key = max(key, (int32_t)dpp_u32<0xB1>((uint32_t)key));   // lane ^ 1
            for (uint32_t d = 2; d < 2u << wide; d <<= 1) key = max(key, __shfl_xor(key, d));
            if ((v & ((2u << wide) - 1)) == 0 && v < vecs) s.keys[v >> (wide + 1)] = (uint16_t)key;
        }
    };
    if (VEC && whole > 0) {
#pragma unroll
        for (int x = 0; x < kAhead; ++x) fetch(x, tid + x * kThreads);
    }
    __syncthreads();
    // Every lane takes part in every vector (as NaN past the row), for the runs.
    const uint32_t round = (vecs + kThreads - 1) / kThreads * kThreads;
    auto arrived = [&](int x) {
        u32x4 y = got[x];
        if constexpr (BIAS) {
#pragma unroll
            for (int w = 0; w < 4; ++w) y[w] = add_round2(y[w], add[x][w]);
        }
        return y;
    };
    uint32_t done = 0;  // vectors of all threads
    if (VEC) {
        for (; done + kAhead * kThreads <= whole; done += kAhead * kThreads) {
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const u32x4 y = arrived(x);
                const uint32_t v = done + x * kThreads + tid;
                fetch(x, v + kAhead * kThreads);
                take(y, v);
            }
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            if (whole > 0 && done < whole) {
                const uint32_t v = done + tid;
                take(v < whole ? arrived(x) : z.at(min(v * 8, V)), v);
                done += kThreads;
            }
        }
    }
    for (; done < round; done += kThreads) take(z.at(min((done + tid) * 8, V)), done + tid);
    const uint32_t low = min((uint32_t)least.x, (uint32_t)least.y);
    {
        uint32_t l = low;
        int32_t h = high;
        for (int m = 32; m; m >>= 1) {
            l = min(l, __shfl_xor(l, m));
            h = max(h, __shfl_xor(h, m));
        }
        if (lane == 0) {
            s.wave_low[wave] = l;
            s.wave_high[wave] = h;
        }
    }
    __syncthreads();
    uint32_t tiny = 0xFFFFu;
    for (uint32_t w = 0; w < kWaves; ++w) {
        tiny = min(tiny, s.wave_low[w]);
        high = max(high, s.wave_high[w]);
    }

    // 2. choose a value
    uint32_t want = 0, nth = 0;
    double p = 0.0;
    bool usual = tiny >= kLeast - 1 && s.bins[kHuge] == 0 && 1492.0 * t <= (double)value_of(c);
    if (usual) {
        Row<VEC, BIAS, false> row{s, z, 0, 0, 0.0, t, inv};
        // a positive maximum is known already
        const uint32_t top = high > 0 ? kSide - 1 - ((uint32_t)high - (kLeast - 1)) : row.find_top();
        const uint32_t h = row.bits_at(top);
        usual = top < row.kOrder && (h < 0x8000u || (h & 0x7FFFu) < c - 128u);
        if (usual) {
            row.top = top;
            row.zmax = (double)value_of(h);
            p = row.choose(a, r, greedy, &want, &nth);
        }
    }
    if (!usual) {
        Row<VEC, BIAS, true> row{s, z, 0xFFFFu, 0, 0.0, t, inv};
        const uint32_t top = row.find_top();
        if (top >= row.kOrder) {  // nothing but NaN and -inf
            if (tid == 0) {
                *dst = 0;
                if (a.prob) a.prob[r] = 0.0f;
            }
            return;
        }
        row.top = top;
        row.zmax = (double)value_of(all_bits_at(top));
        p = row.choose(a, r, greedy, &want, &nth);
    }
    __syncthreads();

    // 3. the nth id (in id order) that holds the value, among the runs that reach
    // it: a wave lists those of its share in order, counts their matches 64 runs
    // at a time, and the one with the id looks at its 64 again.
    if (usual && keyed && want > 0 && want < 0x8000u) {
        const uint32_t runs = (vecs + (2u << wide) - 1) >> (wide + 1);
        const uint32_t share = (runs + kWaves * 64 - 1) / (kWaves * 64) * 64, first = wave * share;
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
                        if (a.prob) a.prob[r] = (float)p;
                        break;
                    }
                    left -= k;
                }
            }
        }
        return;
    }
    // Else each wave counts its share of the row, then the share with the id
    // is walked.
    const uint32_t steps = (V + kWaves * 512 - 1) / (kWaves * 512);  // of 512 logits per wave
    uint32_t mine = 0;
    for (uint32_t i = 0; i < steps; i += 4) {
        u32x4 y[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t e = (wave * steps + i + x) * 512 + lane * 8;
            y[x] = z.at(i + x < steps ? min(e, V) : V);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) mine += __popc(matches(y[x], want));
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
            const uint32_t m = e < V ? matches(z.at(e), want) : 0, n = __popc(m);
            uint32_t to = n;
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t o = __shfl_up(to, d);
                if ((int)lane >= d) to += o;
            }
            const uint32_t all = __shfl(to, 63);
            if (left < all) {
                if (to - n <= left && left < to) {
                    *dst = (int64_t)(e + nth_bit(m, left - (to - n)));
                    if (a.prob) a.prob[r] = (float)p;
                }
                break;
            }
            left -= all;
        }
    }
}

template <bool VEC, bool BIAS>
hipError_t launch_sample(const SampleArgs& a, hipStream_t stream)
{
    hipLaunchKernelGGL((sample_kernel<VEC, BIAS>), dim3(a.rows), dim3(kThreads), 0, stream, a);
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
