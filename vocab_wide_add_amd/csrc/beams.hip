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
// fp32, z Lh - r too but for logits much smaller than the largest, and the rest is a
// factor 1 + (z - m) Ll ln 2, summed beside: sum y and sum y z, of which the second
// enters once, in 64 bits.  What is left is the error of the hardware's 2^x, about
// 2^-24 a term and not all of one sign.  Threads' sums meet
// as 64-bit numbers, with powers of two as factors.  Where a part's largest |z| is
// 2^13 or more, neighbouring bf16 values are 64 or more apart, and the sum is the count
// of the largest.
//
// The K largest.  The largest of every eight logits, a run, goes to LDS as the row goes
// by.  The K-th largest of the threads' maxima, T0, is below K logits; runs above it
// are few, and where they are K or more the K-th largest of theirs is T.  The runs
// above T, and the first K in order that reach T, are read again; their logits not
// below T are ranked by counting.  Ties cost no more than anything else.
//
// Bound by the bytes for many rows; by the two launches and the chain of one workgroup
// for few.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "device_common.h"
#include "host_common.h"
#include "kv_common.h"
#include "xpress_argmax.h"

namespace {

using namespace xpress;

constexpr uint32_t kThreads = 512;
constexpr uint32_t kWaves = kThreads / 64;
constexpr uint32_t kRuns = 16384;          // of a part: 131072 logits
constexpr uint32_t kMostK = 128;
constexpr uint32_t kAbove = 4096;          // runs above T0: fewer than K threads', 32 each
constexpr uint32_t kFound = 2304;          // logits that are ranked
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
    float y = 0.0f, yz = 0.0f, r = -kFarMost;

    __device__ __forceinline__ void add(const float* z, float top)
    {
        if (top * kLh > r + 16.0f) {   // (not for +inf past the first time: r is bounded)
            const float to = fminf(rintf(top * kLh), kFarMost);
            if (to > r) {
                y = ldexpf(y, (int)(r - to));
                yz = ldexpf(yz, (int)(r - to));
                r = to;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // no infinity: 0 times it would be NaN (a NaN logit becomes -3e38 too)
            const float x = fmaxf(z[i], -3e38f);
            const float e = __builtin_amdgcn_exp2f(fmaf(x, kLh, -r));
            y += e;
            yz = fmaf(e, x, yz);
        }
    }
};

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    return v;
}

struct PartShared {
    uint16_t runs[kRuns];
    uint32_t above[kAbove];              // runs above T0
    uint64_t found[kFound];
    uint32_t maxima[kThreads];
    uint32_t firsts[kMostK];
    uint32_t counts[kWaves];
    double part[kWaves];
    uint32_t n_above, n_found, threshold, counted;
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

template <bool VEC, bool BIAS>
__global__ void __launch_bounds__(kThreads) part_kernel(BeamArgs a)
{
    __shared__ PartShared s;
    const uint32_t unit = a.first + blockIdx.x, tid = threadIdx.x;
    const uint32_t row = unit / a.parts, part = unit - row * a.parts;
    const Row<VEC, BIAS> z = {a.base + row * a.stride_base, BIAS ? a.bias + row * a.stride_bias : nullptr, a.V};
    const uint32_t all_vecs = (a.V + 7) / 8, vec0 = part * a.part_vecs;
    const uint32_t vecs = vec0 < all_vecs ? min(a.part_vecs, all_vecs - vec0) : 0;

    Sum sum;
    uint32_t best = 0;   // the thread's largest, in the order
    for (uint32_t i = tid; i < vecs; i += kThreads) {
        const u32x4 v = z.at((vec0 + i) * 8);
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
    }
    if (tid == 0) s.n_above = s.n_found = s.threshold = s.counted = 0;
    s.maxima[tid] = best;
    __syncthreads();

    // T0: the K-th largest of the threads' maxima
    uint32_t better = 0, most = 0;
    for (uint32_t i = 0; i < kThreads; ++i) {
        const uint32_t o = s.maxima[i];
        better += o > best;
        most = max(most, o);
    }
    // the largest value that fewer than K maxima pass but K or more reach
    if (better < a.K) {
        uint32_t equal = 0;
        for (uint32_t i = 0; i < kThreads; ++i) equal += s.maxima[i] == best;
        if (better + equal >= a.K) s.threshold = best;
    }
    __syncthreads();
    uint32_t low = s.threshold;   // 0: fewer than K threads have a logit
    uint32_t span = (vecs + kThreads - 1) / kThreads;   // runs of a thread, one after the other
    const uint32_t run0 = min(tid * span, vecs), run1 = min(run0 + span, vecs);
    for (uint32_t i = run0; i < run1; ++i) {
        if (s.runs[i] > low) {
            const uint32_t at = atomicAdd(&s.n_above, 1u);
            if (at < kAbove) s.above[at] = i;
        }
    }
    __syncthreads();
    const uint32_t n0 = s.n_above;
    __syncthreads();
    if (n0 >= a.K) {
        // T: the K-th largest of these runs' maxima
        for (uint32_t i = tid; i < n0; i += kThreads) {
            const uint32_t o = s.runs[s.above[i]];
            uint32_t more = 0, same = 0;
            for (uint32_t j = 0; j < n0; ++j) {
                const uint32_t p = s.runs[s.above[j]];
                more += p > o;
                same += p == o;
            }
            if (more < a.K && more + same >= a.K) s.threshold = o;
        }
        __syncthreads();
        low = s.threshold;
    }
    // the first K runs, in order, whose largest is T (none where T is none)
    uint32_t reach = 0;
    for (uint32_t i = run0; i < run1; ++i) reach += low > 0 && s.runs[i] == low;
    uint32_t reached;
    uint32_t at = ranks(reach, s.counts, &reached);
    for (uint32_t i = run0; i < run1 && at < a.K; ++i) {
        if (low > 0 && s.runs[i] == low) s.firsts[at++] = i;
    }
    __syncthreads();
    reached = min(reached, a.K);
    // their logits from T on
    for (uint32_t i = tid; i < n0 + reached; i += kThreads) {
        const uint32_t run = i < n0 ? s.above[i] : s.firsts[i - n0];
        if (i < n0 && s.runs[run] <= low) continue;
        const uint32_t e = (vec0 + run) * 8;
        const u32x4 v = z.at(e);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const float f = x & 1 ? bf16_hi(v[x / 2]) : bf16_lo(v[x / 2]);
            const uint32_t o = order_of(f);
            if (o > 0 && o >= low) {
                const uint32_t to = atomicAdd(&s.n_found, 1u);
                if (to < kFound) s.found[to] = (uint64_t)o << 32 | (kNoIndex - (e + x));
            }
        }
    }
    __syncthreads();
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
        // 2^(z L - r) against 2^(m L - R): R the integer next to m L
        const double R = rint((double)m * (double)kLh);
        double v = ((double)sum.y + kRest * kLn2 * ((double)sum.yz - (double)m * (double)sum.y));
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

// A candidate of the join.
struct Candidate {
    double score;
    uint64_t rest;   // larger first: row, then logit and id

    __device__ __forceinline__ bool before(const Candidate& o) const
    {
        return score > o.score || (score == o.score && rest > o.rest);
    }
};

__device__ __forceinline__ Candidate better_of(const Candidate& x, const Candidate& y)
{
    return x.before(y) ? x : y;
}

// A workgroup takes a sequence: every list's first candidate that is not taken yet
// meets the others', K times.
__global__ void __launch_bounds__(kJoinThreads) join_kernel(BeamArgs a)
{
    extern __shared__ double shift[];   // of a beam: its score less the log of its sum, and its largest
    __shared__ double win_score[kJoinThreads / 64];
    __shared__ uint64_t win_key[kJoinThreads / 64];
    const uint32_t n = a.first + blockIdx.x, tid = threadIdx.x;
    const uint32_t lists = a.beams * a.parts;
    double* top = shift + a.beams;
    uint32_t* taken = reinterpret_cast<uint32_t*>(top + a.beams);   // of each list
    for (uint32_t i = tid; i < lists; i += kJoinThreads) taken[i] = 0;
    for (uint32_t b = tid; b < a.beams; b += kJoinThreads) {
        const int64_t unit = (int64_t)(n * a.beams + b) * a.parts;
        uint32_t o = 0;
        for (uint32_t p = 0; p < a.parts; ++p) o = max(o, (uint32_t)(a.lists[(unit + p) * a.K] >> 32));
        const double m = (double)value_at(o);
        double total = 0.0;
        for (uint32_t p = 0; p < a.parts; ++p) {
            const uint32_t q = (uint32_t)(a.lists[(unit + p) * a.K] >> 32);
            if (q) total += a.sums[unit + p] * (q == o ? 1.0 : exp((double)value_at(q) - m));
        }
        const double score = (double)a.scores[n * a.beams + b];
        const bool lives = o && fabs(score) < INFINITY;
        shift[b] = lives ? score - log(total) : -INFINITY;
        top[b] = m;
    }
    __syncthreads();
    for (uint32_t k = 0; k < a.K; ++k) {
        Candidate mine = {-INFINITY, 0};
        uint32_t list = ~0u, beam = 0;
        uint64_t key = 0;
        for (uint32_t l = tid; l < lists; l += kJoinThreads) {
            const uint32_t at = taken[l];
            if (at >= a.K) continue;
            const uint32_t b = l / a.parts;
            const uint64_t x = a.lists[((int64_t)n * lists + l) * a.K + at];
            if (x == 0 || shift[b] == -INFINITY) continue;
            const float z = value_at((uint32_t)(x >> 32));
            const double d = (double)z == top[b] ? 0.0 : (double)z - top[b];
            if (d == -INFINITY) continue;   // beside +inf
            // 16 bits of the beam, reversed, above the key's 48
            const Candidate c = {shift[b] + d, (uint64_t)(65535u - b) << 48 | x};
            if (list == ~0u || c.before(mine)) {
                mine = c;
                list = l;
                beam = b;
                key = x;
            }
        }
        Candidate w = list == ~0u ? Candidate{-INFINITY, 0} : mine;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const Candidate o = {__shfl_xor(w.score, d), (uint64_t)__shfl_xor((unsigned long long)w.rest, d)};
            w = better_of(w, o);
        }
        if ((tid & 63) == 0) {
            win_score[tid / 64] = w.score;
            win_key[tid / 64] = w.rest;
        }
        __syncthreads();
        w = Candidate{win_score[0], win_key[0]};
        for (uint32_t i = 1; i < kJoinThreads / 64; ++i) w = better_of(w, Candidate{win_score[i], win_key[i]});
        const int64_t to = (int64_t)n * a.K + k;
        if (w.rest == 0) {   // nothing is left
            if (tid == 0) {
                a.best[to] = -INFINITY;
                a.rows_out[to] = -1;
                a.ids[to] = -1;
            }
        } else if (list != ~0u && mine.rest == w.rest) {
            taken[list] += 1;
            a.best[to] = (float)w.score;
            a.rows_out[to] = (int32_t)(n * a.beams + beam);
            a.ids[to] = key_index(key);
        }
        __syncthreads();
    }
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

// Parts: two workgroups a compute unit where the rows alone are fewer, but no part of
// fewer vectors than a workgroup has threads; and none that has more than kRuns.
Plan plan_of(const Shape& s)
{
    const int64_t vecs = (s.V + 7) / 8, rows = s.N * s.beams;
    int64_t parts = (vecs + kRuns - 1) / kRuns;
    const int64_t fill = (2 * 256 + rows - 1) / rows, fits = vecs / kThreads;
    const int64_t more = fill < fits ? fill : fits;
    if (more > parts) parts = more;
    Plan p;
    p.part_vecs = (vecs + parts - 1) / parts;
    p.parts = (vecs + p.part_vecs - 1) / p.part_vecs;
    return p;
}

int64_t words_of(const Shape& s, const Plan& p) { return s.N * s.beams * p.parts * (s.K + 1); }

// LDS of a sequence's beams and lists in the join.
int64_t join_bytes(const Shape& s, const Plan& p) { return s.beams * 16 + s.beams * p.parts * 4; }

bool plan_ok(const Shape& s, const Plan& p)
{
    return s.N * s.beams <= kMost / p.parts && join_bytes(s, p) <= 60 * 1024;
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
        hipLaunchKernelGGL(join_kernel, grid, block, (size_t)join_bytes(s, p), stream, a);
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
    // what is written lies apart from what any of them reads or writes
    for (int64_t i = 0; i < count; ++i) {
        const xpress_beam_state& x = states[i];
        if (x.bytes == 0) continue;
        const size_t nx = span(M, x.step_to, x.bytes);
        for (int64_t j = 0; j < count; ++j) {
            const xpress_beam_state& y = states[j];
            if (y.bytes == 0) continue;
            if (y.from && ranges_overlap(x.to, nx, y.from, span(N, y.step_from, y.bytes))) return XPRESS_EINVAL;
            if (j < i && ranges_overlap(x.to, nx, y.to, span(M, y.step_to, y.bytes))) return XPRESS_EINVAL;
        }
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
