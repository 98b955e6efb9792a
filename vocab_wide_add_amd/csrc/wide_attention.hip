// wide_attention.hip -- the sparse form of the attention for more than 64 rows (queries
// times query heads) a key-value head: 32 rows to a wave (gfx950, MFMA 32x32).
//
// As attention.h with LDS stages, but a wave has twice the rows, so that the operands
// which it takes from LDS serve twice as much; values are transposed on their way out of
// LDS; keys' places are found a few stages ahead in a ring of eight stages instead of a
// table, so that a part may be as long as it likes; and the parts are taken by size.  A
// workgroup's four waves hold 128 rows.  With lane l = 32 g + c:
//
//   S^T = K Q^T   v_mfma_f32_32x32x16: A = keys (lane: key c, 8 dims), B = queries
//                 (lane: row c).  The lane gets the scores of row c with keys
//                 8 (i / 4) + 4 g + i % 4: a row's state lives in two lanes.
//   O^T += V^T P  P^T is already in B's layout: slot 8 g + e of step h is key
//                 16 h + 8 (e / 4) + 4 g + e % 4.  A = V^T: dim 32 j + c of the lane's
//                 eight keys for product j, by transposing loads (take_value).
//
// The loop's registers are full: whatever the compiler would have to fetch back from
// memory inside it, and page ids in registers too, would wait for every copy on its way,
// so that places are worked out again where they are needed, the careful form takes few,
// and page ids come by LDS.
//
// Measured (32 query and 8 key-value heads of 128, bf16): 64 nodes of 32 sequences up to
// 4096 tokens 158 to 190 us by their lengths and 11 to 13 for the join (16 rows a wave
// 200 where this took 162): 0.7 PFLOP/s
// with the weights' second part, and 0.34 GB of cache that two workgroups each read.
// Without products and weights the copies take 90, without copies the rest 125.  77 rows of heads
// of 64 on an e4m3 cache, 48 sequences up to 6001: 68 and 5 under the profiler, the whole
// call 69 (100 with 16 rows; 73 with the transposition in registers, and 84 with each value
// row's place in LDS worked out by itself).  4096 new tokens of one sequence under a window
// and sinks: 438 us for a window of 4096, where their products take 107 at the library's
// rate, and 459 for one of 1024, where they take 47: every 128 rows go through the keys of all.  Which
// calls come here: see plan_of.  Tried: eight
// waves of 32 rows, which read the cache once, 205 for the 187; weights of one tile
// beside the products of the next 209; three workgroups a compute unit at 64 dims: no
// change.
//
// A negative scale turns the queries' signs and a scale of zero the queries into zeros
// (what is not finite of them into NaN, as 0 times it is), so that the largest score is
// the largest product, and weights are 2^(s scale - m) by one fused step.
#include "attention.h"

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
typedef int16_t i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i32x2 LocalI32x2;
typedef __attribute__((address_space(3))) i16x4 LocalI16x4;

constexpr uint32_t kRing = 8;      // stages whose keys' places are known

template <bool FP16>
__device__ __forceinline__ f32x16 mfma32(u32x4 x, u32x4 y, f32x16 c)
{
    if constexpr (FP16) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c,
                                                      0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y),
                                                       c, 0, 0, 0);
    }
}

// A value row's pieces (16 bytes) go to piece ^ value_turn(row) in LDS, so that the rows
// of which 32 lanes read 32 dims at once (four in a row, e4m3 twice four, eight apart) lie
// in different banks.
template <bool E4M3, int DP>
__device__ __forceinline__ uint32_t value_turn(uint32_t row)
{
    constexpr uint32_t kRow = DP * (E4M3 ? 1 : 2);   // 256 bytes: all banks
    const uint32_t r = kRow >= 256 ? row & 3 : kRow == 128 ? row >> 1 & 1 : 0;
    constexpr uint32_t kBits = kRow >= 256 ? 2 : kRow == 128 ? 1 : 0;
    return E4M3 ? (r | (row >> 3 & 1) << kBits) * 2 : r * 4;
}

// The two lanes of a row.
__device__ __forceinline__ float pair_max(float v) { return fmaxf(v, __shfl_xor(v, 32)); }

template <bool FP16, bool E4M3, int DP>
struct WideTile {
    using H = Half<FP16>;
    using S = Lines<E4M3, DP>;
    static constexpr int kSteps = DP / 16;              // products of the scores
    static constexpr int kLoads = E4M3 ? DP / 32 : DP / 16;   // 16-byte pieces of a key row per lane
    static constexpr int kOuts = DP / 32;               // of the output
    static constexpr int kWords = E4M3 ? 2 : 4;         // 32-bit words of eight keys' values

    const AttnArgs& a;
    uint32_t c, g;
    u32x4 q[kSteps];
    f32x16 o[kOuts];
    float m, l, scale;
    // the row and what it sees, as in attention.h
    int32_t few, gap, past, place0, query, pos;
    uint64_t nodes;
    const uint32_t *words, *tree;

    static __device__ __forceinline__ uint32_t key_of(int i, uint32_t g) { return (uint32_t)(i / 4) * 8 + g * 4 + i % 4; }

    // First of the eight dims that lane half g supplies to step i.
    __device__ __forceinline__ uint32_t dim_of(int i) const
    {
        return E4M3 ? (uint32_t)(i / 2) * 32 + g * 16 + (uint32_t)(i % 2) * 8 : (uint32_t)i * 16 + g * 8;
    }

    __device__ __forceinline__ int32_t key_at(int32_t i) const { return i >= few ? i + gap : i; }

    __device__ __forceinline__ bool near(int32_t key, int32_t at) const
    {
        return a.window == 0 || (int64_t)key > (int64_t)at - a.window || key < a.sinks;
    }

    __device__ __forceinline__ bool sees(int32_t i) const
    {
        const int32_t key = key_at(i);
        if (!a.tree) return key <= pos && near(key, pos);
        if (key < place0) return key < past && near(key, pos);
        const uint32_t node = (uint32_t)(key - place0);
        if (node < 64) return nodes >> node & 1;
        return query >= 0 && node < a.Q && (words[node / 32] >> (node % 32) & 1);
    }

    // What query i sees (-1: nothing).
    __device__ __forceinline__ void turn_to(int32_t i)
    {
        query = i;
        past = i < 0 ? INT32_MIN : place0;
        pos = i < 0 ? INT32_MIN : place0 + i;
        nodes = 0;
        if (i < 0 || !a.tree) return;
        words = tree + i * a.tree_i;
        const uint32_t count = (a.Q + 31) / 32;
        uint32_t size = 0;
        for (uint32_t w = 0; w < count; ++w) {
            const uint32_t left = a.Q - w * 32, x = words[w] & (left < 32 ? (1u << left) - 1 : ~0u);
            size += __popc(x);
            if (w < 2) nodes |= (uint64_t)x << (32 * w);
        }
        pos = place0 + (int32_t)size - 1;
    }

    __device__ __forceinline__ void reset()
    {
        m = kNone;
        l = 0.0f;
#pragma unroll
        for (int j = 0; j < kOuts; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;
    }

    // Which of the tile's keys the lane's row sees, a bit a key; the row's lanes then look
    // at their 16 of them.  key0: the number of the first.
    __device__ __forceinline__ uint32_t seen(uint32_t exist, int32_t key0) const
    {
        if (gap > 0 && key0 < few && key0 + kTile > few) {
            // the sinks end within the tile
            uint32_t bits = 0;
#pragma unroll 1
            for (int32_t i = 0; i < kTile; ++i) bits |= (uint32_t)sees(key0 + i) << i;
            return exist & bits;
        }
        const int32_t key = key_at(key0);
        auto below = [](int64_t n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };   // the first n bits
        // up to the query, or in a tree all that came before it
        uint32_t bits = below((a.tree ? (int64_t)past : (int64_t)pos + 1) - key);
        if (a.window > 0) bits &= ~below((int64_t)pos - a.window + 1 - key) | below((int64_t)a.sinks - key);
        const int64_t node = (int64_t)key - place0;   // of the first key
        if (a.tree && query >= 0 && node > -32 && node < (int64_t)a.Q) {
            if (node < 0) {
                bits |= (uint32_t)nodes << -node;
            } else if (a.Q <= 64) {
                bits |= (uint32_t)(nodes >> node);
            } else {
                const uint32_t w = (uint32_t)node / 32, sh = (uint32_t)node % 32, size = (a.Q + 31) / 32;
                const uint64_t two = (uint64_t)(w + 1 < size ? words[w + 1] : 0) << 32 | words[w];
                bits |= (uint32_t)(two >> sh) & below((int64_t)a.Q - node);
            }
        }
        return exist & bits;
    }

    // Weights of a tile from its products with the queries: P as two 16-bit parts of each
    // step.  on: which of the tile's keys the row sees; all: every row of the wave sees every key.
    // (The empty assembly here and below keeps what a uniform branch holds in it: made
    // into selects it was 80 of 340 instructions a tile.)
    __device__ __forceinline__ void weigh(f32x16 s, bool all, uint32_t on, u32x4 (&big)[2], u32x4 (&rest)[2])
    {
        if (!all) {
            asm volatile("");
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = on >> key_of(i, g) & 1 ? s[i] : kNone;
        }
        float top = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
        top *= scale;
        if (__any(top > m + H::kRise)) {
            const float to = fmaxf(m, pair_max(top));
            const float f = to == m ? 1.0f : exp2_fast(m - to);
            m = to;
            l *= f;
#pragma unroll
            for (int j = 0; j < kOuts; ++j) o[j] *= f;
        }
        const float from = (m == kNone ? 0.0f : m) - H::kLift;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int i = 8 * h + 2 * p;
                const float w0 = exp2_fast(fmaf(s[i], scale, -from)), w1 = exp2_fast(fmaf(s[i + 1], scale, -from));
                l += w0 + w1;
                const uint32_t w = H::pack(w0, w1);
                big[h][p] = w;
                rest[h][p] = H::pack(w0 - H::lo(w), w1 - H::hi(w));
            }
    }

    // The A operand of product j, step h, from LDS: dim 32 j + c of the lane's eight keys, by
    // transposing loads.  Sixteen lanes give the addresses of 16 dims of four keys, eight
    // bytes each (e4m3: of eight keys), and each gets one dim of all of them.  at: the
    // lane's offset at j = 0, see value_at.
    template <int W>
    static __device__ __forceinline__ void take_value(uint32_t (&to)[W], const char* at)
    {
        if constexpr (E4M3) {
            const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LocalI32x2*)at);
            to[0] = (uint32_t)x[0];
            to[1] = (uint32_t)x[1];
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const u32x2 x = __builtin_bit_cast(
                    u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LocalI16x4*)(at + i * 8 * S::kRow)));
                to[2 * i] = x[0];
                to[2 * i + 1] = x[1];
            }
        }
    }

    // Where the lane reads product 0's dims of step 0, from the tile's first value row;
    // product j's are that ^ j kBlock, as the rows' blocks change places (value_turn).
    static constexpr uint32_t kBlock = 32 * (E4M3 ? 1 : 2);   // bytes of 32 dims
    static __device__ __forceinline__ uint32_t value_at(uint32_t lane)
    {
        const uint32_t i = lane & 15, half = lane >> 4 & 1, g = lane >> 5;
        const uint32_t row = E4M3 ? i / 8 * 8 + g * 4 + i / 2 % 4 : g * 4 + i / 4;
        const uint32_t byte = half * (kBlock / 2) + (E4M3 ? i % 2 : i % 4) * 8;
        return row * S::kRow + (byte ^ value_turn<E4M3, DP>(row) * 16);
    }

    static __device__ __forceinline__ u32x4 operand(const uint32_t (&v)[kWords])
    {
        if constexpr (E4M3) {
            return u32x4{H::template from8<false>(v[0]), H::template from8<true>(v[0]), H::template from8<false>(v[1]),
                         H::template from8<true>(v[1])};
        } else {
            return u32x4{v[0], v[1], v[2], v[3]};
        }
    }

    // One tile whose rows are in LDS.  One path for all tiles: with two, the sums lay in
    // other registers in each and were moved between them.
    __device__ __forceinline__ void tile(const char* ks, const char* vs, bool all, uint32_t on)
    {
        // the lane's places in the tile, worked out here and not kept beside the sums
        uint32_t lane_c = c, lane_g = g;
        asm volatile("" : "+v"(lane_c), "+v"(lane_g));
        const char* krow = ks + lane_c * S::kRow;
        const uint32_t turn = S::turn(lane_c);
        u32x4 k[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            k[i] = *reinterpret_cast<const u32x4*>(krow + (((uint32_t)i * 2 + lane_g) ^ turn) * 16);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (a.D != DP) {
            asm volatile("");
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                if (dim_of(E4M3 ? 2 * i : i) >= a.D) k[i] = u32x4{0, 0, 0, 0};
            }
        }
        f32x16 s;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            u32x4 y;
            if constexpr (E4M3) {
                const uint32_t w0 = k[i / 2][(i % 2) * 2], w1 = k[i / 2][(i % 2) * 2 + 1];
                y = u32x4{H::template from8<false>(w0), H::template from8<true>(w0), H::template from8<false>(w1),
                          H::template from8<true>(w1)};
            } else {
                y = k[i];
            }
            s = mfma32<FP16>(y, q[i], s);
        }
        const uint32_t at0 = value_at(lane_g * 32 + lane_c);
        uint32_t v[2][kOuts][kWords];
#pragma unroll
        for (int j = 0; j < kOuts; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) take_value(v[h][j], vs + (at0 ^ (j * kBlock)) + h * 16 * S::kRow);
        __builtin_amdgcn_sched_barrier(0);
        u32x4 big[2], rest[2];
        weigh(s, all, on, big, rest);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int p = 0; p < kOuts / 2; ++p) {
                const u32x4 even = operand(v[h][2 * p]), odd = operand(v[h][2 * p + 1]);
                o[2 * p] = mfma32<FP16>(even, big[h], o[2 * p]);
                o[2 * p + 1] = mfma32<FP16>(odd, big[h], o[2 * p + 1]);
                o[2 * p] = mfma32<FP16>(even, rest[h], o[2 * p]);
                o[2 * p + 1] = mfma32<FP16>(odd, rest[h], o[2 * p + 1]);
            }
    }

    // The careful form (see attention.h): queries [first, last] one after the other, the
    // rows straight from the pool.  place: of key c of the tile, less than 0 where it does
    // not exist.
    __device__ __forceinline__ void tile_careful(const char* kbase, const char* vbase, int64_t place, int32_t key0,
                                              int32_t first, int32_t last)
    {
        const uint32_t exist = (uint32_t)__ballot(place >= 0);
        const char* row = kbase + (place < 0 ? 0 : place);
        auto key = [&](int i) -> u32x4 {
            u32x4 y = {0, 0, 0, 0};
            const uint32_t d = dim_of(i);
            if (d >= a.D) return y;
            if constexpr (E4M3) {
                const u32x2 x = *reinterpret_cast<const u32x2*>(row + d);
                y = u32x4{H::template from8<false>(x[0]), H::template from8<true>(x[0]),
                          H::template from8<false>(x[1]), H::template from8<true>(x[1])};
            } else {
                y = *reinterpret_cast<const u32x4*>(row + d * 2);
            }
            return y;
        };
        f32x16 s;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) s = mfma32<FP16>(key(i), q[i], s);
        u32x4 big[2], rest[2];
        weigh(s, false, seen(exist, key0), big, rest);
        const int32_t mine = query;
        for (int32_t at = first; at <= last; ++at) {
            turn_to(at);
            const uint32_t its = seen(exist, key0);
            // (one product's values at a time: more at once would take registers from the
            // loop over all tiles)
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const u32x4 bh = h ? big[1] : big[0], rh = h ? rest[1] : rest[0];
#pragma unroll
                for (int j = 0; j < kOuts; ++j) {
                    const uint32_t d = 32 * j + c;
                    uint32_t v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t k = 16 * h + key_of(e, g);
                        const uint32_t lo = __shfl((uint32_t)place, (int)k), hi = __shfl((uint32_t)(place >> 32), (int)k);
                        const bool on = d < a.D && (its >> k & 1);
                        const char* from = vbase + (on ? (int64_t)((uint64_t)hi << 32 | lo) + d * (E4M3 ? 1 : 2) : 0);
                        if constexpr (E4M3) {
                            v[e] = H::template from8<false>(*reinterpret_cast<const uint8_t*>(from));
                        } else {
                            v[e] = *reinterpret_cast<const uint16_t*>(from);
                        }
                        v[e] = on ? v[e] : 0;
                    }
                    // the weights' second part meets finite values only
                    u32x4 x, z;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t b = __builtin_amdgcn_perm(v[2 * w + 1], v[2 * w], 0x05040100u);
                        x[w] = b;
                        z[w] = ((b & H::kExp & 0xFFFFu) == (H::kExp & 0xFFFFu) ? 0 : b & 0xFFFFu) |
                               ((b & H::kExp & 0xFFFF0000u) == (H::kExp & 0xFFFF0000u) ? 0 : b & 0xFFFF0000u);
                    }
                    f32x16 r;
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = 0.0f;
                    r = mfma32<FP16>(x, bh, r);
                    r = mfma32<FP16>(z, rh, r);
                    if (mine == at) o[j] += r;
                }
            }
        }
        turn_to(mine);
    }

    __device__ __forceinline__ bool finite() const
    {
        bool ok = true;
#pragma unroll
        for (int j = 0; j < kOuts; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) ok &= __builtin_fabsf(o[j][i]) < INFINITY;
        return ok;
    }
};

// LDS stages of 64 keys and values, two to four: copies run up to three stages ahead.
template <bool E4M3, int DP>
struct Ahead : Lines<E4M3, DP> {
    using L = Lines<E4M3, DP>;
    static constexpr uint32_t kKeys = 64;
    static constexpr uint32_t kBytes = kKeys * L::kRow;                  // keys or values of a stage
    static constexpr uint32_t kRoom = DP == 256 ? 131072 : 65536;       // two workgroups a compute unit, or one
    static constexpr uint32_t kDepth = kRoom / 2 / kBytes < 4 ? kRoom / 2 / kBytes : 4;
    static constexpr uint32_t kCopies = kKeys * L::kPieces / kThreads;   // of a thread, keys or values

    // Queues the copies of a stage's keys, whose places are at `place`, to LDS byte
    // address `to`.  Rows that do not exist and pieces past the head's end: any bytes of
    // the pool, masked or dropped after.
    template <bool ONCE>
    static __device__ __forceinline__ void copy(const AttnArgs& a, const int64_t* place, const char* kbase,
                                                const char* vbase, uint32_t to, uint32_t thread)
    {
        const uint32_t used = a.D * (E4M3 ? 1 : 2);
        const uint32_t wave_at = (uint32_t)__builtin_amdgcn_readfirstlane((int)(thread / 64 * 1024));
#pragma unroll
        for (uint32_t x = 0; x < kCopies; ++x) {
            const uint32_t at = x * kThreads + thread, row = at / L::kPieces, piece = at % L::kPieces;
            const uint32_t kd = (piece ^ L::turn(row)) * 16, vd = (piece ^ value_turn<E4M3, DP>(row)) * 16;
            const uint32_t here = to + x * (kThreads * 16) + wave_at;
            dma16<ONCE>(reinterpret_cast<const uint16_t*>(kbase + place[row] + (kd < used ? kd : 0)), here);
            dma16<ONCE>(reinterpret_cast<const uint16_t*>(vbase + place[row] + (vd < used ? vd : 0)), here + kBytes);
        }
    }
};

template <bool FP16, bool E4M3, int DP, bool ONCE>
__global__ void __launch_bounds__(kThreads, DP == 256 ? 1 : 2) wide_kernel(AttnArgs a)
{
    using T = WideTile<FP16, E4M3, DP>;
    using S = Ahead<E4M3, DP>;
    using H = Half<FP16>;
    constexpr uint32_t kKeys = S::kKeys;
    __shared__ __align__(16) int64_t place[kRing * kKeys];
    __shared__ uint32_t there[kRing * 2];
    __shared__ __align__(16) uint32_t ids[kRing * kKeys];   // pages on their way to the ring
    __shared__ __align__(16) char pool[S::kDepth * 2 * S::kBytes];   // the stages
    __shared__ __align__(16) uint32_t sizes[kRanked];
    __shared__ uint32_t chosen;

    const uint32_t id = a.first + blockIdx.x;
    const uint32_t unit = id / (8 * a.groups) * 8 + id % 8, group = id / 8 % a.groups;
    if (unit >= a.units) return;
    const uint32_t tid = threadIdx.x, wave = tid / 64, lane = tid & 63;
    // The heads of a (sequence, part) follow each other on one XCD: rows of several heads
    // may share 128-byte lines.  Fewer than eight such: head by head.
    const uint32_t all = a.N * a.splits;
    uint32_t hk = unit % a.Hk, which = unit / a.Hk;
    if (all >= 8) {
        hk = unit / 8 % a.Hk;
        which = unit / (8 * a.Hk) * 8 + unit % 8;
        if (which >= all) return;
    }
    uint32_t n = which % a.N, split = which / a.N;
    if (a.N > 1 && all <= kRanked) {
        const uint32_t x = part_by_size(a, which, sizes, &chosen);
        split = x / a.N;
        n = x - split * a.N;
    }
    const uint32_t owner = n * a.Hk + hk;
    // (a workgroup whose last rows are none leaves another SIMD idle than the next)
    const uint32_t rw = (wave + unit / 8) % kWaves;
    const Keys keys = keys_of<true>(a, n);
    if (split > 0 && split >= keys.parts) return;
    const int32_t part0 = (int32_t)(split * a.chunk);
    const uint32_t count = (uint32_t)min(keys.hi - part0, (int32_t)a.chunk);   // 0: an empty sequence
    const uint32_t stages = (count + kKeys - 1) / kKeys;
    const uint32_t row0 = (group * kWaves + rw) * 32;

    // the page of the part's key j, and from it the place; less than 0: there is none
    auto key_no = [&](uint32_t j) {
        const uint32_t i = (uint32_t)part0 + j;
        return i >= (uint32_t)keys.few ? i + (uint32_t)keys.gap : i;
    };
    auto page_of = [&](uint32_t j) -> uint32_t {
        return j < count ? (uint32_t)a.page_table[(int64_t)n * a.table + key_no(j) / a.page_size] : ~0u;
    };
    auto place_of = [&](uint32_t j, uint32_t page) -> int64_t {
        if (j >= count || page >= a.pages) return -1;
        return (int64_t)page * a.page + (int64_t)(key_no(j) % a.page_size) * a.token;
    };
    auto put_place = [&](uint32_t j, int64_t at) {   // by a whole wave, j = 64 stage + lane
        const uint64_t on = __ballot(at >= 0);
        // a key that does not exist has the place of one that does, so that its value, which
        // meets a weight of zero, is as finite as the others (zeroed in the loop, values took
        // a move of every register)
        const int64_t other = on ? __shfl(at, __builtin_ctzll(on)) : 0;
        place[j % (kRing * kKeys)] = at < 0 ? other : at;
        if (lane < 2) there[j / 32 % (kRing * 2) + lane] = (uint32_t)(on >> (lane * 32));
    };
#pragma unroll
    for (uint32_t j = tid; j < kRing * kKeys; j += kThreads) put_place(j, place_of(j, page_of(j)));

    T t{a, lane & 31, lane / 32};
    {
        const float scale = a.scale * (a.k_scale ? a.k_scale[hk] : 1.0f);
        t.scale = scale == 0.0f ? 1.0f : __builtin_fabsf(scale);
        const uint32_t sign = scale < 0.0f ? 0x80008000u : 0u;
        const uint32_t r = row0 + t.c;
        const bool on = r < a.rows;
        const uint32_t i = on ? r / a.G : 0, h = hk * a.G + (on ? r - i * a.G : 0);
        t.few = keys.few;
        t.gap = keys.gap;
        t.place0 = keys.len - (int32_t)a.Q;
        t.tree = a.tree ? a.tree + n * a.tree_n : nullptr;
        t.turn_to(on ? (int32_t)i : -1);
        const uint16_t* src = a.q + n * a.q_n + i * a.q_i + h * a.q_h;
#pragma unroll
        for (int x = 0; x < T::kSteps; ++x) {
            const uint32_t d = t.dim_of(x);
            u32x4 w = {0, 0, 0, 0};
            if (on && d < a.D) {
                if (a.wide) {
                    w = *reinterpret_cast<const u32x4*>(src + d);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = src[d + 2 * e] | (uint32_t)src[d + 2 * e + 1] << 16;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (scale == 0.0f) {
                    const uint32_t lo = (w[e] & H::kExp & 0xFFFFu) == (H::kExp & 0xFFFFu) ? 0x7FFFu : 0;
                    const uint32_t hi = (w[e] & H::kExp & 0xFFFF0000u) == (H::kExp & 0xFFFF0000u) ? 0x7FFF0000u : 0;
                    w[e] = lo | hi;
                }
                w[e] ^= sign;
            }
            t.q[x] = w;
        }
    }
    t.reset();
    __syncthreads();

    // the wave's queries; the nearest place that all see up to, and the farthest that
    // one of them stands at (see attention.h)
    const uint32_t last_row = min(row0 + 32, a.rows) - 1;
    const bool some = row0 < a.rows;
    const int32_t from_query = (int32_t)(row0 / a.G), to_query = (int32_t)(last_row / a.G);
    const int32_t first = t.place0 + (a.tree ? -1 : from_query);
    const int32_t last = t.place0 + (a.tree ? (int32_t)a.Q - 1 : to_query);
    auto all_seen = [&](uint32_t at, uint32_t exist) {
        const int32_t k0 = part0 + (int32_t)at;
        return exist == ~0u && t.key_at(k0 + kTile - 1) <= first &&
               (a.window == 0 || k0 + kTile <= keys.few ||
                (k0 >= keys.few && (int64_t)t.key_at(k0) > (int64_t)last - a.window));
    };

    const char *kbase = a.kc + hk * a.head, *vbase = a.vc + hk * a.head;
    const uint32_t to = lds_addr(reinterpret_cast<const uint16_t*>(pool));
    // (the thread's pieces are worked out each time: kept, they pushed others out of the
    // registers, and a load of those back waits for all copies)
    auto copy = [&](uint32_t stage) {
        uint32_t me = tid;
        asm volatile("" : "+v"(me));
        S::template copy<ONCE>(a, place + stage % kRing * kKeys, kbase, vbase,
                               to + stage % S::kDepth * (2 * S::kBytes), me);
    };
    const uint32_t ids_at = lds_addr(reinterpret_cast<const uint16_t*>(ids));
    for (uint32_t s = 0; s + 1 < S::kDepth && s < stages; ++s) copy(s);
    for (uint32_t s = 0; s < stages; ++s) {
        // this stage's copies have landed (later loads than those of the stages behind it
        // make the wait longer, not shorter), and every wave is through with the stage
        // before, whose part of LDS and of the ring are free
        if (s + S::kDepth - 1 <= stages) wait_vmcnt<(S::kDepth - 2) * 2 * S::kCopies>();
        else wait_vmcnt<0>();
        __syncthreads();
        const char* here = pool + s % S::kDepth * (2 * S::kBytes);
        // The places of stage s + depth, which is copied from the next stage on, from its
        // pages' ids; a wave asked for these before it asked for this stage's keys, and they
        // have landed with them.
        constexpr uint32_t kAsked = 2 * S::kDepth - 1;
        uint32_t to_come = s + S::kDepth;
        if (to_come >= kRing && to_come < stages && wave == to_come % kWaves) {
            const uint32_t j = to_come * kKeys + lane;
            put_place(j, place_of(j, *(volatile uint32_t*)&ids[to_come % kRing * kKeys + lane]));
        }
        // (ids in registers would be waited for, and every copy before them)
        to_come = s + kAsked;
        if (to_come >= kRing && to_come < stages && wave == to_come % kWaves) {
            const uint32_t j = min(to_come * kKeys + lane, count - 1);
            dma4(a.page_table + (int64_t)n * a.table + key_no(j) / a.page_size, ids_at + to_come % kRing * (kKeys * 4));
        }
        if (s + S::kDepth - 1 < stages) copy(s + S::kDepth - 1);
        if (!some) continue;
#pragma unroll 1
        for (uint32_t off = 0; off < kKeys; off += kTile) {
            const uint32_t at = s * kKeys + off;
            const char *ks = here + off * S::kRow, *vs = ks + S::kBytes;
            const uint32_t exist = __builtin_amdgcn_readfirstlane((int)there[s % kRing * 2 + off / kTile]);
            const bool all = all_seen(at, exist);
            uint32_t on = 0;
            if (!all) on = t.seen(exist, part0 + (int32_t)at);
            t.tile(ks, vs, all, on);
        }
    }
    if (some && __any(!t.finite())) {
        t.reset();
        for (uint32_t at = 0; at < count; at += kTile) {
            const uint32_t j = at + t.c;
            t.tile_careful(kbase, vbase, place_of(j, page_of(j)), part0 + (int32_t)at, from_query, to_query);
        }
    }
    t.l += __shfl_xor(t.l, 32);

    const uint32_t r = row0 + t.c;
    if (r >= a.rows) return;
    const uint32_t i = r / a.G, h = hk * a.G + (r - i * a.G);
    const bool direct = keys.parts <= 1;
    const float inv = t.l == 0.0f ? 0.0f : (a.v_scale ? a.v_scale[hk] : 1.0f) / t.l;
    const int64_t at = ((int64_t)owner * a.rows + r) * a.splits + split;
    uint16_t* out = a.out + n * a.o_n + i * a.o_i + h * a.o_h;
    // the lane's dims: four in a row from 32 j + 8 b + 4 g on
#pragma unroll
    for (int j = 0; j < T::kOuts; ++j)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t d = 32 * j + 8 * b + 4 * t.g;
            if (d >= a.D) continue;
            f32x4 z;
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = t.o[j][4 * b + e];
            if (!direct) {
                *reinterpret_cast<f32x4*>(a.part + at * a.D + d) = z;
                continue;
            }
            u32x2 w;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[e] = H::pack(t.l == 0.0f ? 0.0f : z[2 * e] * inv, t.l == 0.0f ? 0.0f : z[2 * e + 1] * inv);
            }
            if (a.wide) {
                *reinterpret_cast<u32x2*>(out + d) = w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) out[d + e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
            }
        }
    if (t.g == 0) {
        if (!direct) {
            a.part_ml[at] = float2{t.m, t.l};
        } else if (a.lse) {
            a.lse[((int64_t)n * a.Q + i) * a.Hq + h] =
                t.l == 0.0f ? kNone : (t.m - H::kLift + log2f(t.l)) * 0.693147180559945309f;
        }
    }
}

template <bool FP16, bool E4M3, int DP>
void launch_dims_of(AttnArgs a, bool once, hipStream_t stream)
{
    if (a.N * a.splits >= 8) a.units = (a.N * a.splits + 7) / 8 * 8 * a.Hk;   // see the kernel
    const uint32_t grid = (a.units + 7) / 8 * 8 * a.groups;
    for (a.first = 0; a.first < grid; a.first += kMostGroups) {
        const uint32_t n = grid - a.first < kMostGroups ? grid - a.first : kMostGroups;
        if (once) {
            hipLaunchKernelGGL((wide_kernel<FP16, E4M3, DP, true>), dim3(n), dim3(kThreads), 0, stream, a);
        } else {
            hipLaunchKernelGGL((wide_kernel<FP16, E4M3, DP, false>), dim3(n), dim3(kThreads), 0, stream, a);
        }
    }
}

template <bool FP16, bool E4M3>
void launch_types(const AttnArgs& a, bool once, hipStream_t stream)
{
    if (a.D <= 64) return launch_dims_of<FP16, E4M3, 64>(a, once, stream);
    if (a.D <= 128) return launch_dims_of<FP16, E4M3, 128>(a, once, stream);
    launch_dims_of<FP16, E4M3, 256>(a, once, stream);
}

}  // namespace

namespace xpress {

void launch_wide(AttnArgs a, bool fp16, bool e4m3, bool once, hipStream_t stream)
{
    if (fp16) e4m3 ? launch_types<true, true>(a, once, stream) : launch_types<true, false>(a, once, stream);
    else e4m3 ? launch_types<false, true>(a, once, stream) : launch_types<false, false>(a, once, stream);
}

}  // namespace xpress
