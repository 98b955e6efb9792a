// paged_attention.hip -- attention of the newest tokens of every sequence
// over a paged key-value cache (gfx950, wave64, MFMA).
//
// The Q new queries of a sequence and the G query heads of a key-value head
// are Q * G rows that read the same keys: the cache goes by once for all of
// them.  A workgroup (four waves) takes up to 64 rows of one (sequence,
// key-value head) and one part of the keys.  Up to 16 rows, its waves take
// 32-key tiles in turn, straight to registers; more rows are 16 to a wave, and
// the waves take the tiles from LDS, where they are staged once for all of them
// (a wave with four times the rows in its registers spilled 1.4 KB a lane: 350
// us where this form takes 78).  Per tile, with lane l = 16 g + c:
//
//   S^T = K Q^T   v_mfma_f32_16x16x32: A = keys (lane: key c, 8 dims of the
//                 contraction), B = queries (lane: row c).  The lane gets the
//                 scores of row c with keys 4 g + i of each 16-key half, so a
//                 row's softmax state lives in the four lanes with its c.
//   softmax       the running maximum m is only moved when a score passes it
//                 by more than kRise (in base 2), so most tiles need neither a
//                 cross-lane reduction nor a rescaling of the sums; weights
//                 2^(s - m) then reach 2^kRise, which fp32 sums hold as well.
//   O^T += V^T P  P^T is already in B's layout: slot 8 g + e of the contraction
//                 is key 4 g + e of the first half (e < 4) or 4 g + e - 4 of
//                 the second.  A = V^T: the lane reads eight dims 8 c .. 8 c + 7
//                 of its eight keys (whole rows, 16 bytes a lane) and
//                 transposes the 8 x 8 block in registers; dim 8 c + j is row c
//                 of the j-th product.  No LDS round trip for P.
//
// Weights enter the product as two 16-bit parts (rounded weight, rounded
// rest), 16 bits or more in all: with one part their rounding adds as much
// error as the output's own.  Up to 16 rows the cache's bytes hide the second
// product; a block of queries, whose products come on top of its copies in part,
// pays for it.  Scores, m, the sum l and O are fp32.  An fp16 weight is scaled by
// 2^kLift so that weights down to 2^-25 of the largest stay normal numbers.
//
// Each key's place in the pool is worked out once per workgroup, into a table in
// LDS (one division by the page size per key, any page size), which a part of more
// keys fills several times; a bit says whether the key exists.  A key on a missing page, or past the part's end, does
// not: its place is the pool's first row, its score is masked and its value row
// taken as zeros.
//
// A value that is not finite must not reach rows that do not see it, though 0
// times it is NaN.  The product above does not care; a wave whose sums come
// out non-finite runs its tiles again in a careful form, query by query, with
// the value rows which that query does not see set to zero.
//
// The waves' sums meet in LDS.  A sequence of one part is written out
// directly; with more parts (chosen on the host from the number of rows'
// owners and the longest length, see plan_of) the parts' (m, l, O) go to the
// workspace and a second kernel joins them in a fixed order.
//
// Bound by the cache's bytes.  Measured (32 query and 8 key-value heads of 128,
// bf16): 32 sequences up to 4096 tokens 51 us and 5 for the join, 5.9 TB/s; one
// of 131072 tokens with 4 heads 44 + 5, 6.2 TB/s; a block of 16 queries of the 32
// sequences 78 + 11, where the copies to LDS set the pace; 128 sequences up to
// 6000 on an e4m3 cache, heads of 64, 93 + 5, 4.9 TB/s, by instructions a byte;
// one of 1009 tokens 7 + 4, latency.  Whole calls: heads of 256, one workgroup a
// compute unit, 140 us for the 32 sequences (4.1 TB/s); their blocks of 128 and 256
// rows a head 126 and 210, by what every wave does again for its 16 rows (operands
// from LDS, the 8 x 8 blocks); one of 1009 under a bound of 131072, 8 parts of
// 2048 for its 8 of 128, 16.

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "device_common.h"
#include "host_common.h"
#include "kv_common.h"
#include "xpress_argmax.h"

namespace {

using namespace xpress;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;
constexpr int kTile = 32;        // keys of one tile
constexpr int kRound = kTile * kWaves;
constexpr int kUnits = 256;       // compute units of the chip
constexpr int kTable = 2048;     // keys whose places LDS holds at once
constexpr int kTableStaged = 1024;  // the same where LDS also holds the keys
constexpr float kNone = -INFINITY;

struct AttnArgs {
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    float* part;      // [rows of all, splits, D], then (m, l) [rows of all, splits]
    float2* part_ml;
    const int32_t *lens, *page_table;
    const char *kc, *vc;
    const float *k_scale, *v_scale;
    int64_t q_n, q_i, q_h, o_n, o_i, o_h;
    int64_t page, head, token, table;  // cache strides in bytes; page table row stride
    uint32_t N, Q, Hq, Hk, G, D, pages, page_size;
    uint32_t rows, groups, units, chunk, splits;
    int32_t max_len, window;
    float scale;      // times log2(e)
    uint32_t wide;    // q and out rows are 16-byte aligned
    uint32_t first;   // of the launch's workgroups
};

// The keys that any query of a sequence sees, [lo, hi), and its parts.
struct Keys {
    int32_t len, lo, hi;
    uint32_t parts;
};

__device__ __forceinline__ Keys keys_of(const AttnArgs& a, uint32_t n)
{
    Keys k;
    k.len = a.lens[n];
    k.len = k.len < 0 ? 0 : k.len > a.max_len ? a.max_len : k.len;
    const int64_t lo = (int64_t)k.len - a.Q - a.window + 1;
    k.lo = a.window > 0 && lo > 0 ? (int32_t)lo : 0;
    k.hi = k.len;
    k.parts = ((uint32_t)(k.hi - k.lo) + a.chunk - 1) / a.chunk;
    return k;
}

// 16-bit arithmetic of the two query types.
template <bool FP16>
struct Half {
    using Vec = bf16x8;
    static constexpr float kRise = 8.0f, kLift = 0.0f;
    static __device__ __forceinline__ f32x4 mfma(u32x4 x, u32x4 y, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(Vec, x),
                                                       __builtin_bit_cast(Vec, y), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y)
    {
        f32x2 v = {x, y};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return bf16_lo(w); }
    static __device__ __forceinline__ float hi(uint32_t w) { return bf16_hi(w); }
    static constexpr uint32_t kExp = 0x7F807F80u;  // exponent bits of both
    template <bool HIGH>
    static __device__ __forceinline__ uint32_t from8(uint32_t w)
    {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
    }
};

template <>
struct Half<true> {
    using Vec = f16x8;
    static constexpr float kRise = 4.0f, kLift = 11.0f;
    static __device__ __forceinline__ f32x4 mfma(u32x4 x, u32x4 y, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(Vec, x),
                                                      __builtin_bit_cast(Vec, y), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y)
    {
        f16x2 v = {(_Float16)x, (_Float16)y};
        return __builtin_bit_cast(uint32_t, v);
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w).x; }
    static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w).y; }
    static constexpr uint32_t kExp = 0x7C007C00u;
    template <bool HIGH>
    static __device__ __forceinline__ uint32_t from8(uint32_t w)
    {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
    }
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The four lanes of a row (same l % 16).
__device__ __forceinline__ float row_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}

__device__ __forceinline__ float row_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Cache rows in LDS as they are in the pool.  A piece (16 bytes) of a key row
// goes to place piece ^ turn(row), so that the sixteen rows which a quarter wave
// reads at one piece lie in different banks; value rows, read whole, change
// places within four so that the four quarters do.
template <bool E4M3, int DP>
struct Lines {
    static constexpr uint32_t kRow = DP * (E4M3 ? 1 : 2);  // bytes
    static constexpr uint32_t kPieces = kRow / 16;

    static __device__ __forceinline__ uint32_t turn(uint32_t row)
    {
        return kPieces >= 16 ? row & 15 : row * kPieces / 16 & (kPieces - 1);
    }
    static __device__ __forceinline__ uint32_t slot(uint32_t row)
    {
        return kRow >= 256 ? row : row ^ (row >> 2 & (256 / kRow - 1));
    }
};

// Two stages of kKeys keys and values in LDS, for workgroups of several row
// waves; two such workgroups (one at 256 dims) share a compute unit's LDS.  (Four
// stages of 32 keys, the same LDS: 104 us where these take 86; the barriers are
// twice as many.)
template <bool E4M3, int DP>
struct Stage : Lines<E4M3, DP> {
    using L = Lines<E4M3, DP>;
    static constexpr uint32_t kKeys = 64;
    static constexpr uint32_t kBytes = kKeys * L::kRow;                  // keys or values
    static constexpr uint32_t kCopies = kKeys * L::kPieces / kThreads;   // of a thread, keys or values

    // Where a thread's pieces of keys [t, t + kKeys) are.  Rows that do not exist
    // and pieces past the head's end: any bytes of the pool, masked or dropped
    // after.
    struct From {
        const char *k[kCopies], *v[kCopies];
    };
    static __device__ __forceinline__ From find(const AttnArgs& a, const int64_t* place, uint32_t t,
                                                const char* kbase, const char* vbase)
    {
        const uint32_t used = a.D * (E4M3 ? 1 : 2);
        From f;
#pragma unroll
        for (uint32_t x = 0; x < kCopies; ++x) {
            const uint32_t at = x * kThreads + threadIdx.x, row = at / L::kPieces, piece = at % L::kPieces;
            const uint32_t kd = (piece ^ L::turn(row)) * 16, vd = piece * 16;
            f.k[x] = kbase + place[t + row] + (kd < used ? kd : 0);
            f.v[x] = vbase + place[t + L::slot(row)] + (vd < used ? vd : 0);
        }
        return f;
    }

    // Queues their copies to LDS byte address `to`, the wave's part of a stage.
    // ONCE: no other workgroup reads them, so they pass the caches by.
    template <bool ONCE>
    static __device__ __forceinline__ void copy(const From& f, uint32_t to)
    {
#pragma unroll
        for (uint32_t x = 0; x < kCopies; ++x) {
            dma16<ONCE>(reinterpret_cast<const uint16_t*>(f.k[x]), to + x * kThreads * 16);
            dma16<ONCE>(reinterpret_cast<const uint16_t*>(f.v[x]), to + kBytes + x * kThreads * 16);
        }
    }
};

// ONCE: the bytes are read once and pass the caches by.
template <bool ONCE, typename T>
__device__ __forceinline__ T load(const char* p)
{
    if constexpr (!ONCE) {
        return *reinterpret_cast<const T*>(p);
    } else if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p)));
    } else if constexpr (sizeof(T) == 8) {
        return __builtin_bit_cast(T, __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p)));
    } else {
        return __builtin_bit_cast(T, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
    }
}

template <bool FP16, bool E4M3, int DP, int DEEP, bool BOUNCE, bool ONCE>
struct Tile {
    static constexpr int kDims = DP / 32;              // products of the scores
    static constexpr int kOuts = DP / 16;              // products of the output
    static constexpr int kLoads = E4M3 ? DP / 64 : DP / 32;  // 16-byte loads of a key row per lane
    static constexpr int kBlocks = DP > 128 ? DP / 128 : 1;
    static constexpr int kEach = kOuts / kBlocks;      // dims of a value row per lane and block
    static constexpr int kWords = E4M3 ? kEach / 4 : kEach / 2;
    static constexpr int kDeep = DEEP;
    static constexpr bool kBounce = BOUNCE;
    using H = Half<FP16>;
    using S = Lines<E4M3, DP>;
    template <int W> struct Words { uint32_t w[W]; };

    const AttnArgs& a;
    const int64_t* place;   // LDS: byte offsets of the part's keys
    const uint32_t* there;  // LDS: which of a tile's keys exist
    const char *kbase, *vbase;
    uint32_t c, g;
    u32x4 q[kDims];
    u32x4 k[2][kLoads];
    u32x4 k_in[kDeep][2 * kLoads];      // on their way, a slot a tile
    Words<kWords> v[kDeep][8][kBlocks];
    f32x4 o[kOuts];
    float m, l;
    int32_t pos;            // position of the lane's row's query; INT32_MIN: no row
    float scale;

    // First of the eight dims that lane group g supplies to product i.
    __device__ __forceinline__ uint32_t dim_of(int i) const
    {
        return E4M3 ? (uint32_t)(i / 2) * 64 + g * 16 + (uint32_t)(i % 2) * 8 : (uint32_t)i * 32 + g * 8;
    }

    __device__ __forceinline__ uint32_t key_of(int e) const { return (uint32_t)(e / 4) * 16 + g * 4 + e % 4; }

    // The tile's key rows, whole rows after each other over the lanes (a load of
    // 64 bytes of 16 rows each, the product's own layout, reached 4.6 TB/s where
    // this one reaches 5.4).
    template <bool PASS>
    __device__ __forceinline__ void load_rows(u32x4* in, uint32_t t)
    {
        const uint32_t used = a.D * (E4M3 ? 1 : 2), lane = g * 16 + c;
#pragma unroll
        for (int i = 0; i < 2 * kLoads; ++i) {
            const uint32_t at = i * 64 + lane, row = at / S::kPieces, d = at % S::kPieces * 16;
            in[i] = load<PASS, u32x4>(kbase + place[t + row] + (d < used ? d : 0));
        }
    }

    // From the registers to the wave's own part of LDS.
    __device__ __forceinline__ void put(const u32x4* in, char* to)
    {
        const uint32_t lane = g * 16 + c;
#pragma unroll
        for (int i = 0; i < 2 * kLoads; ++i) {
            const uint32_t at = i * 64 + lane, row = at / S::kPieces, piece = at % S::kPieces;
            *reinterpret_cast<u32x4*>(to + row * S::kRow + (piece ^ S::turn(row & 15)) * 16) = in[i];
        }
    }

    // The products' operands of a tile from its rows in LDS.
    __device__ __forceinline__ void take_keys(const char* ks)
    {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                k[s][i] = *reinterpret_cast<const u32x4*>(
                    ks + (s * 16 + c) * S::kRow + (((uint32_t)i * 4 + g) ^ S::turn(c)) * 16);
            }
        trim_keys();
    }

    __device__ __forceinline__ void take_values(const char* vs)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                v[0][e][b] = *reinterpret_cast<const Words<kWords>*>(
                    vs + S::slot(key_of(e)) * S::kRow + (b * 128 + c * kEach) * (E4M3 ? 1 : 2));
            }
    }

    // The same straight from the pool.
    template <bool PASS>
    __device__ __forceinline__ void load_keys(u32x4* in, uint32_t t)
    {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const char* p = kbase + place[t + s * 16 + c];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const uint32_t d = E4M3 ? (uint32_t)i * 64 + g * 16 : (uint32_t)i * 32 + g * 8;
                in[s * kLoads + i] = load<PASS, u32x4>(p + (d < a.D ? d * (E4M3 ? 1 : 2) : 0));
            }
        }
    }

    template <bool PASS>
    __device__ __forceinline__ void load_values(int x, uint32_t t)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const uint32_t d = (uint32_t)b * 128 + c * kEach;
                v[x][e][b] = load<PASS, Words<kWords>>(vbase + place[t + key_of(e)] +
                                                       (d < a.D ? d * (E4M3 ? 1 : 2) : 0));
            }
    }

    // Fills slot x.
    __device__ __forceinline__ void fetch_keys(int x, uint32_t t)
    {
        if constexpr (kBounce) load_rows<ONCE>(k_in[x], t);
        else load_keys<ONCE>(k_in[x], t);
    }

    // Dims past the head's end were loads of its first ones: zeros instead.
    __device__ __forceinline__ void trim_keys()
    {
        if (a.D == DP) return;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if ((uint32_t)i * (E4M3 ? 64 : 32) + g * (E4M3 ? 16 : 8) >= a.D) k[0][i] = k[1][i] = u32x4{0, 0, 0, 0};
        }
    }

    __device__ __forceinline__ u32x4 key_part(int s, int i) const
    {
        u32x4 y;
        if constexpr (E4M3) {
            const uint32_t w0 = k[s][i / 2][(i % 2) * 2], w1 = k[s][i / 2][(i % 2) * 2 + 1];
            y = u32x4{H::template from8<false>(w0), H::template from8<true>(w0),
                      H::template from8<false>(w1), H::template from8<true>(w1)};
        } else {
            y = k[s][i];
        }
        return y;
    }

    // A operands of output products (j, j + 1): dims 2 of the lane's, 8 keys.
    __device__ __forceinline__ void value_parts(int slot, int j, u32x4* even, u32x4* odd) const
    {
        const int b = j / kEach, w = j % kEach;
        uint32_t x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (E4M3) {
                const uint32_t y = v[slot][e][b].w[w / 4];
                x[e] = (w / 2) % 2 ? H::template from8<true>(y) : H::template from8<false>(y);
            } else {
                x[e] = v[slot][e][b].w[w / 2];
            }
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            (*even)[p] = __builtin_amdgcn_perm(x[2 * p + 1], x[2 * p], 0x05040100u);
            (*odd)[p] = __builtin_amdgcn_perm(x[2 * p + 1], x[2 * p], 0x07060302u);
        }
    }

    __device__ __forceinline__ bool sees(int32_t key) const
    {
        return key <= pos && (a.window == 0 || (int64_t)key > (int64_t)pos - a.window);
    }

    // Scores and weights of one tile: P as two 16-bit parts.
    template <bool MASKED>
    __device__ __forceinline__ void weigh(uint32_t t, int32_t key0, u32x4* big, u32x4* rest)
    {
        f32x4 s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kDims; ++i) {
            s0 = H::mfma(key_part(0, i), q[i], s0);
            s1 = H::mfma(key_part(1, i), q[i], s1);
        }
        const uint32_t exist = MASKED ? there[t / kTile] : 0;
        float s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[e] = (e < 4 ? s0[e] : s1[e - 4]) * scale;
            if constexpr (MASKED) {
                const bool on = (exist >> key_of(e) & 1) && sees(key0 + (int32_t)(t + key_of(e)));
                s[e] = on ? s[e] : kNone;
            }
        }
        float top = s[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e]);
        if (__any(top > m + H::kRise)) {
            const float to = fmaxf(m, row_max(top));
            const float f = to == m ? 1.0f : exp2_fast(m - to);
            m = to;
            l *= f;
#pragma unroll
            for (int j = 0; j < kOuts; ++j) o[j] *= f;
        }
        const float from = (m == kNone ? 0.0f : m) - H::kLift;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float w0 = exp2_fast(s[2 * p] - from), w1 = exp2_fast(s[2 * p + 1] - from);
            l += w0 + w1;
            const uint32_t w = H::pack(w0, w1);
            (*big)[p] = w;
            (*rest)[p] = H::pack(w0 - H::lo(w), w1 - H::hi(w));
        }
    }

    __device__ __forceinline__ void reset()
    {
        m = kNone;
        l = 0.0f;
#pragma unroll
        for (int j = 0; j < kOuts; ++j) o[j] = f32x4{0, 0, 0, 0};
    }

    // Value rows that are not there become zeros.
    __device__ __forceinline__ void drop_missing(int x, uint32_t t)
    {
        const uint32_t exist = there[t / kTile];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t keep = exist >> key_of(e) & 1 ? ~0u : 0u;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int w = 0; w < kWords; ++w) v[x][e][b].w[w] &= keep;
        }
    }

    // The output products of one tile, whose values are in v.
    __device__ __forceinline__ void gather(int x, u32x4 big, u32x4 rest)
    {
#pragma unroll
        for (int j = 0; j < kOuts; j += 2) {
            u32x4 even, odd;
            value_parts(x, j, &even, &odd);
            o[j] = H::mfma(even, big, o[j]);
            o[j + 1] = H::mfma(odd, big, o[j + 1]);
            o[j] = H::mfma(even, rest, o[j]);
            o[j + 1] = H::mfma(odd, rest, o[j + 1]);
        }
    }

    // One tile whose rows are in LDS.
    template <bool MASKED>
    __device__ __forceinline__ void tile(const char* ks, const char* vs, uint32_t t, int32_t key0)
    {
        u32x4 big, rest;
        take_keys(ks);
        weigh<MASKED>(t, key0, &big, &rest);
        take_values(vs);
        if constexpr (MASKED) drop_missing(0, t);
        gather(0, big, rest);
    }

    // A wave's LDS accesses are carried out in order: only the compiler has to
    // be kept from moving one lane's reads past another's writes.
    static __device__ __forceinline__ void in_order()
    {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }

    // The tile of slot x; the loads of the tile that takes the slot next are
    // queued as soon as its registers are free.  They are queued always (past
    // the part's end they read the pool's first row): the number of loads in
    // flight is then known, and a wait is for its own loads only.
    template <bool MASKED>
    __device__ __forceinline__ void tile_own(int x, char* own, uint32_t t, uint32_t next, int32_t key0)
    {
        u32x4 big, rest;
        if constexpr (kBounce) {
            in_order();
            put(k_in[x], own);
            fetch_keys(x, next);
            in_order();
            take_keys(own);
        } else {
#pragma unroll
            for (int i = 0; i < 2 * kLoads; ++i) k[i / kLoads][i % kLoads] = k_in[x][i];
            trim_keys();
        }
        weigh<MASKED>(t, key0, &big, &rest);
        if constexpr (!kBounce) fetch_keys(x, next);
        if constexpr (MASKED) drop_missing(x, t);
        gather(x, big, rest);
        load_values<ONCE>(x, next);
    }

    // The careful form of a tile (see the top of the file): positions
    // [first, last] of the workgroup's queries one after the other.
    __device__ __forceinline__ void tile_careful(uint32_t t, int32_t key0, int32_t first, int32_t last)
    {
        load_keys<false>(k_in[0], t);
#pragma unroll
        for (int i = 0; i < 2 * kLoads; ++i) k[i / kLoads][i % kLoads] = k_in[0][i];
        trim_keys();
        u32x4 big, rest;
        weigh<true>(t, key0, &big, &rest);
        for (int32_t at = first; at <= last; ++at) {
            load_values<false>(0, t);
            drop_missing(0, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int32_t key = key0 + (int32_t)(t + key_of(e));
                if (key > at || (a.window > 0 && (int64_t)key <= (int64_t)at - a.window)) {
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                        for (int w = 0; w < kWords; ++w) v[0][e][b].w[w] = 0;
                }
            }
#pragma unroll
            for (int j = 0; j < kOuts; j += 2) {
                u32x4 x[2];
                value_parts(0, j, &x[0], &x[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // the weights' second part meets finite values only
                    u32x4 y;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t z = x[h][w];
                        y[w] = ((z & H::kExp & 0xFFFFu) == (H::kExp & 0xFFFFu) ? 0 : z & 0xFFFFu) |
                               ((z & H::kExp & 0xFFFF0000u) == (H::kExp & 0xFFFF0000u) ? 0 : z & 0xFFFF0000u);
                    }
                    f32x4 r = H::mfma(x[h], big, f32x4{0, 0, 0, 0});
                    r = H::mfma(y, rest, r);
                    if (pos == at) o[j + h] += r;
                }
            }
        }
    }

    __device__ __forceinline__ bool finite() const
    {
        bool ok = true;
#pragma unroll
        for (int j = 0; j < kOuts; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) ok &= __builtin_fabsf(o[j][i]) < INFINITY;
        return ok;
    }
};

// Rows of 16 fp32 sums of a wave, padded against bank conflicts.
template <int DP>
constexpr int row_stride() { return DP + 4; }

// One row's result: 8 dims from its sums over the waves.
__device__ __forceinline__ void store8(const AttnArgs& a, bool fp16, uint16_t* dst, const float* y)
{
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = fp16 ? Half<true>::pack(y[2 * i], y[2 * i + 1]) : Half<false>::pack(y[2 * i], y[2 * i + 1]);
    }
    if (a.wide) {
        *reinterpret_cast<u32x4*>(dst) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
    }
}

// Whether key rows go through LDS: all but the shortest rows, whose tiles are
// too little work beside that (e4m3 rows of 64: 97 us direct, 109 by LDS), and
// the longest, for which the registers do not suffice.
template <bool E4M3, int DP>
constexpr bool keys_bounce()
{
    return E4M3 ? DP == 128 : DP <= 128;
}

// Tiles that a wave loads ahead, as its registers allow.
template <bool E4M3, int DP>
constexpr int tiles_ahead()
{
    return DP * (E4M3 ? 1 : 2) <= 64 ? 3 : DP * (E4M3 ? 1 : 2) <= 128 ? 2 : 1;
}

// RW waves of the workgroup hold 16 rows each, KW = kWaves / RW waves share a
// row's keys.  RW = 1: each wave loads its own tiles to registers, tiles_ahead()
// of them ahead.  RW > 1: the waves' tiles come from LDS, two stages deep.  MANY: the
// part may have more keys than the table of places, which is then filled again.
template <bool FP16, bool E4M3, int DP, int RW, bool ONCE, bool MANY>
__global__ void __launch_bounds__(kThreads, DP == 256 ? 1 : 2) attention_kernel(AttnArgs a)
{
    constexpr int kDeep = RW > 1 ? 1 : tiles_ahead<E4M3, DP>();
    using T = Tile<FP16, E4M3, DP, kDeep, keys_bounce<E4M3, DP>(), ONCE>;
    using S = Stage<E4M3, DP>;
    using H = Half<FP16>;
    constexpr int KW = kWaves / RW;
    constexpr int kRow = row_stride<DP>();
    constexpr int kSums = kWaves * 16 * kRow * 4, kStages = RW > 1 ? 4 * S::kBytes : kWaves * kTile * S::kRow;
    constexpr int kKeysAtOnce = RW > 1 ? kTableStaged : kTable;
    constexpr int kPlaces = RW > 1 ? kTableStaged : kTable + kDeep * kRound;
    __shared__ __align__(16) int64_t place[kPlaces];
    __shared__ uint32_t there[kPlaces / kTile];
    // the stages, then the waves' sums
    __shared__ __align__(16) char pool[kSums > kStages ? kSums : kStages];
    __shared__ float sm[kWaves][16], sl[kWaves][16];
    __shared__ uint32_t holes;
    float(*sums)[16][kRow] = reinterpret_cast<float(*)[16][kRow]>(pool);

    // Workgroup i runs on XCD i % 8: the row groups that read the same keys
    // follow each other on one XCD.
    const uint32_t id = a.first + blockIdx.x;
    const uint32_t unit = id / (8 * a.groups) * 8 + id % 8, group = id / 8 % a.groups;
    if (unit >= a.units) return;
    const uint32_t owner = unit % (a.N * a.Hk), split = unit / (a.N * a.Hk);
    const uint32_t n = owner / a.Hk, hk = owner % a.Hk;
    const uint32_t tid = threadIdx.x, wave = tid / 64, lane = tid & 63;
    const uint32_t rw = wave % RW, kw = wave / RW;
    const Keys keys = keys_of(a, n);
    if (split > 0 && split >= keys.parts) return;
    const int32_t part0 = keys.lo + (int32_t)(split * a.chunk);
    const uint32_t part_count = (uint32_t)min(keys.hi - part0, (int32_t)a.chunk);  // 0: an empty sequence
    const uint32_t row0 = group * (16 * RW);

    // the keys of the table: the whole part, or a piece of it
    int32_t key0 = part0;
    uint32_t count = MANY ? min(part_count, (uint32_t)kKeysAtOnce) : part_count;
    if (tid == 0) holes = 0;
    __syncthreads();
    constexpr uint32_t kPad = RW > 1 ? S::kKeys : kTile;
    uint32_t padded = (count + kPad - 1) / kPad * kPad;
    auto find_places = [&]() {
        const uint32_t filled = RW > 1 ? padded : padded + kDeep * kRound;
        for (uint32_t j0 = wave * 64; j0 < filled; j0 += kThreads) {
            const uint32_t j = j0 + lane;
            int64_t at = -1;
            if (j < count) {
                const uint32_t key = (uint32_t)key0 + j, slot = key / a.page_size;
                const uint32_t page = (uint32_t)a.page_table[(int64_t)n * a.table + slot];
                if (page < a.pages) {
                    at = (int64_t)page * a.page + (int64_t)(key - slot * a.page_size) * a.token;
                } else {
                    holes = 1;
                }
            }
            const uint64_t on = __ballot(at >= 0);
            if (j < filled) place[j] = at < 0 ? 0 : at;
            if (lane < 2 && j0 + lane * kTile < filled) there[j0 / kTile + lane] = (uint32_t)(on >> (lane * kTile));
        }
    };
    find_places();
    // MANY: the table of the keys from part0 + from on, once every wave is through
    // with the one before
    auto turn_to = [&](uint32_t from) {
        key0 = part0 + (int32_t)from;
        count = min(part_count - from, (uint32_t)kKeysAtOnce);
        padded = (count + kPad - 1) / kPad * kPad;
        __syncthreads();
        find_places();
        __syncthreads();
    };

    T t{a, place, there, a.kc + hk * a.head, a.vc + hk * a.head, lane & 15, lane / 16};
    t.scale = a.scale * (a.k_scale ? a.k_scale[hk] : 1.0f);
    {
        const uint32_t r = row0 + rw * 16 + t.c;
        const bool on = r < a.rows;
        const uint32_t i = on ? r / a.G : 0, h = hk * a.G + (on ? r - i * a.G : 0);
        t.pos = on ? keys.len - (int32_t)a.Q + (int32_t)i : INT32_MIN;
        const uint16_t* src = a.q + n * a.q_n + i * a.q_i + h * a.q_h;
#pragma unroll
        for (int x = 0; x < T::kDims; ++x) {
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
            t.q[x] = w;
        }
    }
    t.reset();
    __syncthreads();

    // positions of the wave's first and last query; a wave may have no rows
    const uint32_t first_row = row0 + rw * 16, last_row = min(first_row + 16, a.rows) - 1;
    const bool some = first_row < a.rows;
    const int32_t first = keys.len - (int32_t)a.Q + (int32_t)(first_row / a.G);
    const int32_t last = keys.len - (int32_t)a.Q + (int32_t)(last_row / a.G);
    bool whole = holes == 0;
    // every row sees every key of the tile at t
    auto all_seen = [&](uint32_t at) {
        const int32_t k0 = key0 + (int32_t)at;
        return whole && at + kTile <= count && k0 + kTile - 1 <= first &&
               (a.window == 0 || (int64_t)k0 > (int64_t)last - a.window);
    };
    for (uint32_t from = 0;;) {
        if constexpr (RW == 1) {
            const uint32_t begin = kw * kTile;
            char* own = pool + kw * (kTile * S::kRow);
            if (begin < padded) {
#pragma unroll
                for (int x = 0; x < kDeep; ++x) {
                    t.fetch_keys(x, begin + x * kRound);
                    t.template load_values<ONCE>(x, begin + x * kRound);
                }
                for (uint32_t at = begin;;) {
#pragma unroll
                    for (int x = 0; x < kDeep; ++x) {
                        const uint32_t next = at + kDeep * kRound;
                        if (all_seen(at)) t.template tile_own<false>(x, own, at, next, key0);
                        else t.template tile_own<true>(x, own, at, next, key0);
                        at += kRound;
                        if (at >= padded) goto through;
                    }
                }
            through:;
            }
        } else {
            const uint32_t to = lds_addr(reinterpret_cast<const uint16_t*>(pool)) +
                                (uint32_t)__builtin_amdgcn_readfirstlane((int)(wave * 64 * 16));
            // addresses are looked up before the wait, so that the copies follow it at once
            typename S::From from = {};
            if (padded > 0) {
                S::template copy<ONCE>(S::find(a, place, 0, t.kbase, t.vbase), to);
                if (S::kKeys < padded) from = S::find(a, place, S::kKeys, t.kbase, t.vbase);
            }
            for (uint32_t at = 0; at < padded; at += S::kKeys) {
                // this stage's copies have landed, and every wave is through with
                // the stage before, whose half the next copies fill
                const uint32_t half = at / S::kKeys % 2;
                wait_vmcnt<0>();
                __syncthreads();
                const char* here = pool + half * (2 * S::kBytes);
                if (at + S::kKeys < padded) {
                    S::template copy<ONCE>(from, to + (1 - half) * (2 * S::kBytes));
                    if (at + 2 * S::kKeys < padded) from = S::find(a, place, at + 2 * S::kKeys, t.kbase, t.vbase);
                }
                if (!some) continue;
#pragma unroll
                for (uint32_t x = 0; x < S::kKeys / kTile / KW; ++x) {
                    const uint32_t off = (x * KW + kw) * kTile;
                    const char *ks = here + off * S::kRow, *vs = ks + S::kBytes;
                    if (all_seen(at + off)) t.template tile<false>(ks, vs, at + off, key0);
                    else t.template tile<true>(ks, vs, at + off, key0);
                }
            }
        }
        if constexpr (!MANY) break;
        from += kKeysAtOnce;
        if (from >= part_count) break;
        turn_to(from);
        whole = holes == 0;
    }
    const bool again = some && __any(!t.finite());
    if (again) t.reset();
    if constexpr (MANY) {
        if (__syncthreads_or(again)) {
            for (uint32_t from = 0; from < part_count; from += kKeysAtOnce) {
                turn_to(from);
                if (!again) continue;
                for (uint32_t at = kw * kTile; at < padded; at += KW * kTile) t.tile_careful(at, key0, first, last);
            }
        }
    } else if (again) {
        for (uint32_t at = kw * kTile; at < padded; at += KW * kTile) t.tile_careful(at, key0, first, last);
    }

    // the waves' statistics and sums meet in LDS
    t.l = row_sum(t.l);
    if (lane < 16) {
        sm[wave][lane] = t.m;
        sl[wave][lane] = t.l;
    }
    __syncthreads();
    const bool direct = keys.parts <= 1;
    const float vs = a.v_scale ? a.v_scale[hk] : 1.0f;
    {
        float top = kNone;
#pragma unroll
        for (int w = 0; w < KW; ++w) top = fmaxf(top, sm[w * RW + rw][t.c]);
        const float f = t.m == top ? 1.0f : exp2_fast(t.m - top);
#pragma unroll
        for (int b = 0; b < T::kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < T::kEach; ++j) {
                    sums[wave][t.c][b * 128 + (t.g * 4 + i) * T::kEach + j] = t.o[b * T::kEach + j][i] * f;
                }
    }
    __syncthreads();
    constexpr int kPieces = DP / 8;   // of a row
    for (uint32_t x = tid; x < RW * 16 * kPieces; x += kThreads) {
        const uint32_t lr = x / kPieces, d = x % kPieces * 8, r = row0 + lr;
        if (r >= a.rows || d >= a.D) continue;
        const uint32_t w0 = lr / 16, at16 = lr % 16;
        float hi = kNone, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w) hi = fmaxf(hi, sm[w * RW + w0][at16]);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            const float mw = sm[w * RW + w0][at16];
            sum += sl[w * RW + w0][at16] * (mw == hi ? 1.0f : exp2_fast(mw - hi));
        }
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[e] = sums[w0][at16][d + e];
#pragma unroll
            for (int w = 1; w < KW; ++w) y[e] += sums[w * RW + w0][at16][d + e];
        }
        const uint32_t i = r / a.G, h = hk * a.G + (r - i * a.G);
        if (direct) {
            const float inv = sum == 0.0f ? 0.0f : vs / sum;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = sum == 0.0f ? 0.0f : y[e] * inv;
            store8(a, FP16, a.out + n * a.o_n + i * a.o_i + h * a.o_h + d, y);
            if (d == 0 && a.lse) {
                a.lse[((int64_t)n * a.Q + i) * a.Hq + h] =
                    sum == 0.0f ? kNone : (hi - H::kLift + log2f(sum)) * 0.693147180559945309f;
            }
        } else {
            const int64_t at = ((int64_t)owner * a.rows + r) * a.splits + split;
            f32x4* dst = reinterpret_cast<f32x4*>(a.part + at * a.D + d);
            dst[0] = f32x4{y[0], y[1], y[2], y[3]};
            dst[1] = f32x4{y[4], y[5], y[6], y[7]};
            if (d == 0) a.part_ml[at] = float2{hi, sum};
        }
    }
}

// Joins the parts of rows that have several: a workgroup takes 256 / TPR
// pieces of a row, DIMS dims of it, four to a lane, the parts dealt to the
// piece's TPR / (DIMS / 4) lane groups in order.
template <bool FP16, int TPR, int DIMS>
__global__ void __launch_bounds__(256) join_kernel(AttnArgs a)
{
    constexpr uint32_t kLanes = DIMS / 4, kGroups = TPR / kLanes;
    __shared__ f32x4 so[256];
    __shared__ float sl[256];
    const uint32_t tid = threadIdx.x % TPR, first = threadIdx.x - tid;
    const uint32_t cuts = (a.D + DIMS - 1) / DIMS;
    const uint32_t piece = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    const uint32_t all = piece / cuts;   // (owner, row)
    const uint32_t d = (piece - all * cuts) * DIMS + tid % kLanes * 4, grp = tid / kLanes;
    const uint32_t owner = all / a.rows, r = all - owner * a.rows;
    const uint32_t n = owner / a.Hk, hk = owner - n * a.Hk;
    const uint32_t parts = owner < a.N * a.Hk ? keys_of(a, n).parts : 0;
    const int64_t at = (int64_t)all * a.splits;
    f32x4 y = {0, 0, 0, 0};
    float l = 0.0f, top = kNone;
    if (parts > 1) {
        for (uint32_t s = tid; s < parts; s += TPR) top = fmaxf(top, a.part_ml[at + s].x);
    }
#pragma unroll
    for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    if constexpr (TPR > 64) {
        sl[threadIdx.x] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) top = fmaxf(top, sl[first + w * 64]);
        __syncthreads();
    }
    if (parts > 1) {
#pragma unroll 4
        for (uint32_t s = grp; s < parts; s += kGroups) {
            const float2 ml = a.part_ml[at + s];
            const float f = ml.x == top ? 1.0f : exp2_fast(ml.x - top);
            l += ml.y * f;
            if (d < a.D) y += *reinterpret_cast<const f32x4*>(a.part + (at + s) * a.D + d) * f;
        }
    }
    so[threadIdx.x] = y;
    sl[threadIdx.x] = l;
    __syncthreads();
    if (parts <= 1 || tid >= kLanes || d >= a.D) return;
#pragma unroll
    for (uint32_t x = 1; x < kGroups; ++x) {
        y += so[threadIdx.x + x * kLanes];
        l += sl[threadIdx.x + x * kLanes];
    }
    const uint32_t i = r / a.G, h = hk * a.G + (r - i * a.G);
    const float inv = l == 0.0f ? 0.0f : (a.v_scale ? a.v_scale[hk] : 1.0f) / l;
    uint16_t* dst = a.out + n * a.o_n + i * a.o_i + h * a.o_h + d;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float z = l == 0.0f ? 0.0f : y[e] * inv;
        dst[e] = (uint16_t)Half<FP16>::pack(z, 0.0f);
    }
    if (d == 0 && a.lse) {
        a.lse[((int64_t)n * a.Q + i) * a.Hq + h] =
            l == 0.0f ? kNone : (top - Half<FP16>::kLift + log2f(l)) * 0.693147180559945309f;
    }
}

// Which of the kernels.
struct Way {
    int rw;
    bool e4m3, once;
};

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

struct Plan {
    int rw;                        // waves of 16 rows in a workgroup
    int64_t rows, groups, chunk, splits, units;
};

// Rows: as many waves of 16 as hold them, up to the workgroup's 4, so that a
// block of queries reads the cache once; more go to further workgroups, which
// find the keys in their XCD's L2.
//
// Parts: whole rounds of a workgroup's four waves.  A compute unit holds two
// workgroups (one at 256 dims; three of the e4m3 form and of the staged forms at 64,
// which the rule does not count on).  Where all sequences have the same number of
// keys to read (one sequence, or a window), as many parts as fit at once (24
// windows of 1777, 120 owners: 26 us with 4 parts, 33 with 5); where lengths may
// differ, a quarter more, so that long ones do not run alone (32 sequences up to
// 4096: 61 us with 2 parts, 56 with 3).  A part has no more keys than the table of
// places, but for two cases in which its workgroup goes through several tables:
// the parts' sums would take more than kMostWords (2048 sequences of 1009 under a
// bound of 131072: 2.1 ms with 31 parts, 2.8 with 64), or one sequence's groups of
// rows alone fill the chip four times over, and parts would only add their sums
// (4096 queries over 32768 keys, 32 heads on 8: 4.3 ms, 7.1 in 32 parts; over 8192
// keys 1.30 and 1.50 in 8).
constexpr int64_t kMostWords = (int64_t)1 << 27;   // 1 GiB

// Workspace words (8 bytes) of one part of every row: sums and (m, l).
int64_t words_a_part(const Shape& s) { return s.N * s.Q * s.Hq * (s.dim + 2) / 2; }

Plan plan_of(const Shape& s)
{
    Plan p;
    p.rows = s.Q * (s.Hq / s.heads);
    const int64_t tiles = (p.rows + 15) / 16;
    p.rw = tiles <= 1 ? 1 : tiles <= 2 ? 2 : 4;
    p.groups = (tiles + p.rw - 1) / p.rw;
    int64_t span = s.max_len;
    if (s.window > 0 && s.window + s.Q - 1 < span) span = s.window + s.Q - 1;
    const int64_t owners = s.N * s.heads, wide = owners * p.groups;
    const int64_t slots = (s.dim > 128 ? 1 : 2) * (int64_t)kUnits;
    const bool even = s.N == 1 || s.window > 0 || s.dim > 128;
    int64_t want = even ? slots / wide : (slots * 5 / 4 + wide - 1) / wide;
    if (want < 1) want = 1;
    const int64_t table = p.rw > 1 ? kTableStaged : kTable;
    auto rounds = [](int64_t keys) {   // at most 2^30, so that a part's end is in 32 bits
        const int64_t up = (keys + kRound - 1) / kRound * kRound;
        return up < (1 << 30) ? up : (int64_t)1 << 30;
    };
    p.chunk = rounds((span + want - 1) / want);
    if (p.chunk > table && !(s.N == 1 && wide >= 4 * slots)) p.chunk = table;
    p.splits = (span + p.chunk - 1) / p.chunk;
    if (p.splits > 1 && p.splits * words_a_part(s) > kMostWords) {
        const int64_t fit = kMostWords / words_a_part(s);
        p.chunk = rounds(fit > 1 ? (span + fit - 1) / fit : span);
        p.splits = (span + p.chunk - 1) / p.chunk;
    }
    p.units = owners * p.splits;
    return p;
}

// Workgroups and part sums in 32 bits.
bool plan_ok(const Shape& s, const Plan& p)
{
    return p.units <= 0x7FFFFFFFll / p.groups / 8;
}

int64_t plan_words(const Shape& s, const Plan& p)
{
    return p.splits > 1 ? p.splits * words_a_part(s) : 0;
}

// Workgroups of one launch: a grid has fewer than 2^32 threads.  (A multiple of 8,
// for the XCDs.)
constexpr uint32_t kMostGroups = 1u << 22;

template <bool FP16, bool E4M3, int DP, int RW, bool ONCE, bool MANY>
void launch_one(AttnArgs a, hipStream_t stream)
{
    const uint32_t grid = (a.units + 7) / 8 * 8 * a.groups;
    for (a.first = 0; a.first < grid; a.first += kMostGroups) {
        const uint32_t n = grid - a.first < kMostGroups ? grid - a.first : kMostGroups;
        hipLaunchKernelGGL((attention_kernel<FP16, E4M3, DP, RW, ONCE, MANY>), dim3(n), dim3(kThreads), 0,
                           stream, a);
    }
}

template <bool FP16, bool E4M3, int DP, int RW>
void launch_waves(const AttnArgs& a, bool once, hipStream_t stream)
{
    if (a.chunk > (uint32_t)(RW > 1 ? kTableStaged : kTable)) {
        launch_one<FP16, E4M3, DP, RW, false, true>(a, stream);
    } else if (once) {
        launch_one<FP16, E4M3, DP, RW, true, false>(a, stream);
    } else {
        launch_one<FP16, E4M3, DP, RW, false, false>(a, stream);
    }
}

template <bool FP16, bool E4M3, int DP>
void launch_rows(const AttnArgs& a, const Way& way, hipStream_t stream)
{
    if (way.rw == 1) launch_waves<FP16, E4M3, DP, 1>(a, way.once, stream);
    else if (way.rw == 2) launch_waves<FP16, E4M3, DP, 2>(a, way.once, stream);
    else launch_waves<FP16, E4M3, DP, 4>(a, way.once, stream);
}

template <bool FP16, bool E4M3>
void launch_dims(const AttnArgs& a, const Way& way, hipStream_t stream)
{
    if (a.D <= 64) return launch_rows<FP16, E4M3, 64>(a, way, stream);
    if (a.D <= 128) return launch_rows<FP16, E4M3, 128>(a, way, stream);
    return launch_rows<FP16, E4M3, 256>(a, way, stream);
}

template <bool FP16>
hipError_t launch_attention(const AttnArgs& a, const Way& way, hipStream_t stream)
{
    if (way.e4m3) launch_dims<FP16, true>(a, way, stream);
    else launch_dims<FP16, false>(a, way, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const uint32_t rows = a.N * a.Hk * a.rows;
    // few parts: a wave a row's 128 dims; many: a workgroup 32 dims
    if (a.splits <= 16) {
        const uint32_t pieces = rows * ((a.D + 127) / 128);
        hipLaunchKernelGGL((join_kernel<FP16, 64, 128>), dim3((pieces + 3) / 4), dim3(256), 0, stream, a);
    } else {
        const uint32_t pieces = rows * ((a.D + 31) / 32);
        hipLaunchKernelGGL((join_kernel<FP16, 256, 32>), dim3(pieces), dim3(256), 0, stream, a);
    }
    return hipGetLastError();
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
    // every row's start; the stride of a dimension of one place moves none
    const Dim moves[3] = {{c.pages, c.stride_page}, {c.heads, c.stride_head}, {c.page_size, c.stride_token}};
    if (c.dim * e % 16 != 0 || !is_aligned16(c.k) || !is_aligned16(c.v)) return XPRESS_EINVAL;
    for (const Dim& d : moves) {
        if (d.n > 1 && d.stride * e % 16 != 0) return XPRESS_EINVAL;
    }
    const double scale2 = x.scale * 1.4426950408889634;   // scores are taken in base 2
    if (x.max_len > c.table_width * c.page_size || !isfinite((float)scale2)) return XPRESS_EINVAL;
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

    const Plan p = plan_of(s);
    if (!plan_ok(s, p)) return XPRESS_EINVAL;

    AttnArgs a;
    a.q = (const uint16_t*)x.q;
    a.out = (uint16_t*)x.out;
    a.lse = x.lse;
    a.part = nullptr;
    a.part_ml = nullptr;
    a.lens = x.lens;
    a.page_table = c.page_table;
    a.kc = (const char*)c.k;
    a.vc = (const char*)c.v;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    a.q_n = x.stride_q_n;
    a.q_i = x.stride_q_i;
    a.q_h = x.stride_q_h;
    a.o_n = x.stride_o_n;
    a.o_i = x.stride_o_i;
    a.o_h = x.stride_o_h;
    a.page = c.stride_page * e;
    a.head = c.stride_head * e;
    a.token = c.stride_token * e;
    a.table = c.stride_table;
    a.N = (uint32_t)s.N;
    a.Q = (uint32_t)s.Q;
    a.Hq = (uint32_t)s.Hq;
    a.Hk = (uint32_t)s.heads;
    a.G = (uint32_t)(s.Hq / s.heads);
    a.D = (uint32_t)s.dim;
    a.pages = (uint32_t)c.pages;
    a.page_size = (uint32_t)c.page_size;
    a.rows = (uint32_t)p.rows;
    a.groups = (uint32_t)p.groups;
    a.units = (uint32_t)p.units;
    a.chunk = (uint32_t)p.chunk;
    a.splits = (uint32_t)p.splits;
    a.max_len = (int32_t)x.max_len;
    a.window = (int32_t)x.window;
    a.first = 0;
    a.scale = (float)scale2;
    a.wide = is_aligned16(x.q) && is_aligned16(x.out) &&
             (x.stride_q_n | x.stride_q_i | x.stride_q_h | x.stride_o_n | x.stride_o_i | x.stride_o_h) % 8 == 0;
    if (p.splits > 1) {
        uint64_t* table = nullptr;
        const int rc = workspace_table(stream, plan_words(s, p), &table);
        if (rc != XPRESS_OK) return rc;
        a.part = reinterpret_cast<float*>(table);
        a.part_ml = reinterpret_cast<float2*>(a.part + s.N * s.Q * s.Hq * p.splits * s.dim);
    }
    // Loads pass the caches by where each 128-byte line is read by one workgroup:
    // whole lines in a head's row or run of rows, and no second group of rows
    // (token-major rows of 160 bytes: 62 us through the caches, 80 past them;
    // head-major rows of 256 bytes: 69 and 63).
    const Way way = {p.rw, c.dtype == XPRESS_E4M3,
                     p.groups == 1 && (c.stride_token == c.dim || c.dim * e % 128 == 0)};
    const hipError_t err = x.dtype == XPRESS_FP16 ? launch_attention<true>(a, way, stream)
                                                  : launch_attention<false>(a, way, stream);
    return err == hipSuccess ? XPRESS_OK : hip_fail(err);
}

int xpress_paged_attention_reserve(int64_t N, int64_t Q, int64_t Hq, int64_t heads, int64_t dim,
                                   int64_t max_len, int64_t window, hipStream_t stream)
{
    const Shape s = {N, Q, Hq, heads, dim, max_len, window};
    if (!shape_ok(s)) return XPRESS_EINVAL;
    if (N == 0 || Q == 0) return XPRESS_OK;
    const Plan p = plan_of(s);
    if (!plan_ok(s, p)) return XPRESS_EINVAL;
    if (p.splits == 1) return XPRESS_OK;
    uint64_t* table = nullptr;
    return workspace_table(stream, plan_words(s, p), &table);
}

int xpress_paged_attention_plan(int64_t N, int64_t Q, int64_t Hq, int64_t heads, int64_t dim,
                                int64_t max_len, int64_t window, int* chunk, int* splits, int* rows,
                                int* launches)
{
    const Shape s = {N, Q, Hq, heads, dim, max_len, window};
    if (!shape_ok(s)) return XPRESS_EINVAL;
    Plan p = {1, 0, 0, 0, 0, 0};
    if (N > 0 && Q > 0) {
        p = plan_of(s);
        if (!plan_ok(s, p)) return XPRESS_EINVAL;
    }
    if (chunk) *chunk = (int)p.chunk;
    if (splits) *splits = (int)p.splits;
    if (rows) *rows = 16 * p.rw;
    if (launches) *launches = p.splits > 1 ? 2 : (int)p.splits;
    return XPRESS_OK;
}

}  // extern "C"
