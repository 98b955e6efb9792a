// kv_pages.hip -- the pages of a paged key-value cache: handed out, shared by forks,
// copied where a fork parts from its source, given back, and moved together after a
// tree of drafts was cut down to one path (gfx950).
//
// What is known of the pool is one number a page, how many table entries name it; a
// page that none names is free.  Free pages are taken lowest first, in the order of
// the tables' rows: a result does not depend on the order in which workgroups run, and
// nothing has to be kept beside the counts.  One workgroup hands pages out: it goes
// through the counts 4096 at a time, as far as it needs to, with a running sum over the
// workgroup for the pages' ranks.  (The counts are few: 7399 pages of the 32 sequences
// of 8 beams are two steps; 60000 used pages before the first free one are 15, and cost
// 25 us.)  All other work is spread over the chip.
//
// Bound by latency: a handful of dependent loads a launch.  Measured: a fork of 256 rows
// (pages of 16 tokens, 83 slots a row, 7399 pages) 5.0 us for the plan, 3.8 for the rows and
// 5.6 for the copies, 9 MB; of 4 rows 4.1, 3.0 and 2.9.  256 sequences of up to 8192 tokens
// give back what left their window in 2.8 us and take 64 tokens' pages in 7.0.  64 paths of up
// to 12 nodes move in 5.7 us (with 8 moves at once 6.4).

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "device_common.h"
#include "host_common.h"
#include "kv_common.h"
#include "xpress_argmax.h"

namespace {

using namespace xpress;

constexpr uint32_t kThreads = 1024;     // of a workgroup that hands pages out
constexpr uint32_t kWaves = kThreads / 64;
constexpr uint32_t kStep = kThreads * 4;   // counts looked at in one step
constexpr uint32_t kMostWanted = kThreads * 2;   // pages asked for at once
constexpr uint32_t kWindow = 8192;      // sources whose first child is looked for at once
constexpr uint32_t kRowThreads = 256;

// Sum of v over the threads before this one, and over all of them.
__device__ __forceinline__ uint32_t ranks(uint32_t v, uint32_t* sums, uint32_t* total)
{
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    uint32_t x = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t y = __shfl_up(x, d);
        if (lane >= (uint32_t)d) x += y;
    }
    __syncthreads();   // the sums of the call before have been read
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

// The pool's free pages in ascending order, found as they are asked for.  (Counts loaded
// a step ahead: 7.9 us for 256 sequences' pages where this takes 7.0; each barrier waits
// for them.)
struct FreePages {
    struct Shared {
        int32_t list[kStep + kMostWanted];
        uint32_t sums[kWaves];
    };
    Shared& s;
    const int32_t* refs;
    uint32_t pages, next, have;   // counts looked at; pages in the list

    // At least `want`, kMostWanted or fewer, in the list, if there are as many.
    __device__ void fill(uint32_t want)
    {
        while (have < want && next < pages) {
            const uint32_t at = next + threadIdx.x * 4;
            uint32_t free = 0;
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) free |= (uint32_t)(at + i < pages && refs[at + i] == 0) << i;
            uint32_t found;
            uint32_t to = have + ranks(__popc(free), s.sums, &found);
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                if (free >> i & 1) s.list[to++] = (int32_t)(at + i);
            }
            have += found;
            next = pages - next > kStep ? next + kStep : pages;
        }
        __syncthreads();
    }

    // The first n leave the list.
    __device__ void drop(uint32_t n)
    {
        constexpr uint32_t kEach = (kStep + kMostWanted) / kThreads;
        __syncthreads();
        const uint32_t left = have - n;
        int32_t keep[kEach];
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i) {
            const uint32_t at = i * kThreads + threadIdx.x;
            keep[i] = at < left ? s.list[n + at] : 0;
        }
        __syncthreads();
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i) {
            const uint32_t at = i * kThreads + threadIdx.x;
            if (at < left) s.list[at] = keep[i];
        }
        have = left;
        __syncthreads();
    }
};

struct ForkArgs {
    const int32_t *refs, *table, *lens, *src;
    int32_t *new_refs, *new_table, *copies, *missing;
    int64_t stride_table, stride_new;
    uint32_t pages, page_size, N, M, width;
};

// Tokens of source n.
__device__ __forceinline__ uint32_t length_of(const ForkArgs& a, uint32_t n)
{
    const int32_t len = a.lens[n];
    const uint32_t most = a.width * a.page_size;
    return len <= 0 ? 0 : (uint32_t)len < most ? (uint32_t)len : most;
}

// First launch of a fork.  Workgroup 0: which rows need a page of their own for their
// last tokens, and which page; the others copy the counts.
__global__ void __launch_bounds__(kThreads) fork_plan_kernel(ForkArgs a)
{
    if (blockIdx.x > 0) {
        const uint32_t step = (gridDim.x - 1) * kThreads;
        for (uint32_t i = (blockIdx.x - 1) * kThreads + threadIdx.x; i < a.pages; i += step) {
            a.new_refs[i] = a.refs[i];
            if (a.pages - i <= step) break;
        }
        return;
    }
    __shared__ FreePages::Shared s;
    __shared__ uint32_t first[kWindow];
    // copies[m, 2]: whether row m is its source's first
    for (uint32_t n0 = 0; n0 < a.N; n0 += kWindow) {
        const uint32_t count = min(a.N - n0, kWindow);
        for (uint32_t i = threadIdx.x; i < count; i += kThreads) first[i] = ~0u;
        __syncthreads();
        for (uint32_t m = threadIdx.x; m < a.M; m += kThreads) {
            const uint32_t at = (uint32_t)a.src[m] - n0;
            if (at < count) atomicMin(&first[at], m);
        }
        __syncthreads();
        for (uint32_t m = threadIdx.x; m < a.M; m += kThreads) {
            const uint32_t at = (uint32_t)a.src[m] - n0;
            if (at < count) a.copies[(int64_t)m * 3 + 2] = first[at] == m;
        }
        __syncthreads();
    }
    FreePages pool = {s, a.refs, a.pages, 0, 0};
    uint32_t short_of = 0;
    for (uint32_t m0 = 0; m0 < a.M; m0 += kThreads) {
        const uint32_t m = m0 + threadIdx.x;
        bool want = false;
        uint32_t part = 0, last = 0;
        int32_t p = -1;
        if (m < a.M) {
            const uint32_t n = (uint32_t)a.src[m];
            if (n < a.N) {
                const uint32_t len = length_of(a, n);
                last = len / a.page_size;
                part = len - last * a.page_size;
                if (part > 0) {
                    p = a.table[(int64_t)n * a.stride_table + last];
                    want = (uint32_t)p < a.pages && !(a.copies[(int64_t)m * 3 + 2] != 0 && a.refs[p] == 1);
                }
            }
        }
        uint32_t total;
        const uint32_t rank = ranks(want, s.sums, &total);
        pool.fill(total);
        const bool got = want && rank < pool.have;
        if (m < a.M) {
            const int32_t fresh = got ? s.list[rank] : -1;
            if (part > 0) a.new_table[(int64_t)m * a.stride_new + last] = want ? fresh : p;
            int32_t* c = a.copies + (int64_t)m * 3;
            c[0] = got ? p : -1;
            c[1] = fresh;
            c[2] = got ? (int32_t)part : 0;
        }
        const uint32_t used = min(total, pool.have);
        short_of += total - used;
        if (m0 + kThreads < a.M && m0 + kThreads > m0) pool.drop(used);
        else break;
    }
    if (threadIdx.x == 0 && a.missing) a.missing[0] = (int32_t)short_of;
}

// Second launch: row i of the new table and what it adds to the counts, and what
// becomes of source i's entries.  A source's first row takes over its entries'
// counts, so that rows which go on alone touch none.
__global__ void __launch_bounds__(kRowThreads) fork_rows_kernel(ForkArgs a)
{
    __shared__ uint32_t has_child, has_elder;
    const uint32_t i = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) has_child = has_elder = 0;
    __syncthreads();
    const uint32_t mine = i < a.M ? (uint32_t)a.src[i] : ~0u;
    bool child = false, elder = false;
    for (uint32_t m = tid; m < a.M; m += kRowThreads) {
        const uint32_t n = (uint32_t)a.src[m];
        child |= n == i;
        elder |= n == mine && m < i;
        if (a.M - m <= kRowThreads) break;
    }
    if (child) has_child = 1;
    if (elder) has_elder = 1;
    __syncthreads();
    child = has_child != 0;
    elder = has_elder != 0;
    if (i < a.M) {
        int32_t* to = a.new_table + (int64_t)i * a.stride_new;
        const bool ok = mine < a.N;
        const uint32_t len = ok ? length_of(a, mine) : 0, whole = len / a.page_size;
        const uint32_t kept = len > whole * a.page_size ? whole : ~0u;   // the first launch's
        const int32_t* from = a.table + (int64_t)(ok ? mine : 0) * a.stride_table;
        for (uint32_t s = tid; s < a.width; s += kRowThreads) {
            if (s == kept) continue;
            const int32_t p = s < whole ? from[s] : -1;
            to[s] = p;
            if (elder && (uint32_t)p < a.pages) atomicAdd(&a.new_refs[p], 1);
        }
        if (tid == 0) {
            const int32_t fresh = a.copies[(int64_t)i * 3 + 1];
            if (fresh >= 0) atomicAdd(&a.new_refs[fresh], 1);
        }
    }
    if (i < a.N) {
        const uint32_t len = length_of(a, i), whole = len / a.page_size;
        const bool part = len > whole * a.page_size;
        for (uint32_t s = (child ? whole : 0) + tid; s < a.width; s += kRowThreads) {
            const int32_t p = a.table[(int64_t)i * a.stride_table + s];
            if ((uint32_t)p >= a.pages || (child && part && s == whole && a.refs[p] == 1)) continue;
            atomicSub(&a.new_refs[p], 1);
        }
    }
}

struct CopyArgs {
    const int32_t* copies;
    char *k, *v;
    int64_t page, head, token;   // bytes
    uint32_t count, pages, page_size, heads, pieces;
};

// A workgroup takes one entry's keys or values (blockIdx.y even or odd) and a share of
// its (head, token, piece) items, pieces of W bytes.
template <typename W>
__global__ void __launch_bounds__(kRowThreads) copy_kernel(CopyArgs a)
{
    const uint32_t shares = gridDim.y / 2, share = blockIdx.y / 2;
    char* base = blockIdx.y & 1 ? a.v : a.k;
    for (uint32_t c = blockIdx.x; c < a.count; c += gridDim.x) {
        const uint32_t from = (uint32_t)a.copies[(int64_t)c * 3], to = (uint32_t)a.copies[(int64_t)c * 3 + 1];
        const int32_t asked = a.copies[(int64_t)c * 3 + 2];
        const uint32_t tokens = asked <= 0 ? 0 : min((uint32_t)asked, a.page_size);
        if (from >= a.pages || to >= a.pages || from == to) continue;
        const char* src = base + (int64_t)from * a.page;
        char* dst = base + (int64_t)to * a.page;
        const uint32_t items = tokens * a.heads * a.pieces;
        for (uint32_t i = share * kRowThreads + threadIdx.x; i < items; i += shares * kRowThreads) {
            const uint32_t row = i / a.pieces, piece = i - row * a.pieces;
            const uint32_t head = row / tokens, token = row - head * tokens;
            const int64_t at = head * a.head + token * a.token + (int64_t)piece * sizeof(W);
            *reinterpret_cast<W*>(dst + at) = *reinterpret_cast<const W*>(src + at);
        }
    }
}

struct GrowArgs {
    int32_t *refs, *table, *missing;
    const int32_t *have, *want;
    int64_t stride_table;
    uint32_t pages, page_size, N, width;
};

__device__ __forceinline__ uint32_t slots_of(int32_t len, const GrowArgs& a)
{
    const uint32_t s = len <= 0 ? 0 : ((uint32_t)len - 1) / a.page_size + 1;
    return min(s, a.width);
}

// One workgroup: sequences 1024 at a time, their wanted slots one after the other.
__global__ void __launch_bounds__(kThreads) grow_kernel(GrowArgs a)
{
    __shared__ FreePages::Shared s;
    __shared__ uint32_t begin[kThreads], slot0[kThreads];   // of a sequence's slots among all
    FreePages pool = {s, a.refs, a.pages, 0, 0};
    uint32_t short_of = 0;
    for (uint32_t n0 = 0; n0 < a.N; n0 += kThreads) {
        const uint32_t n = n0 + threadIdx.x;
        uint32_t lo = 0, hi = 0;
        if (n < a.N) {
            lo = slots_of(a.have[n], a);
            hi = slots_of(a.want[n], a);
        }
        const uint32_t mine = hi > lo ? hi - lo : 0;
        uint32_t all;
        const uint32_t at = ranks(mine, s.sums, &all);
        begin[threadIdx.x] = at;
        slot0[threadIdx.x] = lo;
        __syncthreads();
        for (uint32_t i0 = 0; i0 < all; i0 += 2 * kThreads) {
            // two slots a thread, one after the other
            bool lacks[2];
            int32_t* entry[2];
#pragma unroll
            for (uint32_t e = 0; e < 2; ++e) {
                const uint32_t i = i0 + 2 * threadIdx.x + e;
                lacks[e] = false;
                entry[e] = nullptr;
                if (i < all) {
                    uint32_t x = 0;   // the last sequence that begins at or before slot i
#pragma unroll
                    for (uint32_t d = kThreads / 2; d > 0; d /= 2) {
                        if (begin[x + d] <= i) x += d;
                    }
                    entry[e] = a.table + (int64_t)(n0 + x) * a.stride_table + slot0[x] + (i - begin[x]);
                    lacks[e] = (uint32_t)*entry[e] >= a.pages;
                }
            }
            uint32_t total;
            uint32_t rank = ranks((uint32_t)lacks[0] + lacks[1], s.sums, &total);
            if (total == 0) continue;
            pool.fill(total);
#pragma unroll
            for (uint32_t e = 0; e < 2; ++e) {
                if (lacks[e] && rank < pool.have) {
                    const int32_t p = s.list[rank];
                    *entry[e] = p;
                    a.refs[p] = 1;
                }
                rank += lacks[e];
            }
            const uint32_t used = min(total, pool.have);
            short_of += total - used;
            if (i0 + 2 * kThreads >= all && a.N - n0 <= kThreads) break;   // the last
            pool.drop(used);
        }
        __syncthreads();
        if (a.N - n0 <= kThreads) break;
    }
    if (threadIdx.x == 0 && a.missing) a.missing[0] = (int32_t)short_of;
}

struct FreeArgs {
    int32_t *refs, *table;
    const int32_t* lens;
    int64_t stride_table, window, sinks;
    uint32_t pages, page_size, N, width;
};

__global__ void __launch_bounds__(kRowThreads) free_kernel(FreeArgs a)
{
    for (uint32_t n = blockIdx.y; n < a.N; n += gridDim.y) {
        const int64_t len = a.lens[n];
        for (uint32_t s = blockIdx.x * kRowThreads + threadIdx.x; s < a.width; s += gridDim.x * kRowThreads) {
            const int64_t first = (int64_t)s * a.page_size, end = first + a.page_size;
            // the next query stands at len and sees keys from len - window + 1 on
            if (first < len && (a.window == 0 || first < a.sinks || end > len - a.window + 1)) continue;
            int32_t* entry = a.table + (int64_t)n * a.stride_table + s;
            const int32_t p = *entry;
            if (p == -1) continue;
            *entry = -1;
            if ((uint32_t)p < a.pages) atomicSub(&a.refs[p], 1);
        }
    }
}

struct CompactArgs {
    char *k, *v;
    const int32_t *table, *start, *path, *count;
    int64_t page, head, token, stride_table, stride_path;   // of the cache in bytes
    uint32_t pages, page_size, N, width, longest, heads, pieces;
};

constexpr uint32_t kPath = 256;    // kept nodes whose places LDS holds at once
constexpr uint32_t kAtOnce = 16;   // rows a thread reads before it writes them

// A thread owns a piece of W bytes of one head's keys or values of one sequence and
// moves it for the kept nodes in order.  Nodes ascend and so do their places, each at
// or after the one it goes to: a place is read before the thread writes it, without a
// wait between threads.
template <typename W>
__global__ void __launch_bounds__(kRowThreads) compact_kernel(CompactArgs a)
{
    __shared__ int64_t from[kPath], to[kPath];
    __shared__ uint32_t end;
    const uint32_t items = 2 * a.heads * a.pieces;
    for (uint32_t n = blockIdx.y; n < a.N; n += gridDim.y) {
        const int32_t start = a.start[n], asked = a.count[n];
        const uint32_t kept = start < 0 || asked <= 0 ? 0 : min((uint32_t)asked, a.longest);
        const int32_t* path = a.path + (int64_t)n * a.stride_path;
        bool whole = true;
        for (uint32_t j0 = 0; j0 < kept && whole; j0 += kPath) {
            const uint32_t here = min(kept - j0, kPath);
            __syncthreads();
            if (threadIdx.x == 0) end = here;
            __syncthreads();
            if (threadIdx.x < here) {
                const uint32_t j = j0 + threadIdx.x;
                const int32_t node = path[j], before = j ? path[j - 1] : -1;
                if (node <= before) atomicMin(&end, threadIdx.x);   // not ascending: the path ends
                auto find = [&](int64_t place) -> int64_t {
                    const int64_t slot = place / a.page_size;
                    if (slot >= a.width) return -1;
                    const uint32_t p = (uint32_t)a.table[(int64_t)n * a.stride_table + slot];
                    if (p >= a.pages) return -1;
                    return (int64_t)p * a.page + (place - slot * a.page_size) * a.token;
                };
                const bool moves = node > before && node != (int32_t)j;
                const int64_t old = moves ? find((int64_t)start + node) : -1;
                const int64_t at = moves ? find((int64_t)start + j) : -1;
                from[threadIdx.x] = old >= 0 && at >= 0 ? old : -1;
                to[threadIdx.x] = at;
            }
            __syncthreads();
            const uint32_t last = end;
            whole = last == here;
            for (uint32_t i = blockIdx.x * kRowThreads + threadIdx.x; i < items; i += gridDim.x * kRowThreads) {
                const uint32_t row = i / a.pieces, piece = i - row * a.pieces;
                const uint32_t head = row / 2;
                char* base = (row & 1 ? a.v : a.k) + head * a.head + (int64_t)piece * sizeof(W);
                for (uint32_t j = 0; j < last; j += kAtOnce) {
                    W x[kAtOnce];
#pragma unroll
                    for (uint32_t e = 0; e < kAtOnce; ++e) {
                        const int64_t at = j + e < last ? from[j + e] : -1;
                        if (at >= 0) x[e] = *reinterpret_cast<const W*>(base + at);
                    }
#pragma unroll
                    for (uint32_t e = 0; e < kAtOnce; ++e) {
                        if (j + e < last && from[j + e] >= 0) *reinterpret_cast<W*>(base + to[j + e]) = x[e];
                    }
                }
            }
        }
    }
}

// The widest piece, in bytes, that divides every row and its places.
uint32_t piece_of(const xpress_kv_cache& c)
{
    const int64_t e = element_bytes(c.dtype);
    const Dim moves[3] = {{c.pages, c.stride_page}, {c.heads, c.stride_head}, {c.page_size, c.stride_token}};
    uint32_t w = 16;
    for (; w > 1; w /= 2) {
        bool ok = c.dim * e % w == 0 && is_aligned(c.k, w) && is_aligned(c.v, w);
        for (const Dim& d : moves) ok = ok && (d.n <= 1 || d.stride * e % w == 0);
        if (ok) break;
    }
    return w;
}

// A list of int32 arrays none of which may share bytes with another.
struct Range {
    const void* p;
    size_t n;
};

template <int K, int L>
bool all_apart(const Range (&written)[K], const Range (&read)[L])
{
    for (int i = 0; i < K; ++i) {
        if (!written[i].p) continue;
        for (int j = 0; j < i; ++j) {
            if (written[j].p && ranges_overlap(written[i].p, written[i].n, written[j].p, written[j].n)) return false;
        }
        for (int j = 0; j < L; ++j) {
            if (read[j].p && ranges_overlap(written[i].p, written[i].n, read[j].p, read[j].n)) return false;
        }
    }
    return true;
}

int done(hipError_t e) { return e == hipSuccess ? XPRESS_OK : hip_fail(e); }

constexpr int64_t kMost = 0x7FFFFFFFll;

bool numbers_ok(const void* p) { return p && is_aligned(p, 4); }

}  // namespace

extern "C" {

int xpress_kv_fork(const int32_t* refs, int64_t pages, const int32_t* table, int64_t stride_table,
                   const int32_t* lens, int64_t N, const int32_t* src, int64_t M, int64_t width,
                   int64_t page_size, int32_t* new_refs, int32_t* new_table, int64_t stride_new,
                   int32_t* copies, int32_t* missing, hipStream_t stream)
{
    // every row looks through all of src
    const int64_t rows = N > M ? N : M;
    if (N < 0 || M < 0 || rows > 65536 || pages < 1 || pages > kMost) return XPRESS_EINVAL;
    if (!numbers_ok(refs) || !numbers_ok(new_refs) || !is_aligned(missing, 4)) return XPRESS_EINVAL;
    if (N > 0 && (!table_ok(table, N, width, stride_table, page_size) || !numbers_ok(lens))) return XPRESS_EINVAL;
    if (M > 0 && (!table_ok(new_table, M, width, stride_new, page_size) || !numbers_ok(src) ||
                  !numbers_ok(copies))) {
        return XPRESS_EINVAL;
    }
    const Range written[] = {{new_refs, (size_t)pages * 4u},
                             {M > 0 ? new_table : nullptr, table_bytes(M, width, stride_new)},
                             {M > 0 ? copies : nullptr, (size_t)M * 12u},
                             {missing, 4u}};
    const Range read[] = {{refs, (size_t)pages * 4u},
                          {N > 0 ? table : nullptr, table_bytes(N, width, stride_table)},
                          {N > 0 ? lens : nullptr, (size_t)N * 4u},
                          {M > 0 ? src : nullptr, (size_t)M * 4u}};
    if (!all_apart(written, read)) return XPRESS_EINVAL;
    ForkArgs a = {refs, table, lens, src, new_refs, new_table, copies, missing, stride_table, stride_new,
                  (uint32_t)pages, (uint32_t)page_size, (uint32_t)N, (uint32_t)M, (uint32_t)width};
    const uint32_t others = (uint32_t)((pages + kThreads - 1) / kThreads);
    hipLaunchKernelGGL(fork_plan_kernel, dim3(1 + (others < 256u ? others : 256u)), dim3(kThreads), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || rows == 0) return done(e);
    hipLaunchKernelGGL(fork_rows_kernel, dim3((uint32_t)rows), dim3(kRowThreads), 0, stream, a);
    return done(hipGetLastError());
}

int xpress_kv_copy(const xpress_kv_cache* cache, const int32_t* copies, int64_t count, hipStream_t stream)
{
    if (!cache) return XPRESS_EINVAL;
    const xpress_kv_cache& c = *cache;
    size_t bytes = 0;
    if (count < 0 || count > kMost / 3 || !pool_ok(c, &bytes)) return XPRESS_EINVAL;
    if (count == 0) return XPRESS_OK;
    if (!numbers_ok(copies) || !apart_from_cache(c, bytes, copies, (size_t)count * 12u)) return XPRESS_EINVAL;
    const int64_t e = element_bytes(c.dtype);
    const uint32_t w = piece_of(c);
    // a page's pieces in 31 bits
    if (c.heads * c.dim * e / w > kMost / c.page_size) return XPRESS_EINVAL;
    CopyArgs a = {copies, (char*)c.k, (char*)c.v, c.stride_page * e, c.stride_head * e, c.stride_token * e,
                  (uint32_t)count, (uint32_t)c.pages, (uint32_t)c.page_size, (uint32_t)c.heads,
                  (uint32_t)(c.dim * e / w)};
    // a thread takes up to eight pieces of a full page
    const uint64_t items = (uint64_t)a.page_size * a.heads * a.pieces;
    uint64_t shares = (items + 8 * kRowThreads - 1) / (8 * kRowThreads);
    if (shares > 64) shares = 64;
    const dim3 grid(a.count < (1u << 16) ? a.count : 1u << 16, 2 * (uint32_t)shares);
    const dim3 block(kRowThreads);
    if (w == 16) hipLaunchKernelGGL(copy_kernel<u32x4>, grid, block, 0, stream, a);
    else if (w == 8) hipLaunchKernelGGL(copy_kernel<uint64_t>, grid, block, 0, stream, a);
    else if (w == 4) hipLaunchKernelGGL(copy_kernel<uint32_t>, grid, block, 0, stream, a);
    else if (w == 2) hipLaunchKernelGGL(copy_kernel<uint16_t>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(copy_kernel<uint8_t>, grid, block, 0, stream, a);
    return done(hipGetLastError());
}

int xpress_kv_grow(int32_t* refs, int64_t pages, int32_t* table, int64_t stride_table, int64_t N,
                   int64_t width, int64_t page_size, const int32_t* have, const int32_t* want,
                   int32_t* missing, hipStream_t stream)
{
    if (N < 0 || N > kMost || pages < 1 || pages > kMost || !numbers_ok(refs) || !is_aligned(missing, 4)) {
        return XPRESS_EINVAL;
    }
    if (N > 0 && (!table_ok(table, N, width, stride_table, page_size) || !numbers_ok(have) || !numbers_ok(want))) {
        return XPRESS_EINVAL;
    }
    if (N > 0 && width > kMost / (int64_t)kThreads) return XPRESS_EINVAL;   // a step's slots in 32 bits
    const Range written[] = {{refs, (size_t)pages * 4u},
                             {N > 0 ? table : nullptr, table_bytes(N, width, stride_table)},
                             {missing, 4u}};
    const Range read[] = {{N > 0 ? have : nullptr, (size_t)N * 4u}, {N > 0 ? want : nullptr, (size_t)N * 4u}};
    if (!all_apart(written, read)) return XPRESS_EINVAL;
    if (N == 0 && !missing) return XPRESS_OK;
    GrowArgs a = {refs, table, missing, have, want, stride_table,
                  (uint32_t)pages, (uint32_t)page_size, (uint32_t)N, (uint32_t)width};
    hipLaunchKernelGGL(grow_kernel, dim3(1), dim3(kThreads), 0, stream, a);
    return done(hipGetLastError());
}

int xpress_kv_free(int32_t* refs, int64_t pages, int32_t* table, int64_t stride_table, int64_t N,
                   int64_t width, int64_t page_size, const int32_t* lens, int64_t window, int64_t sinks,
                   hipStream_t stream)
{
    if (N < 0 || N > kMost || pages < 1 || pages > kMost || window < 0 || window > kMost || sinks < 0 ||
        sinks > kMost || !numbers_ok(refs)) {
        return XPRESS_EINVAL;
    }
    if (N == 0) return XPRESS_OK;
    if (!table_ok(table, N, width, stride_table, page_size) || !numbers_ok(lens)) return XPRESS_EINVAL;
    const Range written[] = {{refs, (size_t)pages * 4u}, {table, table_bytes(N, width, stride_table)}};
    const Range read[] = {{lens, (size_t)N * 4u}};
    if (!all_apart(written, read)) return XPRESS_EINVAL;
    FreeArgs a = {refs, table, lens, stride_table, window, sinks,
                  (uint32_t)pages, (uint32_t)page_size, (uint32_t)N, (uint32_t)width};
    const uint32_t gx = (uint32_t)((width + kRowThreads - 1) / kRowThreads);
    const uint32_t gy = N < 65535 ? (uint32_t)N : 65535u;
    hipLaunchKernelGGL(free_kernel, dim3(gx < 64u ? gx : 64u, gy), dim3(kRowThreads), 0, stream, a);
    return done(hipGetLastError());
}

int xpress_kv_compact(const xpress_kv_cache* cache, const int32_t* start, const int32_t* path,
                      int64_t stride_path, const int32_t* count, int64_t longest, hipStream_t stream)
{
    if (!cache) return XPRESS_EINVAL;
    const xpress_kv_cache& c = *cache;
    size_t bytes = 0;
    if (!cache_ok(c, &bytes) || longest < 0 || longest > kMost) return XPRESS_EINVAL;
    if (c.seqs == 0 || longest == 0) return XPRESS_OK;
    if (!numbers_ok(start) || !numbers_ok(path) || !numbers_ok(count) || stride_path < 0 ||
        stride_path > ((int64_t)1 << 58) / c.seqs || (c.seqs > 1 && stride_path != 0 && stride_path < longest)) {
        return XPRESS_EINVAL;
    }
    const size_t np = (size_t)((c.seqs - 1) * stride_path + longest) * 4u, ns = (size_t)c.seqs * 4u;
    if (!apart_from_cache(c, bytes, start, ns) || !apart_from_cache(c, bytes, path, np) ||
        !apart_from_cache(c, bytes, count, ns) ||
        !apart_from_cache(c, bytes, c.page_table, table_bytes(c.seqs, c.table_width, c.stride_table))) {
        return XPRESS_EINVAL;
    }
    const int64_t e = element_bytes(c.dtype);
    const uint32_t w = piece_of(c);
    const int64_t pieces = c.dim * e / w;
    if (2 * c.heads * pieces > kMost) return XPRESS_EINVAL;
    CompactArgs a = {(char*)c.k, (char*)c.v, c.page_table, start, path, count, c.stride_page * e,
                     c.stride_head * e, c.stride_token * e, c.stride_table, stride_path, (uint32_t)c.pages,
                     (uint32_t)c.page_size, (uint32_t)c.seqs, (uint32_t)c.table_width, (uint32_t)longest,
                     (uint32_t)c.heads, (uint32_t)pieces};
    const uint32_t items = 2 * a.heads * a.pieces, gx = (items + kRowThreads - 1) / kRowThreads;
    const dim3 grid(gx < 256u ? gx : 256u, a.N < 65535u ? a.N : 65535u), block(kRowThreads);
    if (w == 16) hipLaunchKernelGGL(compact_kernel<u32x4>, grid, block, 0, stream, a);
    else if (w == 8) hipLaunchKernelGGL(compact_kernel<uint64_t>, grid, block, 0, stream, a);
    else if (w == 4) hipLaunchKernelGGL(compact_kernel<uint32_t>, grid, block, 0, stream, a);
    else if (w == 2) hipLaunchKernelGGL(compact_kernel<uint16_t>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(compact_kernel<uint8_t>, grid, block, 0, stream, a);
    return done(hipGetLastError());
}

}  // extern "C"
