/*
 * xpress_argmax.h -- C ABI of the MI355X (gfx950) fused add + argmax readout.
 *
 * The operation (XPress kernels page, "fused_add_argmax_to_blk" and its stage
 * kernels "_xpress_add_argmax_partial_kernel" /
 * "_xpress_add_argmax_reduce_to_blk_kernel"): one Jacobi pass drafts B-1 slots
 * in each of N blocks; draft row r = n*(B-1) + b carries base logits and a
 * refiner bias over a vocabulary of V ids, and the readout writes
 *
 *     blk[n, 1 + b] = argmax_v  bf16( base[r, v] + bias[r, v] )
 *
 * without ever storing the [N*(B-1), V] sum.  Each sum is formed from the two
 * bf16 values and rounded once to bf16 (round-to-nearest, ties to even,
 * subnormals kept) before the comparison, as the stage-1 kernel does by
 * casting the sum back to the input dtype; values compare as reals (-0 equals
 * +0) and the lowest vocabulary id wins a tie (the first-maximum argmax of a
 * chunk followed by a strict ">" scan over chunks in ascending order).  Slot
 * 0 of every block (the verified anchor) is never written; the next pass
 * reads blk in place.  NaN inputs are outside the contract.
 *
 * Everything here is plain C: pointers, 64-bit sizes and a HIP stream.
 * No function keeps a reference to a caller buffer after it returns.
 */
#ifndef XPRESS_ARGMAX_H
#define XPRESS_ARGMAX_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point. */
#define XPRESS_OK 0
#define XPRESS_EINVAL 1   /* an argument describes no valid layout */
#define XPRESS_EHIP 2     /* a HIP call failed; see xpress_last_hip_error() */
#define XPRESS_ENOMEM 3   /* the library could not allocate its workspace */
#define XPRESS_ECAPTURE 4 /* the workspace would have to grow while the stream
                             is being captured into a graph; call
                             xpress_reserve() before capturing */
#define XPRESS_ESCRATCH 5 /* the call needs more than the fixed key table of
                             xpress_add_argmax_to_blk_noalloc */

/*
 * xpress_add_argmax_to_blk -- the fused readout (page and passages above).
 *
 *   base           device pointer to bf16 bit patterns, N*(B-1) rows; row r
 *                  starts at base + r*stride_base_r and holds V elements with
 *                  unit stride.  Read only.
 *   bias           device pointer, the refiner bias, laid out like base with
 *                  its own row stride.  Read only; may alias base.
 *   blk            device pointer to int64 [N, B], row-major and contiguous.
 *                  blk[n*B + 1 + b] receives the winning vocabulary id of row
 *                  n*(B-1) + b; blk[n*B] and all other memory are untouched.
 *                  Must not overlap base or bias.
 *   N              blocks, >= 0.
 *   B              slots per block (anchor + B-1 drafts), >= 1.
 *   V              vocabulary size, 1 <= V <= 2^31 - 1.
 *   stride_base_r  row stride of base in elements, >= V.
 *   stride_bias_r  row stride of bias in elements, >= V.
 *   stream         HIP stream the work is queued on (0 = the null stream).
 *
 * Asynchronous: returns once the kernels are queued; blk is valid after the
 * stream reaches that point.  N == 0 or B == 1 (no draft rows) returns
 * XPRESS_OK and queues nothing.  Any layout is accepted; rows whose starts
 * and strides are 16-byte aligned take the vector path, others a scalar path
 * with identical results.
 *
 * Errors: XPRESS_EINVAL for a negative N, B < 1, V out of range, a stride
 * below V, a null pointer when there are rows, or blk overlapping an input
 * (nothing is queued); XPRESS_ENOMEM / XPRESS_ECAPTURE when the workspace
 * cannot be provided; XPRESS_EHIP when a launch fails.  Faults inside the
 * kernels (e.g. a pointer to too small a buffer) surface at the caller's
 * next synchronisation, as for any HIP kernel.
 *
 * Workspace: when the chosen plan splits a row over several workgroups the
 * library uses a small device workspace of its own (8 bytes per row, or per
 * row and split for the two-pass plan),
 * one per (device, stream), allocated on first use and left zeroed by every
 * call, so repeated calls and graph replays need no clearing.  Calls queued
 * on different streams use different workspaces and may run concurrently.
 * When a later call needs more, the workspace grows (synchronously, outside
 * capture only) into a new allocation and the old one is retired, not freed:
 * queued work and HIP graphs captured before keep valid memory until
 * xpress_release.  A graph holds the workspace of the stream it was captured
 * on: its replays must not run at the same time as other graphs captured there
 * or calls queued there.  The same rules hold for every entry point below that
 * uses the workspace.
 * The caller keeps every buffer alive until the queued work has finished.
 * Host threads: the library's own tables are locked, but a call holds its
 * stream's workspace from lookup to launch, so calls that queue on one
 * stream come from one host thread at a time, and xpress_release runs while
 * no other call of the library is in progress on any thread.
 */
int xpress_add_argmax_to_blk(const uint16_t* base, const uint16_t* bias,
                             int64_t* blk, int64_t N, int64_t B, int64_t V,
                             int64_t stride_base_r, int64_t stride_bias_r,
                             hipStream_t stream);

/*
 * xpress_add_argmax_to_blk_noalloc -- the same readout as
 * xpress_add_argmax_to_blk (same arguments, layout rules, result and errors)
 * for callers that cannot allocate device memory: code being captured into a
 * HIP graph without a prior xpress_reserve, tight serving loops, harnesses
 * that forbid allocation.  It never calls hipMalloc, hipFree or any other
 * allocating routine.  Rows that the plan splits over several workgroups
 * meet in two passes through a fixed key table of 4096 keys, a device array
 * built into the library (one copy per GPU, 32 KiB, held until the process
 * ends); the table holds rows x splits keys, which the automatic plan keeps
 * below 700, and a call that would need more (e.g. a split count forced with
 * xpress_set_plan) returns XPRESS_ESCRATCH and queues nothing.  Atomic and
 * balanced plans set with xpress_set_plan run as two-pass here.  Every call
 * on one GPU shares that table and overwrites it whole: calls that may run
 * at the same time on one GPU (e.g. queued on different streams) race and
 * must not overlap.  Asynchronous, like xpress_add_argmax_to_blk.  The
 * first call on a device (or xpress_reserve there) looks the table's device
 * address up with hipGetSymbolAddress; make one of them outside graph
 * capture before capturing this call.
 */
int xpress_add_argmax_to_blk_noalloc(const uint16_t* base, const uint16_t* bias,
                                     int64_t* blk, int64_t N, int64_t B, int64_t V,
                                     int64_t stride_base_r, int64_t stride_bias_r,
                                     hipStream_t stream);

/*
 * xpress_topc_argmax_to_blk -- the top-C readout (XPress kernels page,
 * "_xpress_topc_argmax_to_blk_kernel" and "fused_topc_argmax_to_blk"): each
 * draft row r = n*(B-1) + j carries C candidates; the first candidate
 * maximising bf16(base_c[r, c] + bias_c[r, c]) -- same element and tie rule
 * as above -- wins, and its vocabulary id is written:
 *
 *     blk[n, 1 + j] = cand[r, first argmax_c bf16(base_c[r, c] + bias_c[r, c])]
 *
 *   base_c, bias_c  device pointers to bf16 bit patterns, [N, B-1, C]
 *                   contiguous (row r at r*C).  Read only.
 *   cand            device pointer to int64 ids, [N, B-1, C] contiguous.
 *                   Read only; the winner's id is copied as is.
 *   blk             device pointer to int64 [N, B]; slots 1..B-1 written,
 *                   slot 0 untouched.  Must not overlap any input.
 *   N, B            as above; C >= 1 candidates per row (<= 2^31 - 1).
 *   stream          HIP stream (0 = the null stream).
 *
 * Asynchronous; same no-op and error rules as xpress_add_argmax_to_blk.
 * With the automatic plan, lists of up to 256 candidates are read by one wave
 * per row that carries the ids along (no second round trip for the gather);
 * longer lists, or any plan set with xpress_set_plan, take the streaming
 * readout with V = C and row strides C and gather the id when writing blk.
 */
int xpress_topc_argmax_to_blk(const uint16_t* base_c, const uint16_t* bias_c,
                              const int64_t* cand, int64_t* blk, int64_t N,
                              int64_t B, int64_t C, hipStream_t stream);

/*
 * xpress_readout_gemm_argmax_to_blk -- the readout with the refiner bias
 * computed in place (XPress kernels page, module description: a pass forms
 * logits = base + x @ W2 with a readout matmul and then takes the argmax; the
 * fused add + argmax consumes the matmul's bf16 result as its bias).  Here
 * the matmul runs on the matrix cores inside the readout and neither the
 * bias nor the logits are ever written:
 *
 *     bias[r, v]    = bf16( sum_k x[r, k] * w[v, k] )   (fp32 accumulation,
 *                                                         rounded once)
 *     blk[n, 1 + b] = first argmax_v bf16( base[r, v] + bias[r, v] )
 *
 *   base           device pointer, bf16 [N*(B-1), V] with row stride
 *                  stride_base_r (elements, >= V, a multiple of 8).
 *   x              device pointer, bf16 [N*(B-1), R] row-major (the latent
 *                  rows the refiner produced for the draft slots).
 *   w              device pointer, bf16 [V, R] row-major (the readout
 *                  weight, one row per vocabulary id; W2 = w^T).
 *   blk            device pointer to int64 [N, B]; slots 1..B-1 written.
 *   N, B, V        as for xpress_add_argmax_to_blk.
 *   R              latent width: 64, 128 or 256.
 *   stream         HIP stream (0 = the null stream).
 *
 * base, x and w must be 16-byte aligned (XPRESS_EINVAL otherwise).  The fp32
 * accumulation order is the matrix cores'; where every partial sum of the
 * dot products is exact (e.g. inputs on a coarse dyadic grid) the result is
 * bit-identical to rounding the exact dot product.  Asynchronous; two
 * launches; uses the (device, stream) workspace (rows x ranges keys, at most
 * rows x 512 x 8 bytes), grown on first use.  xpress_reserve does not size
 * it: before capturing this call into a HIP graph, make one call with at
 * least as many rows on the same stream outside capture (a capture that
 * would have to grow it returns XPRESS_ECAPTURE and queues nothing).  Later
 * growth retires the old table rather than freeing it, so graphs captured
 * earlier stay valid until xpress_release.
 */
int xpress_readout_gemm_argmax_to_blk(const uint16_t* base, const uint16_t* x,
                                      const uint16_t* w, int64_t* blk, int64_t N,
                                      int64_t B, int64_t V, int64_t R,
                                      int64_t stride_base_r, hipStream_t stream);

/*
 * xpress_reserve -- pre-allocate the workspace the readout would use for
 * (N, B, V) on `stream`'s device and stream, so that a later call -- e.g.
 * one being captured into a HIP graph -- allocates nothing; it also looks
 * up the device address of xpress_add_argmax_to_blk_noalloc's table.
 * Synchronous.
 * Returns XPRESS_OK, XPRESS_EINVAL, XPRESS_ENOMEM or XPRESS_EHIP.
 */
int xpress_reserve(int64_t N, int64_t B, int64_t V, hipStream_t stream);

/*
 * xpress_latent_pass -- the latent stage of one Jacobi pass (XPress kernels
 * page, module description and "_xpress_latent_kernel"), which produces the
 * rows the readout matmul consumes.  For every block n and slot b:
 *
 *     prev[b]  = am1[n] for b = 0, blk[n, b-1] otherwise
 *     x[b, :]  = xh[n, b, :] + w1[prev[b], :] @ wlat^T          (fp32)
 *     u[b, r]  = sum_{j < B} mixl[b, j, r] * x[j, r]             (fp32)
 *     g        = bf16(u[b]) @ wg^T,   v = bf16(u[b]) @ wu^T      (fp32)
 *     m        = bf16( g * sigmoid(g) * v )                      (SwiGLU)
 *     lat_out[n, b-1, :] = bf16( u[b] + m @ wd^T ),   b = 1 .. B-1
 *
 * Slot 0 is the verified anchor: its x enters the mixer of the later slots,
 * but no latent is written for it.
 *
 *   blk      device pointer, int64 [N, B] row-major: the block's tokens; slot
 *            b reads blk[n, b-1] (blk[n, B-1] is never read).  Read only.
 *   am1      device pointer, int64 [N]: the token before each block's anchor.
 *   xh       device pointer, bf16 [N, B, R]: the pass-invariant hidden cache.
 *   w1       device pointer, bf16 [V, R]: token embedding, one row per id.
 *   wlat     device pointer, bf16 [R, R]: embedding-to-latent projection,
 *            out-major (row r holds the weights of output channel r).
 *   mixl     device pointer, bf16 [B, B, R]: the folded mixer (L * tril + I)
 *            per channel; every j < B is summed, so entries above the
 *            diagonal must be zero for a causal mixer.
 *   wg, wu   device pointers, bf16 [H, R]: SwiGLU gate and up, out-major.
 *   wd       device pointer, bf16 [R, H]: SwiGLU down, out-major.
 *   lat_out  device pointer, bf16 [N, B-1, R]: written whole.  Must not
 *            overlap any input.
 *   N        blocks, >= 0 (N * B <= 2^31 - 1).
 *   B        slots per block, 2 .. 32.
 *   R        latent rank, a multiple of 64 in [64, 1024].
 *   H        MLP hidden size, a multiple of 64 in [64, 8192].
 *   V        rows of w1, >= 1.
 *   stream   HIP stream (0 = the null stream).
 *
 * xh, w1, wlat, mixl, wg, wu and wd must be 16-byte aligned; blk and am1
 * 8-byte aligned.  A token id outside [0, V) reads as a zero embedding row (no
 * out-of-bounds read; the result for that slot is then meaningless).  The
 * fp32 accumulation order is the matrix cores'; results agree with the exact
 * definition up to fp32 rounding of the sums before each bf16 rounding.
 *
 * Asynchronous; three launches on `stream`.  N == 0 queues nothing.  Uses the
 * (device, stream) workspace for u, bf16(u) and m (rows * (6R + 2H) bytes,
 * rows = N * (B-1)); grow it beforehand with xpress_latent_reserve when the
 * call will be captured into a HIP graph (growth retires the old regions
 * rather than freeing them, as for the readouts).  Errors: XPRESS_EINVAL (sizes,
 * alignment, null pointers, overlap; nothing queued), XPRESS_ENOMEM /
 * XPRESS_ECAPTURE (workspace), XPRESS_EHIP (launch).
 */
int xpress_latent_pass(const int64_t* blk, const int64_t* am1, const uint16_t* xh,
                       const uint16_t* w1, const uint16_t* wlat, const uint16_t* mixl,
                       const uint16_t* wg, const uint16_t* wu, const uint16_t* wd,
                       uint16_t* lat_out, int64_t N, int64_t B, int64_t R, int64_t H,
                       int64_t V, hipStream_t stream);

/*
 * xpress_latent_reserve -- grow the (device, stream) workspace to what
 * xpress_latent_pass needs for (N, B, R, H), so that a captured call
 * allocates nothing.  Synchronous.  Returns XPRESS_OK, XPRESS_EINVAL,
 * XPRESS_ENOMEM or XPRESS_EHIP.  Growing the workspace later (a larger shape
 * on the same stream) retires the old regions, which graphs captured before
 * keep using until xpress_release.
 */
int xpress_latent_reserve(int64_t N, int64_t B, int64_t R, int64_t H, hipStream_t stream);

/*
 * xpress_latent_set_tiles -- workgroup shape override for the three latent
 * kernels, for tests and tuning.  Each workgroup computes 32 * slabs rows of
 * a 32-column tile with its four waves; slabs = 4 gives every wave its own
 * 32-row slab over the whole contraction, slabs = 2 or 1 split the
 * contraction over 2 or 4 waves and sum the partials in LDS; 8 selects the
 * LDS-staged kernels (128 rows per workgroup, operands copied to LDS in
 * coalesced 64-wide contraction chunks, up to four in flight).  Arguments are the
 * choices for the mix, gate and down kernels: 1, 2, 4 or 8, or 0 for the
 * library's choice per shape (staged from 2048 rows on, else the most slabs
 * that still give each compute unit a workgroup).  Results are identical up
 * to fp32 summation order.
 * Process-wide; returns XPRESS_OK or XPRESS_EINVAL.
 */
int xpress_latent_set_tiles(int mix, int gate, int down);

/*
 * ---------------------------------------------------------------------------
 * Serving operators: a paged key-value cache, the append that fills it, the
 * attention that reads it, and the sampled readout.
 * ---------------------------------------------------------------------------
 */

/* Element types. */
#define XPRESS_BF16 0
#define XPRESS_FP16 1
#define XPRESS_E4M3 2 /* OCP 8-bit float, 4 exponent and 3 fraction bits; caches only */

/*
 * xpress_kv_cache -- a paged cache of keys and values and the page table of
 * the sequences that live in it.  Token j of sequence n is on page
 * page_table[n * stride_table + j / page_size], at place j % page_size;
 * element (page, head, place, d) is at
 *     page * stride_page + head * stride_head + place * stride_token + d
 * in k and in v (elements; both caches share the strides).
 *
 *   k, v          device pointers.
 *   k_scale,      device pointers, fp32 [heads], or null (1).  Only for
 *   v_scale       XPRESS_E4M3: a stored code stands for code * scale[head].
 *   page_table    device pointer, int32 [seqs, table_width].
 *   pages         pages in the pool, >= 1; page ids outside [0, pages) name no page.
 *   page_size     tokens of a page, >= 1 (any value; tiles may span pages).
 *   heads         key-value heads, >= 1.
 *   dim           elements of a head, >= 1.
 *   stride_*      elements, >= 1; no two elements may share an address.
 *   dtype         XPRESS_BF16, XPRESS_FP16 or XPRESS_E4M3.
 *   seqs          rows of page_table, >= 0.
 *   table_width   columns of page_table, >= 1 (table_width * page_size <= 2^31 - 1).
 *   stride_table  row stride of page_table in elements, >= table_width
 *                 (0 is allowed with one row).
 */
typedef struct xpress_kv_cache {
    void* k;
    void* v;
    const float* k_scale;
    const float* v_scale;
    const int32_t* page_table;
    int64_t pages, page_size, heads, dim;
    int64_t stride_page, stride_head, stride_token;
    int64_t dtype;
    int64_t seqs, table_width, stride_table;
} xpress_kv_cache;

/*
 * xpress_kv_append -- append the keys and values of T new tokens to a paged
 * cache, with the position rotation applied on the way, and rotate the
 * tokens' queries.  For token t of sequence n at position p, with c_i =
 * cos_sin[p, i] and s_i = cos_sin[p, rot_dim/2 + i], i < rot_dim/2:
 *
 *     rot(x)[a_i] = x[a_i] c_i - x[b_i] s_i
 *     rot(x)[b_i] = x[b_i] c_i + x[a_i] s_i        rot(x)[d] = x[d], d >= rot_dim
 *     q_out[t, h]             = round(rot(q[t, h]))
 *     K(page_table, n, p)[h]  = round(rot(k[t, h]) / k_scale[h])
 *     V(page_table, n, p)[h]  = round(v[t, h] / v_scale[h])
 *
 * where (a_i, b_i) = (i, i + rot_dim/2), or (2i, 2i + 1) when interleaved.
 * The two products and their sum are formed in fp32, each rounded, and the
 * result is rounded once to the stored type (ties to even); XPRESS_E4M3
 * saturates at +-448 and keeps NaN.
 *
 *   q, k, v      device pointers, [T, Hq or heads, dim] of `dtype` (BF16 or
 *                FP16) with token and head strides in elements (any, 0
 *                included) and unit stride along dim: slices of one
 *                projection's rows do.  q and q_out are ignored when Hq is 0.
 *   q_out        device pointer, written whole.  May be q itself with q's
 *                strides; must not share elements with k or v.
 *   positions    device pointer, int32 [T].
 *   seq_of       device pointer, int32 [T], the tokens' sequences; or null:
 *                T is a multiple of cache.seqs and token t belongs to sequence
 *                t / (T / seqs).
 *   cos_sin      device pointer, fp32 [max_pos, rot_dim] contiguous; unused
 *                when rot_dim is 0.
 *   rot_dim      even, 0 <= rot_dim <= dim.
 *
 * A token whose sequence or position is out of range (negative, or past
 * cache.seqs, table_width * page_size, or max_pos) is padding: nothing is
 * stored and its q_out rows are 0.  A token whose page id is outside the
 * pool is rotated but not stored.  Tokens of one call must not share a place:
 * their heads and 16-byte pieces are stored in no order, so each element there
 * would come from one of them, and K and V not necessarily from the same one.
 * cache.dtype is `dtype` or XPRESS_E4M3.
 *
 * Asynchronous; one launch; no workspace.  T == 0 queues nothing.  Any
 * alignment that suits the element types is accepted; accesses are of 8
 * elements where dim, the strides and the pointers allow it and rot_dim is a
 * multiple of 16, of 4 at half of that, else single, with identical results.
 * XPRESS_EINVAL: a size or type outside the above, a null pointer, a pointer not
 * aligned to its element, a cache or q_out whose elements share addresses, or a
 * cache whose span overlaps q, k, v, q_out or an index array.
 */
typedef struct xpress_kv_append_args {
    xpress_kv_cache cache;
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    const int32_t* positions;
    const int32_t* seq_of;
    const float* cos_sin;
    int64_t T, Hq, dtype;
    int64_t rot_dim, max_pos, interleaved;
    int64_t stride_q_t, stride_q_h, stride_k_t, stride_k_h;
    int64_t stride_v_t, stride_v_h, stride_o_t, stride_o_h;
} xpress_kv_append_args;

int xpress_kv_append(const xpress_kv_append_args* args, hipStream_t stream);

/*
 * xpress_kv_append_at -- the same for tokens whose place in the sequence is not
 * their position: the nodes of a tree of drafts, which stand one after the other
 * in the cache while siblings share a position.  places, a device pointer to
 * int32 [T], says where keys and values go: K(page_table, n, places[t]); the
 * rotation takes args->positions, which only max_pos bounds.  A token is padding if
 * its sequence or position is out of range; one whose place is out of range
 * (negative, or past table_width * page_size), or on a page outside the pool, is
 * rotated but not stored.  places null: xpress_kv_append.
 */
int xpress_kv_append_at(const xpress_kv_append_args* args, const int32_t* places, hipStream_t stream);

/*
 * xpress_paged_attention -- attention of the Q newest tokens of every
 * sequence over its paged cache (Q = 1: decoding; Q = B: verifying a drafted
 * block).  With len = lens[n] (the new tokens included, already appended),
 * query i of sequence n stands at position pos = len - Q + i and sees the
 * keys 0 <= j <= pos, j > pos - window when window > 0; query head h reads
 * key-value head h / (Hq / heads):
 *
 *     out[n, i, h] = sum_j softmax_j(scale * q[n, i, h] . K_j) V_j
 *     lse[n, i, h] = log sum_j exp(scale * q[n, i, h] . K_j)
 *
 * A query that sees no key (pos < 0, or every page missing) gives out = 0,
 * lse = -inf.  Keys on pages whose id is outside the pool take no part, and
 * neither they nor cache places that no query sees influence the result,
 * whatever they hold.
 *
 *   q, out       device pointers, [N, Q, Hq, dim] of `dtype` (BF16 or FP16),
 *                strides in elements, unit stride along dim.  N = cache.seqs.
 *   lse          device pointer, fp32 [N, Q, Hq] contiguous, or null.
 *   lens         device pointer, int32 [N]; values are clamped to
 *                [0, max_len].
 *   max_len      1 <= max_len <= table_width * page_size: an upper bound on
 *                lens that the split over the length is planned for.
 *   scale        fp32 factor of the scores; log2(e) times it is finite.
 *   dim          a multiple of 8 (of 16 with an XPRESS_E4M3 cache), at most
 *                256; cache.dtype is `dtype` or XPRESS_E4M3; the cache rows
 *                must start on 16-byte boundaries.
 *
 * Scores, softmax statistics and sums are fp32.  Asynchronous; one launch (one
 * for each 2^22 workgroups), or two when the length is split (partial results meet in the (device,
 * stream) workspace, in at most 1 GiB of it up to max_len 2^30;
 * xpress_paged_attention_reserve grows it before a capture).  The result does not depend on the order in which workgroups
 * run.  N == 0 or Q == 0 queues nothing.  Errors: XPRESS_EINVAL (sizes,
 * types, strides, null or misaligned pointers, out or lse overlapping an
 * input or the caches; nothing queued), XPRESS_ENOMEM / XPRESS_ECAPTURE
 * (workspace), XPRESS_EHIP (launch).
 */
typedef struct xpress_paged_attention_args {
    xpress_kv_cache cache;
    const void* q;
    void* out;
    float* lse;
    const int32_t* lens;
    int64_t Q, Hq, dtype, max_len, window;
    double scale;
    int64_t stride_q_n, stride_q_i, stride_q_h;
    int64_t stride_o_n, stride_o_i, stride_o_h;
} xpress_paged_attention_args;

int xpress_paged_attention(const xpress_paged_attention_args* args, hipStream_t stream);

/*
 * xpress_paged_attention_reserve -- grow the (device, stream) workspace to
 * what xpress_paged_attention needs for N sequences of up to max_len tokens,
 * Q new ones each, and these heads, head size and window.  Synchronous.
 * Returns XPRESS_OK, XPRESS_EINVAL, XPRESS_ENOMEM or XPRESS_EHIP.
 */
int xpress_paged_attention_reserve(int64_t N, int64_t Q, int64_t Hq, int64_t heads, int64_t dim,
                                   int64_t max_len, int64_t window, hipStream_t stream);

/*
 * xpress_paged_attention_plan -- the launch that such a call would make:
 * *chunk, the keys of one part of the split, *splits, the parts of the
 * longest sequence, *rows, the (query, head) rows a workgroup holds, and
 * *launches.  Any output may be null.  Pure host computation.  Returns
 * XPRESS_OK or XPRESS_EINVAL.
 */
int xpress_paged_attention_plan(int64_t N, int64_t Q, int64_t Hq, int64_t heads, int64_t dim,
                                int64_t max_len, int64_t window, int* chunk, int* splits,
                                int* rows, int* launches);

/*
 * xpress_sink_attention -- the same, where a window leaves the first tokens
 * visible: a query at position pos sees the keys 0 <= j <= pos with
 *
 *     j > pos - window   or   j < sinks              (all of them if window is 0)
 *
 * 0 <= sinks < 2^31.  What lies between is not read: pages there may have been
 * given back.  All else as for xpress_paged_attention; the workspace is what
 * xpress_sparse_attention_reserve with tree 0 grows it to.
 */
int xpress_sink_attention(const xpress_paged_attention_args* args, int64_t sinks, hipStream_t stream);

/*
 * xpress_tree_attention -- the same for a tree of drafted tokens: the Q newest
 * tokens of a sequence are nodes, node i at place past + i, past = len - Q.
 * Node i sees
 *
 *     the places j < past with j > pos - window or j < sinks (all if window is 0),
 *         where pos = past + (the number of nodes it sees) - 1, its position;
 *     node j, at place past + j, where bit j % 32 of tree[n, i, j / 32] is set
 *         (itself only if its own bit is; the window does not apply).
 *
 * Any mask is accepted, not ancestors alone: a node that sees no key gives out = 0,
 * lse = -inf.  There is no key at a negative place (len < Q), whatever names it; the row
 * of a query whose own place is negative is computed like any other, from the nodes
 * that its bits name and that there are (its bits 0: out = 0, lse = -inf).
 *
 *   tree     device pointer, int32 words [N, Q, ceil(Q / 32)], strides in words
 *            (not negative, 0 for one tree of all sequences), unit stride along the
 *            words; bits past Q are not looked at.
 *
 * A key that its window's and its tree's rule leave to no node takes no part,
 * whatever it holds.  All else as for xpress_paged_attention; the workspace is what
 * xpress_sparse_attention_reserve with tree 1 grows it to.
 */
int xpress_tree_attention(const xpress_paged_attention_args* args, const int32_t* tree,
                          int64_t stride_tree_n, int64_t stride_tree_i, int64_t sinks,
                          hipStream_t stream);

/*
 * xpress_sparse_attention_reserve -- grow the (device, stream) workspace to what
 * xpress_sink_attention (tree 0) or xpress_tree_attention (tree not 0) needs.
 * Synchronous.  Returns XPRESS_OK, XPRESS_EINVAL, XPRESS_ENOMEM or XPRESS_EHIP.
 */
int xpress_sparse_attention_reserve(int64_t N, int64_t Q, int64_t Hq, int64_t heads, int64_t dim,
                                    int64_t max_len, int64_t window, int64_t sinks, int tree,
                                    hipStream_t stream);

/*
 * The pages of a cache.  refs, int32 [pages] on the device, holds for each page how
 * many entries of all tables name it; a page with refs 0 is free.  Free pages are
 * taken lowest id first, in the order of the tables' rows (and of slots within a
 * row), so that results do not depend on the order of the work.  Entries outside
 * [0, pages) name no page.  Tables are int32 [rows, width] with a row stride of at
 * least width (any with one row) and unit stride along width; width * page_size < 2^31.
 * Where pages run out, the entries that lack one name none (-1 in a fork; what they were
 * in xpress_kv_grow) and *missing (int32 on the device, or null) receives their number;
 * it is written by every call.  All
 * functions are asynchronous and use no workspace.  XPRESS_EINVAL: a size or
 * stride outside what is said here, a null or misaligned pointer, or an array that is
 * written whose span, from its first byte to its last with the gaps between rows, meets
 * another's; nothing is queued.
 *
 * xpress_kv_fork -- M new rows of a table from N old ones.  Row m continues source
 * n = src[m] (outside [0, N): an empty row, all -1) with its lens[n] tokens, clamped to
 * [0, width * page_size]:
 *
 *     new_table[m, s] = table[n, s]    for whole pages, s < lens[n] / page_size;
 *     a part-filled last page stays with the lowest m of its source if no other
 *         entry names it (refs 1); the others, which will write to it, get a free page
 *         each, and copies[m] = (old page, new page, tokens) says what to copy there;
 *     -1 after that.
 *
 * copies [M, 3] is (-1, -1, 0) where nothing is to be copied.  new_refs [pages] are
 * the counts with the new table in place of the old one: refs - (entries of table that
 * name the page) + (entries of new_table).  refs, table and the pages themselves are
 * left as they are, and pages are taken from those free in refs: a fork may be made
 * again, as by a graph that is replayed.  Sources that no row continues give
 * their pages back.  Two launches.  N and M are 65536 at most.
 */
int xpress_kv_fork(const int32_t* refs, int64_t pages, const int32_t* table, int64_t stride_table,
                   const int32_t* lens, int64_t N, const int32_t* src, int64_t M, int64_t width,
                   int64_t page_size, int32_t* new_refs, int32_t* new_table, int64_t stride_new,
                   int32_t* copies, int32_t* missing, hipStream_t stream);

/*
 * xpress_kv_copy -- for each of copies [count, 3] = (from, to, tokens): the first
 * `tokens` places (clamped to [0, page_size]) of page `from` are copied to page `to`,
 * keys and values of all heads.  Entries with a page outside the pool do nothing.  A
 * page that is written must be in one entry of a call only.  cache->page_table, seqs
 * and the table's sizes are not looked at.  A page has fewer than 2^31 pieces (16
 * bytes, or what alignment leaves).
 */
int xpress_kv_copy(const xpress_kv_cache* cache, const int32_t* copies, int64_t count, hipStream_t stream);

/*
 * xpress_kv_grow -- free pages for the tokens have[n] <= p < want[n] of each sequence:
 * every slot s with ceil(have / page_size) <= s < ceil(want / page_size), s < width,
 * whose entry names no page gets one, with refs 1.  One launch of one workgroup; for
 * N > 0 width < 2^21.
 */
int xpress_kv_grow(int32_t* refs, int64_t pages, int32_t* table, int64_t stride_table, int64_t N,
                   int64_t width, int64_t page_size, const int32_t* have, const int32_t* want,
                   int32_t* missing, hipStream_t stream);

/*
 * xpress_kv_free -- gives back the pages of which no coming query sees a token: of
 * sequence n's entries those stay whose slot s has s * page_size < lens[n] and, with
 * window > 0, s * page_size < sinks or (s + 1) * page_size > lens[n] - window + 1
 * (what the token at position lens[n] will see; a node of a tree that sees no node, not
 * itself either, would see one place more).  Every other entry becomes -1, and
 * the count of the page it named goes down by one.  A finished sequence has lens 0;
 * rejected drafts are behind lens.
 */
int xpress_kv_free(int32_t* refs, int64_t pages, int32_t* table, int64_t stride_table, int64_t N,
                   int64_t width, int64_t page_size, const int32_t* lens, int64_t window, int64_t sinks,
                   hipStream_t stream);

/*
 * xpress_kv_compact -- the tokens of a path through a tree of drafts move together:
 * for j = 0, 1, .. below count[n] (clamped to [0, longest]) the key and value at place
 * start[n] + path[n, j] go to place start[n] + j of sequence n.  A path ascends from
 * 0 or more; it ends at the first entry that does not pass the one before.  A move
 * from or to a place past the table, or on a page outside the pool, is left out; a
 * negative start moves nothing.  Pages that other rows name too are written all the
 * same.  path int32 [seqs, longest], row stride stride_path (0: one path for
 * all), start and count int32 [seqs].
 */
int xpress_kv_compact(const xpress_kv_cache* cache, const int32_t* start, const int32_t* path,
                      int64_t stride_path, const int32_t* count, int64_t longest, hipStream_t stream);

/*
 * xpress_beam_select -- beam search's selection.  Row r = n * beams + i holds the
 * logits of beam i of sequence n, and
 *
 *     z_v = bf16(base[r, v] + bias[r, v])         (base[r, v] when bias is null)
 *     score(r, v) = scores[r] + z_v - log sum_w exp(z_w)
 *
 * best, rows and ids [N, K] receive the K candidates of each sequence with the
 * largest score, in descending order: the score, the row r and the id v.  Among equal
 * scores the lower row comes first, in a row the larger logit, then the lower id.
 * Scores are formed in 64 bits from sums of 32-bit terms (relative error of the sum
 * below 6e-7, usually 3e-8) and rounded once.
 *
 * NaN logits and -inf are no candidates and add nothing to the sum; a +inf logit
 * leaves only the +inf ones, with equal shares.  A beam whose score is not finite
 * takes no part (-inf: a beam that is not in use).  Where candidates run out: best
 * -inf, rows -1, ids -1, which xpress_kv_fork and xpress_beam_reorder take as empty.
 *
 *   base, bias     as for xpress_add_argmax_to_blk; bias may be null.
 *   scores         device pointer, fp32 [N * beams].
 *   best           device pointer, fp32 [N, K] contiguous.
 *   rows           device pointer, int32 [N, K] contiguous.
 *   ids            device pointer, int64 [N, K] contiguous.
 *   beams          1 .. 4096, and as many as LDS holds the lists of; K 1 .. 128.
 *
 * Asynchronous; two launches (one more of each for every 2^22 workgroups), whose lists
 * meet in the (device, stream) workspace; xpress_beam_select_reserve grows it before
 * a capture.  N == 0 queues nothing.  Errors as for xpress_add_argmax_to_blk
 * (stride_bias_r is not looked at without bias).
 */
int xpress_beam_select(const uint16_t* base, const uint16_t* bias, const float* scores, float* best,
                       int32_t* rows, int64_t* ids, int64_t N, int64_t beams, int64_t V, int64_t K,
                       int64_t stride_base_r, int64_t stride_bias_r, hipStream_t stream);

/*
 * xpress_beam_select_reserve -- grow the (device, stream) workspace to what
 * xpress_beam_select needs.  Synchronous.  Returns XPRESS_OK, XPRESS_EINVAL,
 * XPRESS_ENOMEM or XPRESS_EHIP.
 */
int xpress_beam_select_reserve(int64_t N, int64_t beams, int64_t V, int64_t K, hipStream_t stream);

/* One state of all beams: rows of `bytes` bytes, step_from and step_to bytes apart. */
typedef struct xpress_beam_state {
    const void* from;
    void* to;
    int64_t step_from, step_to, bytes;
} xpress_beam_state;

/*
 * xpress_beam_reorder -- every state's row src[m] of N goes to its row m of M; where
 * src[m] is outside [0, N), row m becomes zeros.  states is host memory, read during
 * the call; up to 4096 of them.  src is int32 [M] on the device.  The span that
 * is written of a state, from row 0's first byte to row M - 1's last with the gaps
 * between rows, must not meet that of anything which the call reads or writes
 * besides: XPRESS_EINVAL (states that lie between each other's rows are one state of
 * longer rows).
 * Asynchronous; one launch for every 8 states; accesses are of 16 bytes where rows and
 * steps allow it, else of 4 or 1.
 */
int xpress_beam_reorder(const xpress_beam_state* states, int64_t count, const int32_t* src, int64_t N,
                        int64_t M, hipStream_t stream);

/*
 * xpress_sample_to_blk -- the sampled readout: one token per draft row, drawn
 * with a given uniform number, written where the argmax readout would write
 * it.  For row r = n*(B-1) + b:
 *
 *     z_v = bf16(base[r, v] + bias[r, v])      (base[r, v] when bias is null)
 *
 * The ids are ordered by z (larger first; -0 equals +0; the lower id first
 * among equals), with weights w_v = exp((z_v - max z) / temperature[r]).
 * Three rules each keep a prefix of that order, and the shortest holds (at
 * least one id always):
 *
 *     top_k[r] > 0        the first top_k ids (mass Z; without it Z is the whole);
 *     top_p[r] < 1        ids before which less than top_p * Z has accumulated;
 *     min_p[r] > 0        ids with w_v >= min_p.
 *
 * With M the mass of the kept ids, blk[n, 1 + b] is the first id in the order
 * at which the accumulated mass exceeds u[r] * M, and prob[r] = w / M, its
 * probability.  temperature[r] not above 0 (NaN included) takes the largest z,
 * probability 1.  The masses are sums of counts times weights in 64 bits, so
 * the draw does not depend on the order of the work.
 *
 * NaN logits and -inf are never drawn; a row with nothing else gives id 0,
 * prob 0.  A +inf logit leaves only the +inf ones.  u is clamped to
 * [0, 1 - 2^-24] (NaN: 0); a NaN top_p or min_p is as if not given.
 *
 *   base, bias     as for xpress_add_argmax_to_blk; bias may be null.
 *   blk            device pointer to int64 [N, B]; slots 1..B-1 written.
 *   prob           device pointer, fp32 [N*(B-1)], or null.
 *   temperature,   device pointers, fp32 [N*(B-1)].
 *   top_p, min_p,
 *   u
 *   top_k          device pointer, int32 [N*(B-1)].
 *   N, B, V, strides, stream   as for xpress_add_argmax_to_blk.
 *
 * Asynchronous.  With a bias, up to 32 rows of 98304 to about 2 million logits
 * are counted in parts by several workgroups each, in two launches, whose lists
 * meet in the (device, stream) workspace (xpress_sample_reserve grows it before
 * a capture); where the memory cannot be had, and else, one launch (one for each
 * 2^21 rows) and no workspace, with the same results.  Errors as for xpress_add_argmax_to_blk, but
 * for XPRESS_ENOMEM and XPRESS_ECAPTURE, which are not returned (stride_bias_r is
 * not looked at without bias).
 */
int xpress_sample_to_blk(const uint16_t* base, const uint16_t* bias, int64_t* blk, float* prob,
                         const float* temperature, const int32_t* top_k, const float* top_p,
                         const float* min_p, const float* u, int64_t N, int64_t B, int64_t V,
                         int64_t stride_base_r, int64_t stride_bias_r, hipStream_t stream);

/*
 * xpress_sample_reserve -- grow the (device, stream) workspace to what
 * xpress_sample_to_blk uses for N*(B-1) rows of V logits.  Synchronous.  Returns
 * XPRESS_OK, XPRESS_EINVAL, XPRESS_ENOMEM or XPRESS_EHIP.
 */
int xpress_sample_reserve(int64_t N, int64_t B, int64_t V, hipStream_t stream);

/*
 * xpress_release -- free every workspace the library holds on the current
 * device, live and retired (after synchronising that device).  Optional; for
 * tests and for callers that want the memory back.  No other call of the
 * library may be in progress meanwhile, and graphs captured before hold freed
 * workspace and must not be replayed; the next call allocates afresh.
 */
int xpress_release(void);

/*
 * xpress_set_workspace_limit -- cap, in bytes, on the workspace (live plus
 * retired) the library may hold per device; 0 (the default) means no cap.
 * A call whose workspace would have to grow past the cap returns
 * XPRESS_ENOMEM and queues nothing, exactly as when the device is out of
 * memory.  Process-wide.  Returns XPRESS_OK, or XPRESS_EINVAL for a negative
 * cap.
 */
int xpress_set_workspace_limit(int64_t bytes);

/*
 * xpress_workspace_bytes -- *live_and_retired = the bytes of workspace the
 * library holds on the current device.  Returns XPRESS_OK, XPRESS_EINVAL
 * (null pointer) or XPRESS_EHIP.
 */
int xpress_workspace_bytes(int64_t* live_and_retired);

/*
 * Plan override, for tests and tuning.  combine selects how a row's partial
 * results meet:
 *   XPRESS_COMBINE_AUTO    the library's measured choice per shape;
 *   XPRESS_COMBINE_SINGLE  one workgroup per row, no cross-workgroup step;
 *   XPRESS_COMBINE_ATOMIC  several workgroups per row; each folds its packed
 *                          (value, ~index) key into a per-row 64-bit word that
 *                          also counts arrivals, by compare-and-swap; the last
 *                          to arrive writes blk and clears the word (one
 *                          launch);
 *   XPRESS_COMBINE_TWO_PASS several workgroups per row write their packed key
 *                          to a [rows, splits] table, a second small kernel
 *                          reduces each row (two launches);
 *   XPRESS_COMBINE_BALANCED the rows' 16-byte vectors, in row-major order, are
 *                          cut into equal contiguous ranges, one per
 *                          workgroup, over a whole number of workgroups per
 *                          CU; rows shared by several ranges are folded as in
 *                          ATOMIC (one launch; needs the aligned layout and
 *                          V >= 8, else it falls back to SINGLE).
 * splits is the number of workgroups per row (0 = automatic; ignored by
 * SINGLE); for BALANCED it is the number of workgroups per CU.  block_threads
 * is the workgroup size (0 = automatic, else 64, 128, 256, 512 or 1024).  The
 * setting is process-wide and applies to later calls.  Returns XPRESS_EINVAL
 * for an unknown combine or block size.
 */
#define XPRESS_COMBINE_AUTO 0
#define XPRESS_COMBINE_SINGLE 1
#define XPRESS_COMBINE_ATOMIC 2
#define XPRESS_COMBINE_TWO_PASS 3
#define XPRESS_COMBINE_BALANCED 4
int xpress_set_plan(int combine, int splits, int block_threads);

/*
 * xpress_set_reverse_order -- a debug setting for checking that results do
 * not depend on the order in which workgroups run.  With reversed nonzero,
 * later launches of the streaming readout (every combine, and the top-C
 * readout when it takes that path) visit their (row, split) units, or their
 * balanced ranges, from last to first, and the readout with in-place bias
 * maps its workgroups to (vocabulary range, row block) pairs from last to
 * first within each XCD; the work each workgroup does is unchanged, only
 * which runs early and which late, so the combines see their keys arrive in
 * another order.  Every result must be bit-identical to the default order's.
 * Process-wide; 0 restores the default.  Always returns XPRESS_OK.
 */
int xpress_set_reverse_order(int reversed);

/*
 * xpress_describe_plan -- what a call with these sizes and alignments would
 * launch: *combine, *splits, *block_threads, *vector_path (1 = 16-byte loads)
 * and *launches.  Pure host computation.  Returns XPRESS_OK or XPRESS_EINVAL.
 */
int xpress_describe_plan(const uint16_t* base, const uint16_t* bias, int64_t N,
                         int64_t B, int64_t V, int64_t stride_base_r,
                         int64_t stride_bias_r, int* combine, int* splits,
                         int* block_threads, int* vector_path, int* launches);

/*
 * xpress_describe_gemm_plan -- the launch shape xpress_readout_gemm_argmax_to_blk
 * would use for (N, B, V): *waves per workgroup (1, 2 or 8; each wave holds
 * 64 draft rows), *ranges (the vocabulary is cut into this many contiguous
 * ranges of whole 32-id tiles, a multiple of 8), *row_wgs (workgroups per
 * range) and *tiles (ceil(V / 32)).  Any output may be null.  Pure host
 * computation on the current device's compute-unit count.  Returns
 * XPRESS_OK or XPRESS_EINVAL.
 */
int xpress_describe_gemm_plan(int64_t N, int64_t B, int64_t V, int* waves, int* ranges,
                              int* row_wgs, int* tiles);

/*
 * xpress_bf16_add_round_table -- the readout's element step alone, for
 * checking it against the definition over every input pair.  For each i in
 * [0, n_a) and each of the 65536 bf16 patterns b it writes
 * out[i*65536 + b] = bf16(a_vals[i] + b) with the same device code the
 * readout kernels use.  a_vals (n_a entries) and out (n_a*65536 entries) are
 * device pointers.  Asynchronous on stream.  Returns XPRESS_OK,
 * XPRESS_EINVAL (n_a < 0, null pointer) or XPRESS_EHIP.
 */
int xpress_bf16_add_round_table(const uint16_t* a_vals, int64_t n_a,
                                uint16_t* out, hipStream_t stream);

/*
 * xpress_read_probe -- a plain streaming read of the readout's two inputs,
 * with no arithmetic on them: the practical read ceiling against which the
 * readout's rate is reported.  Not part of the readout.  base and bias are
 * rows rows of V bf16 at row stride `stride` (elements; V and stride
 * multiples of 8, 16-byte aligned pointers).  mode XPRESS_READ_ROWS reads
 * every row's V elements with one 256-thread workgroup per row (the
 * readout's launch shape at a few hundred rows); XPRESS_READ_FLAT sweeps
 * every element from the first row's start to the last row's end (padding
 * between rows included) with two workgroups per compute unit in
 * grid-stride order.  sink is a device pointer to one uint32 that is written
 * only if the folded data happens to equal a fixed constant (it keeps the
 * loads live).  Asynchronous.  Returns XPRESS_OK, XPRESS_EINVAL or
 * XPRESS_EHIP.
 */
#define XPRESS_READ_ROWS 0
#define XPRESS_READ_FLAT 1
int xpress_read_probe(const uint16_t* base, const uint16_t* bias, int64_t rows, int64_t V,
                      int64_t stride, int mode, uint32_t* sink, hipStream_t stream);

/* The HIP error code of the last failing HIP call on this thread. */
int xpress_last_hip_error(void);

/* A static, human-readable description of a status code. */
const char* xpress_error_string(int status);

/* Library version, "major.minor.patch". */
const char* xpress_version(void);

#ifdef __cplusplus
}
#endif

#endif /* XPRESS_ARGMAX_H */
