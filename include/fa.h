/*
 * fa.h — C ABI of the GB300 (sm_103a) exact-attention forward library
 * (libfa.so).
 *
 * The operation is exact softmax attention computed tile by tile with the
 * online softmax, never writing the N×N score matrix to memory:
 *
 *   S = scale · Q Kᵀ,   causal: S[i, j] = -inf for j > i
 *   P = softmax(S) by rows
 *   O = P V,            LSE_i = ln Σ_j exp(S[i, j])
 *
 * Definition: "Mini FlashAttention", §1 "What attention is" (the three-line
 * math and the causal-mask sentence). Streaming form: "Mini FlashAttention",
 * §4 "The flash trick: online softmax" (running max, running sum, rescale of
 * the running output, O = acc / l after the last chunk); "How Did I Write My
 * First FlashAttention Kernel in CUDA?", the pseudo-algorithm steps 1-5 and the
 * surrogate running-output paragraph. Initialisation and final normalisation:
 * the grasp.study lesson on the complete forward pass, "1. Initialization" and
 * "3. Finalization".
 *
 * Plain C types only: device pointers are `const void*` / `void*`, the CUDA
 * stream is passed as `void*` (a cudaStream_t; NULL is the legacy default
 * stream).
 *
 * Every forward kernel allows programmatic dependent launch: a kernel that the
 * caller launches next on the same stream with programmatic stream
 * serialization may start before the forward kernel has finished, and must
 * call cudaGridDependencySynchronize (griddepcontrol.wait) before it reads O
 * or LSE. Launches without that attribute keep plain stream order.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. 0 is success; every error is negative. */
typedef enum fa_status {
    FA_OK = 0,
    FA_ERR_NULL_PTR = -1,             /* q, k, v or o is NULL */
    FA_ERR_BAD_SHAPE = -2,            /* B, H or N < 1, or a size past the limits below */
    FA_ERR_UNSUPPORTED_HEAD_DIM = -3, /* d is not 64 or 128 */
    FA_ERR_MISALIGNED = -4,           /* q, k, v, o not 16-byte aligned, or lse not 4-byte aligned */
    FA_ERR_NO_DEVICE = -5,            /* no CUDA device, or the current device cannot be queried */
    FA_ERR_UNSUPPORTED_ARCH = -6,     /* the current device is not compute capability 10.3 */
    FA_ERR_LAUNCH = -7,               /* tensor-map encoding or the kernel launch failed, or a call was
                                         captured into a CUDA graph before the device's first ordinary call */
    FA_ERR_DEVICE_TIMEOUT = -8,       /* a kernel gave up waiting on an mbarrier (see fa_device_status) */
    FA_ERR_BAD_SCALE = -9,            /* scale is not finite, or not > 0 */
    FA_ERR_ALIAS = -10,               /* o or lse overlaps q, k or v, or lse overlaps o */
    FA_ERR_WORKSPACE = -11,           /* workspace NULL or smaller than the call needs */
    FA_ERR_BAD_TYPE = -12             /* cache element type is not one of FA_CACHE_* */
} fa_status;

/*
 * fa_fwd — attention forward pass on the current CUDA device.
 *
 * q, k, v  device, bf16, contiguous [B, H, N, d] (row-major: d fastest).
 *          Read only.
 * o        device, bf16, contiguous [B, H, N, d]. Written: O = P V.
 * lse      device, fp32, contiguous [B, H, N], or NULL to skip it. Written:
 *          the natural-log log-sum-exp of each query row's scaled scores
 *          over the keys the row may see.
 * B, H, N  batch, heads, sequence length (queries = keys = N), each >= 1;
 *          B*H <= 2^31-1 and 2*B*H*ceil(N/256) <= 2^31-1 - 65536 (work
 *          items and one over-claim per CTA fit the int counter).
 * d        head dimension: 64 or 128.
 * scale    score scale (the pages use 1/sqrt(d)); finite and > 0.
 * causal   nonzero: key j is hidden from query i when j > i (top-left
 *          aligned; every row keeps at least its own key).
 * stream   cudaStream_t to run on, as void*; NULL = legacy default stream.
 *
 * Ownership: the caller allocates and owns every buffer; the library keeps
 * no pointer after the call returns and allocates no device memory, neither
 * per call nor once: its only device state is a fixed 32 KB array inside the
 * library (work-queue counters: 256 slots of 128 bytes) and the device status
 * word, which every GPU that loads the library holds until the process exits.
 * Per device it caches the SM count, the kernels' shared-memory attributes
 * and that array's device address, all set by the first ordinary call of any
 * forward entry point on that device (with the device current). Each launch
 * uses one of 64 counter slots in turn and leaves it zeroed, so up to 64
 * launches may be in flight at once on different streams. A non-causal
 * problem whose last wave of work units would leave most SMs idle runs those
 * units as half units (one 128-row query tile whose key tiles the CTA's two
 * softmax warpgroups share out, merged inside the CTA), and so does every
 * unit of a causal problem with at most half as many units as SMs: no
 * scratch memory.
 * The call is asynchronous: argument errors are returned before anything is
 * queued; faults inside the kernel appear at the caller's next
 * synchronisation, and a kernel that gave up on a wait leaves its O/LSE rows
 * unwritten and reports through fa_device_status(). The current device must
 * be compute capability 10.3 (sm_103a).
 *
 * CUDA graphs: fa_fwd, fa_fwd_varlen and fa_fwd_noalloc may be called while
 * `stream` is being captured (cudaStreamBeginCapture, torch.cuda.graph),
 * once the device has had one ordinary call of a forward entry point: that
 * call sets what a capture may not (the kernels' shared-memory sizes, the
 * counter array's address). A call captured before then returns
 * FA_ERR_LAUNCH and enqueues nothing. The tensor maps are encoded from the
 * pointers given at capture, so a replay reads and writes those buffers,
 * which must stay allocated while the graph may be replayed (a replay after
 * one was freed reads or writes unmapped or reused memory; torch.cuda.graph
 * returns the allocator's free blocks to the driver when a capture begins). A
 * captured call keeps the counter slot it drew for every replay, from 192
 * slots that ordinary calls never use, so replays may overlap ordinary
 * launches and replays of other graphs on other streams (until 192 calls have
 * been captured on the device, when the slots wrap). fa_fwd_noalloc's one
 * shared slot stays shared when captured.
 */
int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
           int B, int H, int N, int d, float scale, int causal, void* stream);

/*
 * fa_fwd_noalloc — the same attention forward pass as fa_fwd, for callers
 * that cannot let a library call allocate device memory: code running inside
 * an allocator or memory-pool callback, under a memory budget that must
 * account for every byte, or in a runtime that plans all device memory
 * before it starts. (The pages describe no such entry point; it is part of
 * this library's interface only.)
 *
 * Arguments, layouts, ownership, limits and errors are those of fa_fwd,
 * and it gives fa_fwd's results bit for bit. It never calls cudaMalloc,
 * cudaFree or any allocating routine (fa_fwd does not either; this entry
 * point states it as its contract and keeps its own counters): its scratch
 * (one 128-byte work-queue slot) is a fixed array inside the library that
 * every GPU which loads the library keeps until the process exits. The
 * first call on a device looks up that array's device address (with that
 * device current); make the first call before any stream capture. Each call
 * clears the slot's counters on `stream` before its kernel, and every call
 * shares the one slot: calls whose kernels overlap on the GPU (different
 * streams, no ordering between them) race on it and must not be issued. The
 * scratch does not grow with the problem.
 */
int fa_fwd_noalloc(const void* q, const void* k, const void* v, void* o, float* lse,
                   int B, int H, int N, int d, float scale, int causal, void* stream);

/*
 * fa_fwd_varlen — the same forward pass over a batch of B sequences of
 * different lengths, each with its own number of queries and keys ("Mini
 * FlashAttention", §4 "The flash trick: online softmax", checks the loop on
 * ragged sequences).
 *
 *   q, o   bf16 [total_q, H, d], token-major (a token's H heads side by side),
 *          device, contiguous, 16-byte aligned
 *   k, v   bf16 [total_k, H, d], likewise
 *   lse    fp32 [H, total_q], device, or NULL; natural-log log-sum-exp
 *   cu_seqlens_q, cu_seqlens_k
 *          int32 [B + 1], device: sequence b holds query tokens
 *          cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1 and key tokens
 *          cu_seqlens_k[b] .. cu_seqlens_k[b+1]-1. The caller guarantees
 *          cu[0] = 0, non-decreasing offsets, cu_seqlens_q[B] = total_q,
 *          cu_seqlens_k[B] = total_k and every query count <= max_seqlen_q;
 *          the library reads them only on the GPU. Offsets that break this
 *          give undefined values but no write outside o[0, total_q) and
 *          lse's rows (reads past total_k see zeros).
 *   max_seqlen_q
 *          the largest query count of the batch (it sizes the launch)
 *   causal non-zero: the mask is aligned at the end of each sequence, so
 *          query i (0-based within its sequence) sees keys j <= i + Nk - Nq;
 *          with Nq = Nk this is fa_fwd's mask, and a single query (decode)
 *          sees every key. A query that sees no key gets O = 0, LSE = -inf.
 *
 * Same return codes as fa_fwd (FA_ERR_BAD_SHAPE for negative totals,
 * max_seqlen_q > total_q, or B*H*ceil(max_seqlen_q/256) >= 2^31 - 65536; q/o
 * and k/v may be NULL when total_q, resp. total_k, is 0); a batch with no
 * query returns FA_OK at once.
 *
 * Work is split into units of (sequence, head, 256 queries). When there are
 * few units for the GPU's SMs (decode: a few sequences of one query against
 * long key sets), each unit's key tiles are shared out among the CTAs of a
 * thread-block cluster (2-8 of them; fa_varlen_num_splits gives how many).
 * Each CTA keeps its partial O, normalised, and its LSE in its own shared
 * memory, and the cluster's first CTA merges them through distributed
 * shared memory: O = sum_s 2^(L_s - L) O_s with L = log2 sum_s 2^L_s (base-2
 * LSEs), the online-softmax rescaling applied across the shares. No device
 * memory is allocated (fa_fwd's ownership rules apply).
 */
int fa_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                  const int* cu_seqlens_q, const int* cu_seqlens_k, int B, int H, int total_q,
                  int total_k, int max_seqlen_q, int d, float scale, int causal, void* stream);

/*
 * fa_varlen_num_splits — host-only, no device call: among how many CTAs
 * (a cluster) fa_fwd_varlen shares out each unit's key range for these sizes
 * on a GPU with `sm_count` SMs (1 = no split, at most 8). Returns
 * FA_ERR_BAD_SHAPE under the same shape rules as fa_fwd_varlen, or when
 * sm_count < 1.
 */
int fa_varlen_num_splits(int B, int H, int total_k, int max_seqlen_q, int sm_count);

/*
 * ---------------------------------------------------------------------------
 * Serving from a paged key-value cache.
 *
 * A step of a server: fa_page_maps gives the step's new tokens their pages,
 * slots and positions; fa_cache_append turns q and k by their rotary positions
 * and writes k and v to their slots; fa_decode_paged attends one new token per
 * request over its pages (prompts: fa_fwd_varlen on the rotated q, k and v).
 * fa_rotary is the rotary step alone, for training, with its gradient.
 * (The source pages have no counterpart to any of these.)
 *
 * All are asynchronous on `stream`, allocate nothing, keep no pointer and
 * check their arguments on the host before anything is queued, as fa_fwd does;
 * they may be captured into CUDA graphs once the device has had one ordinary
 * call of any of them (a captured call before then returns FA_ERR_LAUNCH).
 * They keep no state on the device either: calls on different streams and
 * replays of different graphs share nothing but the buffers given to them.
 * Their kernels allow programmatic dependent launch as fa_fwd's do, and are
 * themselves launched that way: they wait for what precedes them on the stream
 * before they read or write.
 * ---------------------------------------------------------------------------
 */

/* Element types of a cache. */
#define FA_CACHE_BF16 0
#define FA_CACHE_E4M3 1 /* 8-bit floats; a value is code * scale[head] */

/*
 * fa_paged_cache — one layer's keys and values in pages ("blocks") of
 * page_size tokens. Value x of head h of token t of block b is at
 * k[b*k_block + t*k_token + h*k_head + x] (strides in elements), so token-major
 * blocks [page_size, heads, d], head-major blocks [heads, page_size, d] and
 * keys and values side by side in one tensor are all covered.
 *
 * page_size is a power of two, 16 to 65536; d is 64 or 128, its values
 * contiguous. k and v are 16-byte aligned; strides are multiples of 16 bytes
 * and at least d (that of a dimension of size 1 is not used).
 * k_scale, v_scale: device fp32 [heads], or NULL for 1. They apply to caches
 * of either type when reading, and to FA_CACHE_E4M3 when writing.
 */
typedef struct fa_paged_cache {
    void* k;
    void* v;
    const float* k_scale;
    const float* v_scale;
    long long k_block, k_token, k_head;
    long long v_block, v_token, v_head;
    int type; /* FA_CACHE_BF16 or FA_CACHE_E4M3 */
    int num_blocks, page_size, heads, d;
} fa_paged_cache;

/*
 * fa_decode_paged — attention of one new token per request over its pages:
 *   O = softmax(scale · q Kᵀ) V over the first seq_lens[b] keys of request b,
 *   LSE = ln Σ exp of the scaled scores.
 *
 *   q, o         bf16 [B, Hq, d], device, contiguous, 16-byte aligned
 *   lse          fp32 [B, Hq], device, or NULL
 *   cache        see above; Hq is a multiple of cache->heads, and query head i
 *                reads key head i / (Hq / heads)
 *   block_table  int32 [B][table_stride], device; entry i < table_width of row b
 *                is the block of keys i*page_size .. of request b
 *   seq_lens     int32 [B], device: keys of each request, the new token's own
 *                among them (append it first). 0 or less: O = 0, LSE = -inf.
 *                More than table_width*page_size counts as that many
 *                (at most 2^31 - 65536).
 *   workspace    device, 16-byte aligned, at least fa_decode_paged_workspace()
 *                bytes (NULL if that is 0: a small batch needs none); needs no
 *                initial value, holds nothing after the call's kernels. Calls
 *                (or graph replays) that may overlap in time need workspaces
 *                of their own.
 *
 * Keys whose block is outside [0, num_blocks) are hidden, as if they were not
 * there; table entries past a request's last key are not read. Values in
 * hidden and unfilled places of a page (NaN included) have no effect. In visible
 * ones NaN is passed on, and an infinity of v gives an infinity (NaN where two of
 * opposite sign meet, or a weight is below fp32's range).
 * Weights and sums are fp32; over FA_CACHE_E4M3 a weight is off by 2^-44 of the row's
 * largest at most beside its own rounding, and values of q 2^-28 below their head's
 * largest lose bits (fp16's smallest step).
 * seq_lens, block_table and the cache must not change while the call runs (lengths
 * that do give wrong values, but no access outside the buffers given).
 * The result does not depend on what else runs; which partial sums are joined
 * depends on the batch, so the same request may differ in the last bits
 * between batches.
 */
int fa_decode_paged(const void* q, const fa_paged_cache* cache, const int* block_table, const int* seq_lens, void* o,
                    float* lse, int B, int Hq, int table_width, long long table_stride, float scale, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * fa_decode_paged_workspace — host-only: workspace bytes of fa_decode_paged
 * for these sizes on a GPU with sm_count SMs (0 to 21 MB on 152 SMs), or a negative
 * status under the call's own rules.
 */
long long fa_decode_paged_workspace(int B, int Hq, int Hkv, int d, int cache_type, int page_size, int table_width,
                                    int sm_count);

/*
 * fa_rotary — rotary positions of x [B, H, N, d] (bf16, device), into y.
 * Pair i < rotary_dim/2 of each head is turned by a = position · inv_freq[i]:
 *   (y1, y2) = factor · (x1 cos a - x2 sin a, x2 cos a + x1 sin a)
 * where the pair is values (i, i + rotary_dim/2), or (2i, 2i+1) when
 * `interleaved`; values from rotary_dim on are copied. `inverse` uses -a: the
 * transposed map, which is the gradient of y with respect to x.
 *
 *   positions   int32, device: that of (b, n) is positions[b*position_stride + n]
 *               (0: shared by the batch). Any int32 value.
 *   inv_freq    fp64 [rotary_dim/2], device, finite, in radians per position.
 *               The angle is off by |position|·2^-59 + 2^-30 radians at most
 *               (frequencies up to 1), its cos and sin by 2^-24 beside that.
 *   x_strides, y_strides  host arrays: elements from one b, h, n to the next
 *               (multiples of 8; x's may be 0; those of a dimension of size 1
 *               are not used); d's values are contiguous. y's rows do not
 *               overlap (each stride is past all that the smaller ones span); y
 *               may be x itself with the same strides, or overlap nothing of it.
 *   rotary_dim  a multiple of 16, 0 to d.  factor finite (1: a pure rotation).
 *   B*N at most 2^31 - 65536, H at most 32767.
 *
 * Sums and products are fp32, rounded to bf16 once.
 */
int fa_rotary(const void* x, void* y, const int* positions, const double* inv_freq, int B, int H, int N, int d,
              const long long* x_strides, const long long* y_strides, long long position_stride, int rotary_dim,
              int interleaved, int inverse, float factor, void* stream);

/*
 * fa_cache_append — one step's tokens: q and k turned as by fa_rotary, q into
 * q_out, k (and v as it is) into the cache at their slots.
 *
 *   q, q_out    bf16 [T, Hq, d]; k, v, k_out  bf16 [T, heads, d], device: a
 *               token's heads contiguous, tokens *_stride elements apart (a
 *               multiple of 8), so that slices of one projection's output can
 *               be given. k_out may be NULL. q_out may be q and k_out may be k,
 *               with the same stride; apart from that outputs overlap nothing.
 *   positions, slots  int32 [T], device. Slot s is token s % page_size of block
 *               s / page_size. A token whose slot is negative or past the cache
 *               is padding: nothing of it is written, in no output.
 *               The cache's rows do not overlap, as y's above, nor k's with v's
 *               (caches of one buffer with other strides each are taken if what
 *               their differing dimensions span lies apart).
 *               Slots of one call are distinct (of two tokens with the same
 *               slot, either's values are kept, in pieces of 8 or 16 values).
 *
 * FA_CACHE_E4M3: code = e4m3(x / scale[head]), the quotient of fp32 values
 * rounded to fp32 and that to nearest even, past ±448 to ±448, NaN kept.
 */
int fa_cache_append(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                    long long v_stride, const int* positions, const int* slots, const double* inv_freq,
                    const fa_paged_cache* cache, void* q_out, void* k_out, long long q_out_stride,
                    long long k_out_stride, int T, int Hq, int rotary_dim, int interleaved, float factor,
                    void* stream);

/*
 * fa_page_maps — block tables and slot maps of one step, from request lengths.
 * Request b < B (1 to 8192) holds context_lens[b] tokens and gets new_lens[b]
 * more (negative counts as 0). All arrays int32, device.
 *
 *   block_table   [B][table_stride], in and out: the entries of the pages that
 *                 the context holds are kept; those of pages that the new tokens
 *                 need beyond them are written, from unused_blocks in order,
 *                 request by request (-1 once it has run out). Others are kept.
 *   unused_blocks [num_unused], read only: the caller drops the first counts[0].
 *   cu_seqlens    [B + 1]: exclusive sums of the new lengths (fa_fwd_varlen's
 *                 cu_seqlens_q)
 *   seq_lens      [B]: context + new (fa_decode_paged's seq_lens)
 *   slots, positions  [T]: of token t, the (t - cu_seqlens[b])-th new one of its
 *                 request b; slot -1 where its page is missing (none left, past
 *                 table_width, or a negative entry). Tokens past the last
 *                 request's get slot -1, position 0 (a padded batch); tokens past
 *                 T are not written.
 *   counts        [4]: pages taken, pages missing, new tokens in all, requests
 *                 longer than table_width*page_size
 *
 * Sums past 2^31 - 1 stay there. The arrays written overlap no other.
 */
int fa_page_maps(const int* context_lens, const int* new_lens, int* block_table, const int* unused_blocks, int* slots,
                 int* positions, int* cu_seqlens, int* seq_lens, int* counts, int B, int table_width,
                 long long table_stride, int num_unused, int page_size, int T, void* stream);

/* Static English text for a return code (never NULL). */
const char* fa_strerror(int status);

/*
 * fa_device_status — synchronises `stream` (a cudaStream_t as void*, NULL =
 * legacy default), then reads and clears the current device's status word.
 * Returns FA_OK if no kernel gave up on a wait since the last call,
 * FA_ERR_DEVICE_TIMEOUT if one did (then *bits, if not NULL, receives the
 * word: which kind of wait gave up), or FA_ERR_NO_DEVICE / FA_ERR_LAUNCH if
 * the synchronisation or the read failed.
 */
int fa_device_status(void* stream, unsigned* bits);

/*
 * fa_set_wait_limit_ns — how long a kernel waits on one mbarrier phase before
 * giving up (default 2e9 ns). Applies to launches made after the call, on
 * every device. 0 restores the default.
 */
void fa_set_wait_limit_ns(unsigned long long ns);

/*
 * fa_selftest_wait_timeout — failure-detection self-test. Launches, on
 * `stream`, one warp that waits on an mbarrier phase nothing completes, using
 * the forward kernel's bounded wait with a limit of `limit_ns` (200 µs to 1 s,
 * else FA_ERR_BAD_SHAPE). The wait gives up, records "other wait" (bit 4) in
 * the device status word and the kernel returns; nothing faults or hangs, and
 * the context stays usable. fa_device_status() then reports
 * FA_ERR_DEVICE_TIMEOUT. Returns FA_OK once launched, FA_ERR_NO_DEVICE /
 * FA_ERR_UNSUPPORTED_ARCH / FA_ERR_LAUNCH otherwise. The pages have no
 * counterpart (they have no failure handling).
 */
int fa_selftest_wait_timeout(void* stream, unsigned long long limit_ns);

/*
 * fa_selftest_exp2 — numerics self-test of the exponential. For i < n, writes
 * y_approx[i] = 2^x[i] computed by the instruction the softmax uses
 * (ex2.approx.ftz.f32: subnormal arguments and results flush to zero, 2^-inf
 * = +0) and y_exp2f[i] = CUDA's exp2f(x[i]). x, y_approx, y_exp2f are device
 * fp32 arrays of n elements, 4-byte aligned, owned by the caller; the call is
 * asynchronous on `stream`. Returns FA_OK (also for n = 0), FA_ERR_BAD_SHAPE
 * for n < 0, FA_ERR_NULL_PTR / FA_ERR_MISALIGNED for bad pointers, else the
 * device and launch codes of fa_fwd. The pages have no counterpart (they call
 * exp / expf without stating its accuracy).
 */
int fa_selftest_exp2(const float* x, float* y_approx, float* y_exp2f, int n, void* stream);

/*
 * fa_selftest_ex2_rate — throughput probe of the exponential unit, the
 * softmax's second ceiling beside the tensor cores (one ex2 per query and
 * visible key). Launches `blocks` blocks of 1024 threads, one per SM (each
 * asks for 120 KB of shared memory); every thread runs 8 independent chains
 * of `iters` dependent ex2.approx.ftz.f32. cycles (device, int64 [blocks],
 * 8-byte aligned) receives each block's span in SM clocks; sink (device,
 * fp32 [blocks * 1024], 4-byte aligned) receives the chains' final values so
 * that no work is elided. The rate is 8192 * iters / cycles[b] ex2 per clock
 * of block b's SM. Asynchronous on `stream`. Returns FA_OK once launched,
 * FA_ERR_BAD_SHAPE unless 1 <= blocks <= 4096 and 1 <= iters <= 2^20,
 * FA_ERR_NULL_PTR / FA_ERR_MISALIGNED for bad pointers, else the device and
 * launch codes of fa_fwd. The pages have no counterpart.
 */
int fa_selftest_ex2_rate(long long* cycles, float* sink, int blocks, int iters, void* stream);

/* ABI version of this header (bumped on any incompatible change). */
int fa_abi_version(void);

#define FA_ABI_VERSION 1

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
