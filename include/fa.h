/*
 * fa.h -- C ABI of the B200 (sm_100a) exact IO-aware attention library.
 *
 * What the library computes is exact attention, O = softmax(scale * Q K^T) V,
 * tiled so that the N x N scores S and probabilities P live only in on-chip
 * memory (TMEM / shared memory) and are never written to HBM; the forward saves
 * one per-row statistic and the backward recomputes P tile by tile from it.
 * Sources: explainers.rudrite.com "flash-attention-anatomy" (Q&As "Why is
 * attention memory-bound, and how does FlashAttention fix it?", "What is online
 * softmax and how does tiling keep it exact?", "How does FlashAttention save
 * memory in the backward pass?", "What changed between FlashAttention 1, 2, and
 * 3?"); chipfoundryservices.com glossary "flash attention" ("Tiling plus an
 * online softmax removes the round trip"); kipu-akw.pages.dev "flash-attention /
 * where-it-matters" (section "The Real Complexity").
 *
 * Conventions shared by every entry point:
 *   - Layout: contiguous [B, H, N, d] row-major, d innermost, for every
 *     [.., N, d] tensor; LSE and other per-row values are contiguous [B, H, N].
 *   - Device pointers.  The caller owns every buffer (including the backward
 *     workspace); the library allocates no device or pinned memory, keeps no
 *     pointer after a call returns, and never synchronises the stream.
 *   - Tensor pointers (q, k, v, o, dO, dq, dk, dv, workspace) must be 16-byte
 *     aligned; lse must be 4-byte aligned.
 *   - d (head dimension) must be 64 or 128.  N >= 1 is arbitrary: ragged tails
 *     are masked.  B, H, N == 0 is a valid empty call that launches nothing.
 *   - causal != 0 selects top-left aligned causal masking (key j is visible to
 *     query i iff j <= i; Nq == Nk == N).  Fully masked tiles are skipped.
 *   - scale is the softmax scale (the configurations use 1/sqrt(d)).  It must
 *     be finite and >= 0; scale = 0 is valid and makes every visible key
 *     equally weighted (O is the mean of the visible V rows, LSE = ln of
 *     their count, dQ = dK = 0).  A negative or non-finite scale returns
 *     FA_ERR_INVALID_ARG.
 *   - stream is a cudaStream_t passed as an opaque pointer (NULL = legacy
 *     default stream).
 *   - Arguments are checked on the host before anything is launched; a bad
 *     argument returns an error code and launches nothing.  A launch failure
 *     returns FA_ERR_LAUNCH.  Asynchronous device faults surface at the
 *     caller's next synchronisation.  Every device-side wait is bounded; one
 *     that runs out records a status readable with fa_device_status().
 *   - Thread safety: calls are re-entrant; the first call on a device also
 *     configures the kernels' shared-memory limits for that device.
 *   - CUDA graphs: the attention calls (fa_fwd*, fa_bwd*, fa_fwd_decode*,
 *     fa_fwd_standard), fa_rope, fa_page_tables and fa_cache_append_fp8 only
 *     enqueue kernel launches on the stream, so a
 *     caller may capture them into a graph and replay it.  Make the first
 *     call on each device outside any capture (it looks up device attributes
 *     and symbol addresses once).  fa_bwd_events also records the caller's
 *     events, which time nothing inside a capture; fa_device_status
 *     synchronises and cannot be captured.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FA_API __attribute__((visibility("default")))
#else
#define FA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fa_status {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,     /* null pointer, bad size or dimension, bad scale */
  FA_ERR_UNSUPPORTED = 2,     /* head dimension other than 64 / 128 */
  FA_ERR_ALIGNMENT = 3,       /* pointer not 16-byte (4-byte for lse) aligned */
  FA_ERR_ARCH = 4,            /* current device is not sm_100 (B200 class) */
  FA_ERR_LAUNCH = 5,          /* CUDA runtime rejected a launch or attribute */
  FA_ERR_DEVICE_TIMEOUT = 6,  /* a bounded device wait ran out (fa_device_status) */
  FA_ERR_WORKSPACE = 7,       /* workspace missing or too small */
  FA_ERR_SCRATCH_LIMIT = 8,   /* shape needs more than fa_bwd_noalloc's fixed scratch */
  FA_ERR_BAD_PAGE = 9         /* a kernel met a page or slot outside the cache and skipped it (fa_device_status) */
} fa_status;

/*
 * Forward pass, bf16.
 * Computes O = softmax(scale * Q K^T) V per (batch, head) with a running row
 * maximum m and denominator l carried across key tiles and the partial output
 * rescaled by exp(m_old - m_new) when m grows ("What is online softmax and how
 * does tiling keep it exact?"); writes only O and LSE = m + ln l, never S or P
 * ("How does FlashAttention save memory in the backward pass?": the per-row
 * softmax statistics are the only residual).
 *   q, k, v : in,  bf16 [B,H,N,d]
 *   o       : out, bf16 [B,H,N,d]
 *   lse     : out, fp32 [B,H,N], natural-log log-sum-exp of each score row
 */
FA_API fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
                 float scale, int causal, void* stream);

/*
 * Bytes of device workspace fa_bwd needs for this shape (0 when empty).
 * The workspace holds D = rowsum(dO o O) and the log2-domain LSE, both fp32
 * per row padded to a multiple of 128 rows, and the fp32 dQ accumulator.
 * Returns (size_t)-1 when the arguments are invalid.
 */
FA_API size_t fa_bwd_workspace_size(int B, int H, int N, int d);

/*
 * Backward pass, bf16, for a loss L with dL/dO = dO.
 * Recomputes S and P = exp(S - LSE) tile by tile from Q, K and the saved LSE
 * instead of reading a stored P ("How does FlashAttention save memory in the
 * backward pass?"; "The Real Complexity", recomputation on the backward pass),
 * then forms D = rowsum(dO o O), dV = P^T dO, dP = dO V^T, dS = P o (dP - D),
 * dQ = scale dS K, dK = scale dS^T Q (chain rule through S = scale Q K^T).
 * dQ is accumulated across key tiles with fp32 atomics, so its low bits may
 * differ from run to run.
 *   q, k, v, o, dO : in,  bf16 [B,H,N,d]  (o: the forward's output)
 *   lse            : in,  fp32 [B,H,N]    (the forward's LSE)
 *   dq, dk, dv     : out, bf16 [B,H,N,d]
 *   workspace      : scratch device memory of >= workspace_bytes bytes, at
 *                    least fa_bwd_workspace_size(B,H,N,d); contents on entry
 *                    are ignored and on exit are unspecified.  Must not be
 *                    used by another call that overlaps this one on the GPU.
 */
FA_API fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                 void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal,
                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa_bwd with per-launch timing: the same computation, arguments and errors
 * as fa_bwd, and additionally records four CUDA events (cudaEvent_t values
 * passed as opaque pointers, created by the caller) on `stream`:
 *   events[0] before the preprocess launch (D = rowsum(dO o O)),
 *   events[1] before the recompute kernel (S, P, dV, dP, dS, dK, dQ),
 *   events[2] after it, before the dQ conversion to bf16,
 *   events[3] after the last launch.
 * The elapsed time between events[1] and events[2] is the main kernel's own
 * duration on the launching stream.  Any NULL event returns
 * FA_ERR_INVALID_ARG before anything is launched.
 */
FA_API fa_status fa_bwd_events(const void* q, const void* k, const void* v, const void* o, const void* dO,
                               const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                               float scale, int causal, void* workspace, size_t workspace_bytes,
                               void* const* events, void* stream);

/*
 * Backward pass with a deterministic dQ: same arguments, outputs and workspace
 * as fa_bwd, but dQ is produced by a separate query-tile-parallel pass that
 * recomputes S, P and dP per query tile and accumulates dQ_i += dS K_j in
 * on-chip memory, writing each row once (no atomics).  Repeated calls on the
 * same inputs return bit-identical dQ, dK and dV.  Costs two more GEMMs per
 * tile pair (the recomputed S and dP) than fa_bwd.
 */
FA_API fa_status fa_bwd_deterministic(const void* q, const void* k, const void* v, const void* o, const void* dO,
                                      const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                                      float scale, int causal, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * Launch plan of fa_fwd and fa_fwd_fp8 for a shape, computed on the host as
 * the forward computes it (no launch; uses the current device's SM count, or
 * 148 when no device is visible).  A work item is one 128-row Q tile or a
 * pair of them of one (batch, head):
 *   *ctas       : CTAs launched (d = 64 non-causal runs at most one
 *                 persistent CTA per SM over the items)
 *   *items      : work items
 *   *pair_items : items that hold a pair of Q tiles; on non-causal grids the
 *                 pairs of a last round that would fill at most half of the
 *                 SMs are split into single-tile items dispatched last.
 * scale is not an argument; the other arguments are checked as in fa_fwd.
 */
FA_API fa_status fa_fwd_plan(int B, int H, int N, int d, int causal, int* ctas, int* items, int* pair_items);

/*
 * Forward pass with float8 e4m3 inputs and per-tensor scales ("What changed
 * between FlashAttention 1, 2, and 3?": low-precision FP8 forward).
 * The real inputs are q8 * q_descale, k8 * k_descale, v8 * v_descale.  The
 * score and value descales are folded into the exponent argument and the
 * final normalisation; P is rounded to e4m3 for the P V product while the
 * denominator l is summed in fp32.
 *   q8, k8, v8 : in,  e4m3 (fn) bytes [B,H,N,d]
 *   o          : out, bf16 [B,H,N,d]
 *   lse        : out, fp32 [B,H,N]
 * d must be 128 (a head row is one 128-byte swizzle span); causal is supported.
 */
FA_API fa_status fa_fwd_fp8(const void* q8, const void* k8, const void* v8, float q_descale, float k_descale,
                     float v_descale, void* o, float* lse, int B, int H, int N, int d, float scale, int causal,
                     void* stream);

/*
 * Backward pass of fa_fwd_fp8: gradients with respect to the real inputs
 * q8 * q_descale, k8 * k_descale, v8 * v_descale of the e4m3 forward
 * ("What changed between FlashAttention 1, 2, and 3?" names low-precision
 * FP8 as the forward's speed lever; the backward is the chain rule of the same
 * attention, as in fa_bwd).
 * Every e4m3 value is exactly a bf16 value, so the e4m3 Q, K and V are first
 * widened to bf16 in the workspace (no rounding) and the bf16 backward
 * kernels run on them; the descales are folded into the score factor
 * (scale * q_descale * k_descale), into dP (v_descale), dK (scale * q_descale)
 * and dQ (scale * k_descale).  The probabilities P and the gradient dS stay
 * bf16: normalised P is about 1/N (below e4m3's smallest subnormal, 2^-9, at
 * N >= 1024 with diffuse attention) and dS has a data-dependent range, so
 * neither fits a per-tensor e4m3 scale.
 *   q8, k8, v8 : in,  e4m3 (fn) bytes [B,H,N,d] (the forward's inputs)
 *   o          : in,  bf16 [B,H,N,d] (fa_fwd_fp8's output)
 *   dO         : in,  bf16 [B,H,N,d]
 *   lse        : in,  fp32 [B,H,N] (fa_fwd_fp8's LSE)
 *   dq, dk, dv : out, bf16 [B,H,N,d], in the real (descaled) units
 *   workspace  : >= fa_bwd_fp8_workspace_size(B,H,N,d) bytes (fa_bwd's
 *                workspace plus the three widened tensors, 6 N d bytes per head)
 * d must be 128 (as fa_fwd_fp8); causal is supported; descales must be
 * finite and > 0.  dQ is reduced with fp32 atomics as in fa_bwd.
 */
FA_API fa_status fa_bwd_fp8(const void* q8, const void* k8, const void* v8, float q_descale, float k_descale,
                            float v_descale, const void* o, const void* dO, const float* lse, void* dq, void* dk,
                            void* dv, int B, int H, int N, int d, float scale, int causal, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Bytes of workspace fa_bwd_fp8 needs ((size_t)-1 for invalid arguments or d != 128). */
FA_API size_t fa_bwd_fp8_workspace_size(int B, int H, int N, int d);

/*
 * Backward pass for callers that cannot allocate device memory.  The pages
 * have no counterpart: this is a packaging variant of fa_bwd, not a step of
 * the method.  Some callers cannot call cudaMalloc where they run the
 * backward -- a plugin inside a framework that owns every device allocation
 * and gives the plugin no allocator, or a serving loop that reserves its
 * memory at start-up and must not allocate (or risk a device-wide
 * synchronisation) afterwards.  This entry point takes the same arguments as
 * fa_bwd minus the workspace, and allocates nothing: its scratch is a fixed
 * array of fa_bwd_noalloc_max_bytes() bytes (64 MiB) inside the library,
 * which every GPU that loads the library holds until the process exits.
 *   - Shapes whose fa_bwd_workspace_size() exceeds that limit are rejected
 *     with FA_ERR_SCRATCH_LIMIT before anything is launched.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - All calls share the array and it keeps the last call's contents; the
 *     part that must start at zero is cleared by each call itself.  Calls
 *     whose GPU work overlaps (other streams, unordered host threads) race
 *     on it and must be serialised by the caller.
 */
FA_API fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dO,
                                const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                                float scale, int causal, void* stream);

/* Size in bytes of fa_bwd_noalloc's fixed scratch array. */
FA_API size_t fa_bwd_noalloc_max_bytes(void);

/*
 * Decode against a KV cache: Nq (1..16) new queries per (batch, head) attend
 * over Nk cached keys (chipfoundryservices glossary "flash attention", closing
 * section: the method serves inference against a KV cache).  The key range is split
 * across CTAs; each split keeps its own running max and sum, and the splits
 * are combined by their log-sum-exp (O = sum_s exp(LSE_s - LSE) O_s).  HBM-
 * bound: K and V are read once.
 *   q      : in,  bf16 [B,H,Nq,d]
 *   k, v   : in,  bf16 [B,H,Nk,d]
 *   o      : out, bf16 [B,H,Nq,d]
 *   lse    : out, fp32 [B,H,Nq]
 *   causal : query i of the Nq sees keys j <= Nk - Nq + i (the queries are the
 *            last Nq positions of the sequence); needs Nk >= Nq.
 *   workspace : >= fa_fwd_decode_workspace_size(B,H,Nq,Nk,d) bytes of device
 *            scratch for the per-split partial results (may be NULL when that
 *            size is 0 or the plan uses a single split).
 * Errors: FA_ERR_UNSUPPORTED for Nq > 16 or d not in {64,128};
 * FA_ERR_INVALID_ARG for Nk == 0 (with queries) or causal with Nk < Nq.
 */
FA_API fa_status fa_fwd_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                               int Nq, int Nk, int d, float scale, int causal, void* workspace,
                               size_t workspace_bytes, void* stream);

/* Bytes of workspace fa_fwd_decode needs ((size_t)-1 for invalid arguments). */
FA_API size_t fa_fwd_decode_workspace_size(int B, int H, int Nq, int Nk, int d);

/*
 * Standard (materialising) attention, the baseline the method is measured
 * against (explainers.rudrite.com "flash-attention-anatomy", Q&A "Why is
 * attention memory-bound, and how does FlashAttention fix it?": S is written
 * to HBM, read back for the softmax, P written, and read again for P V).
 * Same arguments and results as fa_fwd (O bf16, LSE fp32 natural log, causal
 * top-left aligned), computed in three passes through the workspace:
 *   S = scale Q K^T   fp32 [B,H,N,Np]   (Np = N rounded up to 128)
 *   P = softmax(S)    bf16 [B,H,N,Np]   (normalised; causal mask applied here)
 *   O = P V
 * workspace: >= fa_fwd_standard_workspace_size(B,H,N,d) bytes of device
 * memory, 256-byte aligned; about 6 N^2 bytes per head.
 */
FA_API fa_status fa_fwd_standard(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                                 int N, int d, float scale, int causal, void* workspace, size_t workspace_bytes,
                                 void* stream);

/* Bytes of workspace fa_fwd_standard needs ((size_t)-1 for invalid arguments). */
FA_API size_t fa_fwd_standard_workspace_size(int B, int H, int N, int d);

/*
 * Serving over an 8-bit paged KV cache: fa_page_tables, fa_rope,
 * fa_cache_append_fp8 and fa_fwd_decode_paged_fp8 are a decode step's calls
 * around the model's projections (chipfoundryservices glossary "flash
 * attention", closing section: inference against a KV cache).
 *
 * The cache.  A page holds page_size (16, 32, 64 or 128) tokens of every KV
 * head: k_cache and v_cache are e4m3 [num_pages, Hkv, page_size, d], and each
 * page and head has one scale, k_scale and v_scale fp32 [num_pages, Hkv]; a
 * stored value is code * scale.  block_table int32 [B, max_pages] lists each
 * request's pages in order, a slot is page * page_size + row of the page.
 * All lengths and tables are device memory that the kernels read: a step can
 * be captured into a CUDA graph and replayed as the lengths grow.
 *
 * What the host cannot check is checked by the kernels: a length below zero
 * or beyond the table counts as the nearest possible one; a page or slot
 * outside the cache is skipped (its keys count as not visible) and
 * fa_device_status then returns FA_ERR_BAD_PAGE.
 *
 * Limits (FA_ERR_UNSUPPORTED beyond): B * H <= 65535, or B <= 8192 and H <=
 * 65535 (Hkv in fa_cache_append_fp8); fa_page_tables B <= 65535; B * N, num_pages
 * * Hkv and num_pages * page_size below 2^31, max_pages * page_size up to 2^30.
 */

/* Scalings of the rotary frequencies f_i = base^(-2 i / rot_dim). */
typedef enum fa_rope_scaling {
  FA_ROPE_NONE = 0,    /* f_i */
  FA_ROPE_LINEAR = 1,  /* f_i / factor: positions interpolated */
  FA_ROPE_NTK = 2,     /* the base raised to base * factor^(rot_dim / (rot_dim - 2)) */
  FA_ROPE_YARN = 3,    /* between f_i / factor and f_i by a ramp over i, whose ends are the pairs that make `high`
                          and `low` turns within original_length; the rotation is multiplied by 0.1 ln(factor) + 1 */
  FA_ROPE_BANDS = 4    /* between f_i / factor and f_i by the number of turns within original_length: f_i / factor
                          up to `low` turns, f_i from `high` turns on, linear in between */
} fa_rope_scaling;

/*
 * Rotary frequencies of rot_dim / 2 pairs, computed on the host in 64 bits
 * (no GPU involved): inv_freq[i] in radians per position, *attention_factor
 * the factor of the rotation (1 but for FA_ROPE_YARN).  factor >= 1;
 * original_length, low and high are used by FA_ROPE_YARN and FA_ROPE_BANDS
 * (0 < low < high).  The caller copies inv_freq to the device once.
 */
FA_API fa_status fa_rope_frequencies(double* inv_freq, double* attention_factor, int rot_dim, double base,
                                     int scaling, double factor, double original_length, double low, double high);

/*
 * Rotary positions: turns each pair (u, w) of the first rot_dim elements of
 * every head row by a = position * inv_freq[pair],
 *   u' = factor * (u cos a - w sin a),  w' = factor * (w cos a + u sin a),
 * and copies the other d - rot_dim elements.  transpose != 0 turns by -a: the
 * gradient of the call with respect to x, applied to the gradient of y.
 *   x, y        : in/out, bf16 [B,H,N,d] with strides: xb, xh, xn and yb, yh, yn
 *                 are the elements from one batch, head and token to the next;
 *                 d is contiguous.  y may be x with equal strides (in place);
 *                 otherwise they must not overlap.  An input may repeat rows
 *                 (stride 0), an output may not.
 *   positions   : in, int32 [B,N] (any value), or NULL for 0..N-1
 *   inv_freq    : in, fp64 [rot_dim/2], device memory, 8-byte aligned
 *   interleaved : pairs are elements (2i, 2i+1), else (i, i + rot_dim/2)
 * rot_dim is a multiple of 16, at most d; strides are multiples of 8 elements.
 * Angles are reduced in 64 bits, so positions of 10^6 and more keep their accuracy.
 */
FA_API fa_status fa_rope(const void* x, void* y, const int* positions, const double* inv_freq, float factor, int B,
                         int H, int N, int d, int rot_dim, int interleaved, int transpose, long long xb,
                         long long xh, long long xn, long long yb, long long yh, long long yn, void* stream);

/*
 * Page tables of a batch, built on the GPU from request lengths.  Request b
 * holds ctx_lens[b] tokens and asks for new_lens[b] more (0..N), or has
 * finished (new_lens[b] < 0).
 *   1. The pages of finished requests go back, in order of the requests, in
 *      front of the free ones: free_pages[*free_head ..] grows downwards.
 *   2. Requests take the pages they need from the front, in order.  A request
 *      is granted if it needs none or if the needs up to and with its own fit;
 *      one that does not fit, that asks for more than N tokens or that would
 *      not fit its row of the table keeps its length and gets no slot.
 *   ctx_lens    : in,  int32 [B]
 *   new_lens    : in,  int32 [B]
 *   free_pages  : in/out, int32 [n_free]; free from index *free_head on
 *   free_head   : in,  int32 [1], device memory
 *   block_table : in/out, int32 [B, max_pages]; only the entries of pages that
 *                 are taken are written (a finished request's row stays)
 *   slots       : out, int32 [B,N]: slot of new token t, -1 where there is none
 *   positions   : out, int32 [B,N]: ctx_lens[b] + t, 0 where there is none
 *   seq_lens    : out, int32 [B]: new length (0 when finished); may be ctx_lens
 *   free_head_out : out, int32 [1]; may be free_head
 * A request was granted iff seq_lens[b] = ctx_lens[b] + new_lens[b].  N = 0
 * only gives pages back.  A page belongs to one request: one that stands in the
 * rows of two finished requests (a shared prompt) would go back twice.  If more
 * pages come back than ever were taken (the returned ones exceed *free_head),
 * none does and FA_ERR_BAD_PAGE is recorded.  A request holds the pages of
 * ctx_lens and no others, so a caller that lowers ctx_lens across a page's border
 * (rejected tokens of a draft) loses the page behind it: fa_page_tables_held is
 * for that.
 */
FA_API fa_status fa_page_tables(const int* ctx_lens, const int* new_lens, int* free_pages, const int* free_head,
                                int* block_table, int* slots, int* positions, int* seq_lens, int* free_head_out,
                                int B, int N, int n_free, int max_pages, int page_size, void* stream);

/*
 * fa_page_tables for requests that may also shrink between calls.
 *   held_pages  : in/out, int32 [B]: how many entries of its row of block_table
 *                 are the request's (0 for a new one), at least the pages of
 *                 ctx_lens[b] and at most max_pages (another number counts as the
 *                 nearest of these); or NULL, for fa_page_tables
 * Pages behind a lowered ctx_lens[b] stay the request's: new tokens go into them
 * before pages are taken, and they go back with the others when it has finished.
 * held_pages[b] gets the number after the call, 0 for a finished request.
 */
FA_API fa_status fa_page_tables_held(const int* ctx_lens, const int* new_lens, int* free_pages, const int* free_head,
                                     int* block_table, int* slots, int* positions, int* seq_lens, int* free_head_out,
                                     int* held_pages, int B, int N, int n_free, int max_pages, int page_size,
                                     void* stream);

/*
 * Writes new keys and values into the 8-bit cache.
 *   k, v    : in, bf16 [B,Hkv,N,d]
 *   slots   : in, int32 [B,N]; a negative slot's token is not written
 * Tokens of one request that follow one another on one page are quantised
 * together, and a page is written by one such run only (a page that two runs
 * name ends up with the codes of both under the scale of either).  Where two
 * tokens of a run name one slot, the later one is stored.  With amax the
 * largest finite absolute value of the run in that head:
 *   e     = smallest exponent in [-60, 60] with amax <= 448 * 2^e (-60 for amax = 0)
 *   scale = 2^e if the run writes the page's row 0 (the page starts anew, its
 *           old codes and scale mean nothing), else max(old scale, 2^e)
 *   code  = e4m3(x / scale), round to nearest even; what is not finite is
 *           stored as NaN, what exceeds 448 * 2^60 as the largest value.
 * If the scale grows, the page's other codes become e4m3(code * old / new).
 * Scales that the call makes are powers of two, so that step is exact down to
 * the type's subnormals; a page's old scale may be any positive number.  An old scale that is not positive and finite keeps nothing of
 * the page (its other codes become 0).
 */
FA_API fa_status fa_cache_append_fp8(const void* k, const void* v, const int* slots, void* k_cache, void* v_cache,
                                     float* k_scale, float* v_scale, int B, int Hkv, int N, int d, int num_pages,
                                     int page_size, void* stream);

/*
 * Decode against the 8-bit paged cache: Nq (1..16) new queries of each head
 * attend over the first seq_lens[b] tokens of request b (the queries' own
 * tokens are in the cache and counted).  H is a multiple of Hkv; query heads
 * h * H/Hkv .. (h+1) * H/Hkv - 1 share KV head h.
 * A chunk of a prompt behind cached tokens has no call of its own: it goes in
 * slices of up to 16 queries, each of which reads the cache again.
 *   q           : in,  bf16 [B,H,Nq,d]
 *   o           : out, bf16 [B,H,Nq,d]
 *   lse         : out, fp32 [B,H,Nq], natural log
 *   causal      : query i sees keys j <= seq_lens[b] - Nq + i
 *   workspace   : >= fa_fwd_decode_paged_fp8_workspace_size(B,H,Hkv,Nq,d) bytes
 *                 of device scratch, contents on entry ignored; not to be used
 *                 by another call that overlaps this one on the GPU.  After
 *                 FA_ERR_DEVICE_TIMEOUT it is to be zeroed before a captured
 *                 call that uses it is replayed
 * A row that sees no key (length 0, or causal with i < Nq - seq_lens[b]) gets
 * O = 0 and LSE = -inf.  Bytes of the cache at or behind a request's length
 * have no effect, whatever they are.  A key or query with a NaN makes the rows
 * that see it NaN, a value's NaN those rows' outputs in its column.  The
 * scales that count must be 0 or within 2^-60..2^60; a NaN scale, or a negative
 * V scale, shows as NaN in the rows that see a key of its page.  Of keys that one row
 * sees, one is left out of LSE, and of the sum that O is divided by, where its
 * weight times its V scale is below 2^-126 of the largest such product: with V
 * scales of one request and head within a factor of 2^90 of one another, that is
 * a weight below 2^-36.  In O's sum over the values themselves, weight times V
 * scale has 11 bits down to 2^-23 of the largest such product and is rounded to
 * multiples of 2^-33 of it at the coarsest below; under 2^-34 of it a key may be
 * gone.  A column of O in which only such light keys have codes other than 0 has
 * no more bits than that.
 */
FA_API fa_status fa_fwd_decode_paged_fp8(const void* q, const void* k_cache, const void* v_cache,
                                         const float* k_scale, const float* v_scale, const int* block_table,
                                         const int* seq_lens, void* o, float* lse, int B, int H, int Hkv, int Nq,
                                         int d, int num_pages, int page_size, int max_pages, float scale, int causal,
                                         void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace fa_fwd_decode_paged_fp8 needs ((size_t)-1 for invalid arguments). */
FA_API size_t fa_fwd_decode_paged_fp8_workspace_size(int B, int H, int Hkv, int Nq, int d);

/* Human-readable text for a status code (static storage, never NULL). */
FA_API const char* fa_strerror(fa_status status);

/*
 * Reads and clears the library's device status word on the current device.
 * Synchronises `stream` first.  Returns FA_OK, or FA_ERR_DEVICE_TIMEOUT if a
 * bounded wait inside a kernel ran out since the last call (the kernel then
 * abandoned its tile and returned; its outputs are undefined), or
 * FA_ERR_BAD_PAGE if a kernel skipped a page or slot outside the cache.
 * *where, if not NULL, receives a code naming the wait or the check.
 */
FA_API fa_status fa_device_status(void* stream, uint32_t* where);

/*
 * fa_device_status(stream, NULL): the device status check without the code
 * of the wait site.
 */
FA_API fa_status fa_get_device_status(void* stream);

/*
 * Self-test of the bounded-wait machinery: launches one block that waits on a
 * barrier nobody arrives at, with the given limit in microseconds (1..10^6),
 * so the wait runs out and the status word is set.  Used by the tests to
 * check that a stuck wait ends with a status, not a hang.
 */
FA_API fa_status fa_watchdog_selftest(uint32_t limit_us, void* stream);

/* Library version as major*10000 + minor*100 + patch. */
FA_API int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
