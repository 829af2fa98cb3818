/*
 * star.h — C ABI of the Star Attention hot path for NVIDIA B200 (sm_100a).
 *
 * Star Attention (arXiv 2411.17116) encodes a long context in two phases:
 *   Phase 1  the context is split into blocks c_1..c_n of b tokens; every
 *            block i >= 2 is prefixed with the anchor block c_1, which keeps
 *            its original position IDs, and attends causally only inside that
 *            augmented block; the anchor's KV entries are then dropped
 *            [pith 2WVXFXZ2, "What carries the argument"; minor comment on
 *            Section 2.1: c'_1 = c_1 has b tokens, only blocks i >= 2 carry
 *            the anchor].
 *   Phase 2  query and generated tokens attend to every cached token: each
 *            block ("host") returns a local attention output and a softmax
 *            statistic, and the query side re-weights them into exact
 *            global attention [pith 2WVXFXZ2, Referee summary; Circularity
 *            check; minor comment on Algorithm 2: weight exp(s_h - s_global)].
 * On one GPU the pages' hosts become blocks processed in parallel.
 *
 * Conventions shared by every call
 *   - Memory is owned by the caller (device pointers unless stated). The
 *     library allocates nothing and keeps no state besides a thread-local
 *     error message and per-device properties it caches on first use.
 *   - Every call is asynchronous on `cuda_stream` (a cudaStream_t; NULL is
 *     the legacy default stream). None synchronises, except
 *     star_device_status.
 *   - Arguments are validated before anything is launched; on a non-OK
 *     status nothing was enqueued (except STAR_ERR_CUDA from a launch).
 *   - Element types: bf16 for Q/K/V/O and the KV cache, fp32 for LSE and
 *     partials. LSE values are natural logarithms.
 *   - Softmax scale 1/sqrt(D). Query head h uses KV head h / (Hq / Hkv)
 *     (contiguous GQA groups).
 *   - RoPE is rotate-half with base theta: pair (x_i, x_{i+D/2}) turns by the
 *     angle p * theta^(-2i/D); token t of the context sits at position t, so
 *     the anchor keeps positions 0..a-1 in every block.
 *   - Supported head_dim D: 64 and 128; at most 2048 heads. Pointers must be
 *     16-byte aligned.
 *   - Device errors found inside kernels (a bounded wait that gave up, an
 *     index outside its buffer) are recorded in a status word at the start of
 *     the call's workspace and read back by star_device_status.
 *   - A workspace must be zero-filled once before its first use. After that
 *     the library keeps it consistent: status bits are sticky (calls OR them
 *     in, only star_device_status reads and clears them), and the counters of
 *     the decode path, which every Phase-2 call keeps at the start of its
 *     workspace, return to zero at the end of every call (after a device
 *     error star_device_status clears them too). A workspace that decode
 *     calls use may be shared with other Phase-2 calls of the same B, Hkv,
 *     Lcap and block_len; before any other reuse it must be zero-filled
 *     again. No call resets the workspace, so consecutive decode kernels run
 *     back to back: the decode kernel is launched as a programmatic dependent
 *     launch and may start while the previous kernel in the stream drains.
 *     It streams cache rows [0, L) at once and waits for that kernel to end
 *     before it reads q, k or v, touches the tail rows, or writes anything.
 *     Cache rows [0, L) must therefore not be written by the kernel launched
 *     just before a decode call (Phase 1 never is: its last kernel only reads
 *     the cache), and consecutive decode calls on one cache keep the context
 *     length L and grow only the tail. This is how Phase 2 proceeds: the
 *     context is fixed after Phase 1.
 */
#ifndef STAR_H_
#define STAR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  STAR_OK = 0,
  STAR_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size or shape */
  STAR_ERR_UNSUPPORTED = 2,   /* head_dim or device not supported */
  STAR_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed */
  STAR_ERR_DEVICE_TIMEOUT = 4,/* a kernel's bounded wait gave up */
  STAR_ERR_DEVICE_BOUNDS = 5  /* a kernel found an index outside its buffer */
} star_status;

/* Message describing the calling thread's last non-OK status ("" if none).
 * The pointer stays valid until the next call on the same thread. */
const char* star_last_error(void);

/* Library version string; it ends with the digest of the sources, headers and
 * build flags the library was built from. */
const char* star_version(void);

/*
 * star_rope — rotate-half RoPE at given positions
 * [pith 2607.20457, "What carries the argument": original global position
 * IDs preserve RoPE distances; pith 2WVXFXZ2: the anchor keeps c_1's
 * original positional indices].
 *
 *   y[b,s,h,:] = RoPE(x[b,s,h,:], p_s),  p_s = pos[s] if pos != NULL else pos0 + s
 *
 * x, y: bf16, D contiguous; x_stride / y_stride give the element strides of
 * the (B, S, H) dimensions (each a multiple of 8). x and y may be the same
 * buffer (in place) but must not otherwise overlap. pos: device int32[S] or
 * NULL. Angles, their reduction modulo 2*pi and sine/cosine are fp64; y is
 * the correctly rounded bf16 (nearest even) of the exact rotation.
 */
star_status star_rope(const void* x, const int64_t x_stride[3], void* y,
                      const int64_t y_stride[3], const int32_t* pos, int64_t pos0, int B,
                      int S, int H, int D, double theta, void* cuda_stream);

/* Workspace bytes star_phase1_encode needs: the rotated Q (bf16
 * [B, L, Hq, D]) plus a 256-byte status header. */
size_t star_phase1_workspace_bytes(int B, int L, int Hq, int D);

/*
 * star_phase1_encode — Phase 1, anchor-block blockwise-local causal encoding
 * [pith 2WVXFXZ2, "What carries the argument"; minor comment on
 * Section 2.1; abstract: "the context is processed using blockwise-local
 * attention ... in parallel"].
 *
 * Inputs (pre-RoPE, token-major): q[B, L, Hq, D], k/v[B, L, Hkv, D].
 * Row r of block i = r / block_len attends to
 *   i == 0 : keys [0, r]                       (c'_1 = c_1, plain causal)
 *   i >= 1 : keys [0, anchor_len) U [i*block_len, r]
 * The anchor's keys are block 1's cache rows (same tokens, same positions),
 * so they are computed once and shared; no anchor copy is ever stored.
 * Outputs:
 *   o[B, L, Hq, D]             bf16, softmax-normalised
 *   k_cache/v_cache[B, Hkv, Lcap, D]  rows [0, L) written: K rotated, V copied
 *                              (head-major; rows >= L untouched)
 *   lse[B, Hq, L]              fp32 natural-log statistic, or NULL
 * anchor_len in [0, block_len]; 0 disables the anchor (the pages' "no
 * anchor" ablation); block_len >= L gives full causal attention.
 * Requires Lcap >= L, workspace_bytes >= star_phase1_workspace_bytes().
 */
star_status star_phase1_encode(const void* q, const void* k, const void* v, void* o,
                               void* k_cache, void* v_cache, int Lcap, float* lse, int B, int L,
                               int Hq, int Hkv, int D, int block_len, int anchor_len,
                               double theta, void* workspace, size_t workspace_bytes,
                               void* cuda_stream);

/*
 * star_phase1_encode_rotated — star_phase1_encode when the caller has already
 * rotated Q and written the cache (for example with star_linear_rope):
 * q_rot[B, L, Hq, D] holds RoPE'd queries at positions 0..L-1 and
 * k_cache/v_cache[B, Hkv, Lcap, D] rows [0, L) hold the rotated keys and the
 * values. Only the block-sparse attention runs; the visibility rule, o and
 * lse are those of star_phase1_encode. workspace: >= 256 bytes (the status
 * word), zero-filled once. Errors as star_phase1_encode.
 */
star_status star_phase1_encode_rotated(const void* q_rot, void* o, const void* k_cache,
                                       const void* v_cache, int Lcap, float* lse, int B, int L,
                                       int Hq, int Hkv, int D, int block_len, int anchor_len,
                                       void* workspace, size_t workspace_bytes,
                                       void* cuda_stream);

/* Workspace bytes star_phase1_encode_ext needs for a prefix table of G
 * rows: as star_phase1_encode plus the table's rotated K and its V (bf16
 * [B, Hkv, G, D] each). */
size_t star_phase1_ext_workspace_bytes(int B, int L, int Hq, int Hkv, int D, int G);

/*
 * star_phase1_encode_ext — Phase 1 with a generalised prefix. Instead of the
 * anchor of star_phase1_encode, every block sees a slice of one gathered
 * prefix table of G rows:
 *   table row g  = context row prefix_src[g] of k/v when prefix_src[g] >= 0,
 *                  row -1 - prefix_src[g] of extra_k/extra_v otherwise; its
 *                  key is rotated at position prefix_pos[g];
 *   block i sees table rows [prefix_bounds[2i], prefix_bounds[2i+1]), all
 *                  visible, then its own rows causally at their own positions.
 * This covers the Star anchor (rows 0..a-1 at positions 0..a-1, blocks i >= 1
 * see [0, a)) [pith 2WVXFXZ2, "What carries the argument"]; the anchor
 * ablations — no anchor, anchor position IDs moved or randomised, anchor
 * content replaced (atlas.scime.ai summary, measured-effects table); and
 * Pulsar's [sink || Sigma_0 || ... || Sigma_{i-1} || B_i] with every row at
 * its original global position, one table of which block i sees a leading
 * part [pith 2607.20457, "What carries the argument"]. A row listed twice
 * counts twice; block 0 takes its slice too.
 *
 * prefix_src, prefix_pos : device int32 [G]; prefix_bounds: device int32
 *   [n][2], n = ceil(L / block_len). All three may be NULL when G == 0.
 * extra_k, extra_v : device bf16 [B, n_extra, Hkv, D] pre-RoPE, 16-byte
 *   aligned; NULL when n_extra == 0.
 * ctx_pos0 : position of context row 0 (row r of q/k/v sits at ctx_pos0 + r;
 *   0 for a whole sequence). A shard of a sequence split by blocks over
 *   several GPUs passes the global position of its first row, with the
 *   anchor as given rows at positions 0..a-1 [pith 2WVXFXZ2, "What carries
 *   the argument": every host gets the anchor block with its original
 *   positions]. Block boundaries are counted from row 0 of the call.
 * Other arguments, the outputs and the KV cache as for star_phase1_encode.
 * Errors: invalid arguments as for star_phase1_encode (STAR_ERR_INVALID_ARG,
 *   nothing launched). A prefix_src outside [-n_extra, L) gives a zero row; a
 *   slice outside [0, G] (or reversed) is clamped to it; either records
 *   STAR_ERR_DEVICE_BOUNDS in the workspace status word (star_device_status).
 */
star_status star_phase1_encode_ext(const void* q, const void* k, const void* v, void* o,
                                   void* k_cache, void* v_cache, int Lcap, float* lse, int B, int L,
                                   int Hq, int Hkv, int D, int block_len, const int32_t* prefix_src,
                                   const int32_t* prefix_pos, int G, const int32_t* prefix_bounds,
                                   const void* extra_k, const void* extra_v, int n_extra,
                                   int ctx_pos0, double theta, void* workspace,
                                   size_t workspace_bytes, void* cuda_stream);

/* Workspace bytes star_phase2_partial needs for up to T new tokens with a
 * cache of capacity Lcap (context L plus tail) split into blocks of
 * block_len: the header (256-byte status block, then the decode path's
 * split and head counters, kept on every Phase-2 path), the rotated q and,
 * on the decode path (T * Hq / Hkv <= 16), the chunk partials. */
size_t star_phase2_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int Lcap, int block_len);

/*
 * star_phase2_partial — Phase 2 per-block partial attention
 * [pith 2WVXFXZ2, Referee summary: the query is broadcast and each host
 * computes local softmax statistics; abstract: query and response tokens
 * attend to all prior cached tokens].
 *
 * T new tokens (a query chunk, or one decode token) with pre-RoPE
 * q[B, T, Hq, D], k/v[B, T, Hkv, D] sit at positions L + tail_len + t. The
 * call rotates q and k, appends k/v into cache rows L + tail_len + t, then
 * for every split writes the split-local softmax-normalised output and its
 * LSE:
 *   split j < n (n = ceil(L / block_len)): context block j, keys
 *                 [j*block_len, min((j+1)*block_len, L)), all visible
 *   split n (tail): cache rows [L, L + tail_len + t], causal per token
 *   part_o[B, Hq, n+1, T, D] fp32, part_lse[B, Hq, n+1, T] fp32
 * *nsplit_out (host int, may be NULL) receives n + 1.
 * Requires Lcap >= L + tail_len + T and cache rows [0, L + tail_len) filled
 * by earlier calls; workspace_bytes >= star_phase2_workspace_bytes().
 */
star_status star_phase2_partial(const void* q, const void* k, const void* v, int T, void* k_cache,
                                void* v_cache, int Lcap, int L, int block_len, int tail_len,
                                float* part_o, float* part_lse, int* nsplit_out, int B, int Hq,
                                int Hkv, int D, double theta, void* workspace,
                                size_t workspace_bytes, void* cuda_stream);

/*
 * star_phase2_attend — star_phase2_partial followed by the exact merge of its
 * partials (as star_lse_merge) in the same call [pith 2WVXFXZ2, Referee
 * summary; minor comment on Algorithm 2]. part_o / part_lse are written as
 * by star_phase2_partial; o[B, T, Hq, D] bf16 (required) and lse[B, Hq, T]
 * fp32 (nullable) receive the merged global attention. On the decode path
 * (T * Hq / Hkv <= 16) the merge runs inside the decode kernel: the last CTA
 * to finish the splits of a (batch, KV head) merges them, so no extra launch
 * is made. Workspace as for star_phase2_partial.
 */
star_status star_phase2_attend(const void* q, const void* k, const void* v, int T, void* k_cache,
                               void* v_cache, int Lcap, int L, int block_len, int tail_len,
                               float* part_o, float* part_lse, void* o, float* lse,
                               int* nsplit_out, int B, int Hq, int Hkv, int D, double theta,
                               void* workspace, size_t workspace_bytes, void* cuda_stream);

/*
 * star_phase2_partial_ext — star_phase2_partial for one shard of a sequence
 * whose context blocks are spread over several GPUs [pith 2WVXFXZ2, Referee
 * summary: the query is broadcast, every host computes a local attention
 * output and softmax statistic over its own KV cache, the query host
 * re-weights them; "What carries the argument": KV caches never move].
 *   cache row r (r < L + tail_len) sits at position ctx_pos0 + r;
 *   new token t is rotated at position q_pos0 + t;
 *   with_tail = 1 (the query host): as star_phase2_partial — the new tokens'
 *     k/v are rotated and appended at cache rows L + tail_len + t, which
 *     requires q_pos0 == ctx_pos0 + L + tail_len, and split n is the causal
 *     tail; nsplit = n + 1;
 *   with_tail = 0 (any other host): context splits only; k and v are unused
 *     (may be NULL), tail_len must be 0, nothing is written to the cache;
 *     nsplit = n.
 * n = ceil(L / block_len) counts the shard's own blocks. part_o [B, Hq,
 * nsplit, T, D] and part_lse [B, Hq, nsplit, T] fp32 as star_phase2_partial.
 * Workspace: star_phase2_workspace_bytes(B, T, Hq, Hkv, D, Lcap, block_len).
 * Errors: STAR_ERR_INVALID_ARG for negative positions, with_tail not 0/1,
 * q_pos0 inconsistent with the tail, or positions past int32.
 */
star_status star_phase2_partial_ext(const void* q, const void* k, const void* v, int T,
                                    void* k_cache, void* v_cache, int Lcap, int L, int block_len,
                                    int tail_len, int ctx_pos0, int q_pos0, int with_tail,
                                    float* part_o, float* part_lse, int* nsplit_out, int B, int Hq,
                                    int Hkv, int D, double theta, void* workspace,
                                    size_t workspace_bytes, void* cuda_stream);

/*
 * star_lse_merge — exact merge of per-split partials into global attention
 * [pith 2WVXFXZ2, minor comment on Algorithm 2 (corrected update
 * exp(s_h - s_global) * A_h); assumptions: online softmax aggregation gives
 * the exact global softmax]:
 *   m = max_h lse_h,  w_h = exp(lse_h - m),
 *   o = sum_h w_h o_h / sum_h w_h   -> o[B, T, Hq, D] bf16
 *   lse = m + log(sum_h w_h)        -> lse[B, Hq, T] fp32 (NULL to skip)
 * Splits whose lse is -inf carry weight 0. Inputs as star_phase2_partial
 * writes them.
 */
star_status star_lse_merge(const float* part_o, const float* part_lse, int nsplit, void* o,
                           float* lse, int B, int T, int Hq, int D, void* cuda_stream);

/*
 * star_lse_merge_ranks — star_lse_merge over partials gathered from several
 * ranks (the query host's aggregation step [pith 2WVXFXZ2, Referee summary]).
 * Every rank owns an equal slot of B * Hq * nsplit_stride * T * D floats of
 * part_o and B * Hq * nsplit_stride * T floats of part_lse (an all-gather of
 * equal-sized send buffers); rank r's slot begins with its nsplit_of_rank[r]
 * splits as star_phase2_partial_ext writes them, [B, Hq, nsplit_of_rank[r],
 * T, D] and [B, Hq, nsplit_of_rank[r], T]; the rest of the slot is ignored.
 * nsplit_of_rank is a host array, 0 <= nsplit_of_rank[r] <= nsplit_stride,
 * 1 <= nranks <= 64. Output and errors as star_lse_merge.
 */
star_status star_lse_merge_ranks(const float* part_o, const float* part_lse, int nranks,
                                 const int* nsplit_of_rank, int nsplit_stride, void* o, float* lse,
                                 int B, int T, int Hq, int D, void* cuda_stream);

/*
 * star_phase2_decode_static — star_phase2_partial for decode steps
 * (T * (Hq / Hkv) <= 16) without a workspace argument. The pages have no
 * counterpart: this entry point exists for callers that cannot allocate
 * device memory themselves, such as a plugin whose host application owns
 * every device allocation, or a serving loop that must never block in
 * cudaMalloc/cudaFree. Its scratch (the split counters and the per-chunk
 * partials) lives in a 16 MiB device array inside the library, which every
 * GPU that loads the library keeps until the process exits; the caller still
 * passes inputs and outputs, with the same meaning and layout as
 * star_phase2_partial.
 *   - The array's address is looked up once per device on the first call made
 *     with that device current; make that first call before any stream
 *     capture.
 *   - All calls on a device share the array, which keeps the previous call's
 *     contents: each call clears the split counters and rewrites the partials
 *     before reading them; device errors are ORed into a status word that
 *     stays set until star_phase2_decode_static_status reads it. Calls whose
 *     work overlaps on the GPU race on the array: serialise them (one stream,
 *     or explicit ordering).
 *   - Sizes whose scratch cannot fit 16 MiB even with the largest chunk, or
 *     T * g > 16, return STAR_ERR_INVALID_ARG before anything is enqueued.
 *     Nothing is allocated.
 */
star_status star_phase2_decode_static(const void* q, const void* k, const void* v, int T,
                                      void* k_cache, void* v_cache, int Lcap, int L,
                                      int block_len, int tail_len, float* part_o,
                                      float* part_lse, int* nsplit_out, int B, int Hq, int Hkv,
                                      int D, double theta, void* cuda_stream);

/*
 * star_phase2_decode_static_status — the device-error read-back of
 * star_phase2_decode_static, which has no workspace for star_device_status
 * to read. The pages have no counterpart. Synchronises `cuda_stream`, reads
 * the status word kept at the start of the current device's static array
 * (device errors of every star_phase2_decode_static call since the last
 * read are ORed into it: a bounded wait that gave up, an index outside its
 * buffer) and clears it. Returns STAR_OK, STAR_ERR_DEVICE_TIMEOUT or
 * STAR_ERR_DEVICE_BOUNDS (message in star_last_error), or STAR_ERR_CUDA.
 * After a device error the outputs of the calls since the last read are not
 * valid. Allocates nothing; the first call on a device looks up the array's
 * address like star_phase2_decode_static does.
 */
star_status star_phase2_decode_static_status(void* cuda_stream);

/*
 * Layers around Star attention in a decoder stack. Star Attention replaces
 * only attention and needs no retraining [pith 2WVXFXZ2, the paper's
 * abstract]; in a stack every layer encodes its own anchor, whose hidden
 * state is block 1's at that layer because the anchor is a causal prefix of
 * every augmented block [pith 2WVXFXZ2, "What carries the argument"]. These
 * two calls supply the row-wise parts of an attention block:
 *
 * star_rmsnorm — y[r, :] = x[r, :] / sqrt(mean(x[r, :]^2) + eps) * gamma,
 *   x, y bf16 [rows, dm] (row-major, may alias), gamma bf16 [dm]; fp32
 *   arithmetic, one rounding to bf16. dm a multiple of 8, pointers 16-byte
 *   aligned. STAR_ERR_INVALID_ARG otherwise; STAR_ERR_CUDA if the launch fails.
 *
 * star_linear — y[M, N] = x[M, K] * w[N, K]^T (accumulate = 0), or
 *   y = bf16(y + bf16(x * w^T)) (accumulate = 1: the stored projection, then
 *   the residual add), bf16 row-major operands, fp32 accumulation. It runs in
 *   the library's own tcgen05 GEMM (128 x 256 tiles, TMA-fed, persistent).
 *   N and K multiples of 8, x/w/y 16-byte aligned. workspace (caller-owned,
 *   256-byte aligned, >= 256 bytes, zero-filled once) holds the status word a
 *   bounded wait writes on a time-out (star_device_status reads it).
 *   STAR_ERR_INVALID_ARG for bad shapes or pointers, STAR_ERR_UNSUPPORTED off
 *   sm_100, STAR_ERR_CUDA for a failed launch.
 */
star_status star_rmsnorm(const void* x, const void* gamma, void* y, int rows, int dm, float eps,
                         void* cuda_stream);
star_status star_linear(const void* x, const void* w, void* y, int M, int N, int K, int accumulate,
                        void* workspace, size_t workspace_bytes, void* cuda_stream);

/*
 * star_linear_rope — a Q/K/V projection whose output goes straight to where
 * Star attention reads it [pith 2WVXFXZ2, "What carries the argument": keys
 * keep their original position IDs; pith 2607.20457: original global
 * positions preserve RoPE distances]:
 *   p = bf16(x[M, K] * w[N, K]^T), rows m = b * seq_len + t (token t of
 *   sequence b), N = H * head_dim columns (H heads);
 *   rotate = 1: every head is rotated as star_rope does (rotate-half, base
 *   theta, position pos0 + t), from the bf16 values p, correctly rounded, so
 *   the bits equal star_linear followed by star_rope;
 *   cache_rows = 0: y is row-major [M, N] (token-major [B, seq_len, H, D]);
 *   cache_rows > 0: y is a head-major KV cache [B, H, cache_rows, head_dim]
 *   and token t of sequence b lands in row t (rows >= seq_len untouched).
 * A Phase-1 layer projects Q with rotate = 1, cache_rows = 0, K with
 * rotate = 1 into its k_cache and V with rotate = 0 into its v_cache, then
 * calls star_phase1_encode_rotated: no separate RoPE pass.
 * head_dim 64 or 128; N a multiple of head_dim; M a multiple of seq_len;
 * cache_rows 0 or >= seq_len; at least one of rotate and a cache layout.
 * workspace: >= star_linear_rope_workspace_bytes(seq_len, head_dim, rotate)
 * bytes, 256-byte aligned, zero-filled once: the status word, then (rotate)
 * the call's fp32 cos/sin table of its seq_len positions, built by a small
 * kernel the call launches before the GEMM. Operands and errors as
 * star_linear.
 */
size_t star_linear_rope_workspace_bytes(int seq_len, int head_dim, int rotate);

/*
 * star_linear_kv_cache — a layer's K and V projections as one GEMM, written
 * straight into its KV cache: w_kv[2N, K] holds the K projection's N rows
 * and then the V projection's N rows (N = Hkv * head_dim). With
 * p = bf16(x[M, K] * w_kv^T): columns [0, N) are the keys, rotated as
 * star_linear_rope rotates them (position pos0 + t), into k_cache; columns
 * [N, 2N) are the values, unrotated, into v_cache; both caches head-major
 * [M / seq_len, Hkv, cache_rows, head_dim], token t of sequence b in row t.
 * The bits equal star_linear_rope(K, rotate = 1) and star_linear_rope(V,
 * rotate = 0) on the two halves; one launch fills the GPU better than two
 * narrow ones. cache_rows >= seq_len; workspace as star_linear_rope with
 * rotate = 1. Errors as star_linear_rope.
 */
star_status star_linear_kv_cache(const void* x, const void* w_kv, void* k_cache, void* v_cache,
                                 int M, int N, int K, int head_dim, int seq_len, int64_t pos0,
                                 double theta, int cache_rows, void* workspace,
                                 size_t workspace_bytes, void* cuda_stream);
star_status star_linear_rope(const void* x, const void* w, void* y, int M, int N, int K,
                             int head_dim, int rotate, int seq_len, int64_t pos0, double theta,
                             int cache_rows, void* workspace, size_t workspace_bytes,
                             void* cuda_stream);

/*
 * Serving many requests from an 8-bit paged cache.
 *
 * The calls above keep one bf16 cache of equal-length sequences. The five
 * below serve a ragged batch of requests whose keys and values are held in 8
 * bits, in pages: star_batch_plan gives each request's new tokens positions
 * and page rows, star_rope_scaled rotates their queries and keys,
 * star_kv8_append writes their keys and values into the pages, and
 * star_kv8_attend attends over the pages. A decode step reads half the bytes
 * of the bf16 cache.
 *
 *   pages   k_pages, v_pages [num_pages, Hkv, page_len, D], 8-bit codes;
 *           page_len 16, 32, 64 or 128 tokens; D 64 or 128
 *   scales  k_scale, v_scale fp32 [num_pages, Hkv]: a code stands for
 *           code * scale. star_kv8_append writes powers of two; star_kv8_attend
 *           takes any positive normal scale (0: a page of zeros)
 *   type    kv_type STAR_KV8_E4M3 (finite 8-bit floats up to 448, bit 7 the
 *           sign, 0x7f and 0xff NaN) or STAR_KV8_INT8 (two's complement,
 *           -127..127)
 *   table   block_table int32 [B, max_pages]: request b's token p is row
 *           p % page_len of page block_table[b, p / page_len]
 *   tokens  the new tokens of all requests are packed: request b's are rows
 *           cu_new[b] .. cu_new[b + 1] - 1; rows from cu_new[B] on are padding
 * At most 4096 requests a call; num_pages * page_len and max_pages * page_len
 * fit int32. Device arrays of lengths and indices are checked by the kernels:
 * what they would place outside a buffer is left out and recorded as
 * STAR_ERR_DEVICE_BOUNDS in the workspace's status word. A workspace is
 * zero-filled once and serves one call at a time: calls that may run at the
 * same time (two streams, two graphs) need one each.
 */
enum { STAR_KV8_E4M3 = 0, STAR_KV8_INT8 = 1 };
enum {
  STAR_ROPE_NONE = 0,   /* f_i = theta^(-2i/rot_dim) */
  STAR_ROPE_LINEAR = 1, /* f_i / factor */
  STAR_ROPE_NTK = 2,    /* base theta * factor^(rot_dim/(rot_dim-2)) */
  STAR_ROPE_YARN = 3,   /* by the turns of a pair within orig_len: see below */
  STAR_ROPE_LLAMA3 = 4
};

/*
 * star_rope_frequencies — inverse frequencies of rot_dim / 2 pairs (host
 * arithmetic in fp64; nothing is launched), scaled for contexts beyond the
 * trained length orig_len by `factor`:
 *   YARN    with d(n) = rot_dim * ln(orig_len / (2 pi n)) / (2 ln theta), lo =
 *           max(floor(d(a)), 0), hi = min(ceil(d(b)), rot_dim - 1) and r_i =
 *           clamp((i - lo) / (hi - lo), 0, 1) (hi - lo = 0.001 where they are
 *           equal): f_i / factor * r_i + f_i * (1 - r_i); a, b are the fast
 *           and slow turn counts; *mscale = 0.1 ln(factor) + 1
 *   LLAMA3  with n_i = orig_len * f_i / (2 pi), u_i = clamp((n_i - a) /
 *           (b - a), 0, 1): (1 - u_i) f_i / factor + u_i f_i; a, b are the low
 *           and high turn counts
 * *mscale is 1 except for YARN. inv_freq: host double [rot_dim / 2]. a, b and
 * orig_len are ignored where the scaling has none. STAR_ERR_INVALID_ARG for an
 * odd or non-positive rot_dim, rot_dim > 128, values that are not finite and
 * positive, factor < 1, theta <= 1, NTK with rot_dim 2, YARN with a < b, LLAMA3
 * with a >= b.
 */
star_status star_rope_frequencies(int rot_dim, double theta, int scaling, double factor,
                                  double orig_len, double a, double b, double* inv_freq,
                                  double* mscale);

/*
 * star_rope_scaled — rotary positions with given frequencies, over all or the
 * leading rot_dim elements of each head, at positions p_s (pos[b *
 * pos_stride_b + s], or pos0 + s when pos is NULL):
 *   half         pairs (x_i, x_{i + rot_dim/2}), i < rot_dim / 2
 *   interleaved  pairs (x_{2i}, x_{2i + 1})
 *   y_first  = mscale * (x_first cos(p f_i) - x_second sin(p f_i))
 *   y_second = mscale * (x_second cos(p f_i) + x_first sin(p f_i))
 * transpose = 1 turns by -p f_i instead, which is the gradient of x given
 * that of y. Elements from rot_dim on are copied. Angles are fp64 and y the
 * correctly rounded bf16, as star_rope: with rot_dim = D, mscale 1, the half
 * layout and unscaled frequencies the bits are star_rope's.
 * x, y: bf16 [B, S, H, D] with strides as star_rope; in place when x == y and
 * the strides agree, not overlapping otherwise. rot_dim: a multiple of 16, at
 * most D. inv_freq: host double [rot_dim / 2], read during the call.
 * mscale and frequencies finite.
 */
star_status star_rope_scaled(const void* x, const int64_t x_stride[3], void* y,
                             const int64_t y_stride[3], const int32_t* pos, int64_t pos_stride_b,
                             int64_t pos0, int B, int S, int H, int D, int rot_dim,
                             const double* inv_freq, double mscale, int interleaved,
                             int transpose, void* cuda_stream);

/* Entries that run_start of star_batch_plan needs, less one: the write runs
 * that n_tokens new tokens of B requests can make. */
int star_batch_plan_runs(int n_tokens, int B, int page_len);
/* Workspace bytes of star_batch_plan. */
size_t star_batch_plan_workspace_bytes(int B);

/*
 * star_batch_plan — one serving step's bookkeeping on the GPU, from request
 * lengths. Request b has ctx_len[b] cached tokens, in the pages that its row of
 * block_table lists, and brings new_len[b] >= 0 tokens. Pages that these need
 * beyond the listed ones are taken, request by request, from free_pages at
 * index *free_begin on and entered into block_table (in place).
 *   cu_new[B + 1]   token offsets; kv_len[B] = ctx_len + new_len
 *   pos[n_cap]      position of each new token (0 beyond the last)
 *   slot[n_cap]     page * page_len + row of each new token (-1 beyond)
 *   run_start[run_cap + 1]  first tokens of the write runs: the longest spans of
 *                   one request's new tokens within one page, in token order;
 *                   the entries after them hold the token count
 *   *free_next      *free_begin + the pages taken
 * All arrays are device int32, n_cap and run_cap host sizes (run_cap >=
 * star_batch_plan_runs(n_cap, B, page_len)). kv_len may be ctx_len, and
 * free_next may be free_begin: a captured step then advances with each replay.
 * No other outputs may overlap inputs or each other.
 * A step that does not fit (more tokens than n_cap, pages than free_pages
 * holds, a request beyond max_pages, a negative length) is refused as a
 * whole: cu_new and run_start are 0, slot -1, kv_len = ctx_len, *free_next =
 * *free_begin, block_table is untouched and the status word records
 * STAR_ERR_DEVICE_BOUNDS.
 */
star_status star_batch_plan(const int32_t* ctx_len, const int32_t* new_len, int B,
                            const int32_t* free_pages, int num_free, const int32_t* free_begin,
                            int page_len, int32_t* block_table, int max_pages, int32_t* cu_new,
                            int32_t* pos, int32_t* slot, int n_cap, int32_t* run_start,
                            int run_cap, int32_t* kv_len, int32_t* free_next, void* workspace,
                            size_t workspace_bytes, void* cuda_stream);

/*
 * star_kv8_append — writes new tokens' keys (already rotated) and values into
 * their pages in 8 bits. k, v: bf16 [n_tokens, Hkv, D], element strides
 * k_stride / v_stride of (token, head), multiples of 8, D contiguous. Run u
 * (run_start[u] < run_start[u + 1]) writes its tokens to consecutive rows from
 * slot[run_start[u]] on; a run whose slot is negative is skipped. Per head of
 * the run's page, with amax over the run's finite values:
 *   s = 2^ceil(log2(amax / 448)) (127 for int8), at least 2^-100
 *   a run that begins at row 0 starts the page: its scale becomes s. Otherwise
 *   the scale becomes max(old, s), and where it grew the earlier rows' codes are
 *   rounded again: code * old / s.
 * Codes are the nearest values, ties to even; infinities saturate; a NaN is
 * stored as NaN (e4m3) or 0 (int8). A page may be written by one run of a call
 * only. Rows behind the run keep their bytes. workspace: >= 256 bytes (the
 * status word). Runs outside their page, the tokens or the pages are left out
 * and recorded as STAR_ERR_DEVICE_BOUNDS.
 */
star_status star_kv8_append(const void* k, const int64_t k_stride[2], const void* v,
                            const int64_t v_stride[2], int n_tokens, int Hkv, int D,
                            const int32_t* slot, const int32_t* run_start, int run_cap,
                            void* k_pages, void* v_pages, float* k_scale, float* v_scale,
                            int num_pages, int page_len, int kv_type, void* workspace,
                            size_t workspace_bytes, void* cuda_stream);

/* Workspace bytes of star_kv8_attend for up to n_tokens new tokens, at most
 * max_new of one request. */
size_t star_kv8_attend_workspace_bytes(int B, int n_tokens, int Hq, int Hkv, int D, int max_new);

/*
 * star_kv8_attend — attention of the new tokens over their requests' pages.
 * q: bf16 [n_tokens, Hq, D], already rotated, element strides q_stride of
 * (token, head), multiples of 8. Request b has kv_len[b] tokens in its pages,
 * its T = cu_new[b + 1] - cu_new[b] new ones the last of them: new token t sees
 * keys [0, kv_len[b] - T + t + 1) of its request; a row that sees none gets o =
 * 0, lse = -inf. Scale 1/sqrt(D); query head h uses KV head h / (Hq / Hkv).
 *   o [n_tokens, Hq, D] bf16, lse [Hq, n_tokens] fp32 (NULL to skip)
 * Rows from cu_new[B] on are left as they are, and so is what lies in pages
 * behind kv_len, which may hold anything. o and lse overlap no input. max_new
 * bounds T, and max_kv kv_len (1 .. max_pages * page_len, at most 2^31 - 257):
 * they choose kernels and grids, lengths beyond them are an error. max_new * Hq
 * / Hkv is at most 2^24, and a call is refused where Hkv * (n_tokens * Hq / Hkv
 * / R + B) * max_kv / 128 reaches 2^31, R the rows of a tile (8 up to 8 rows of
 * a KV head and request, 16 up to 32, then 256). Scores are fp32 sums of exact
 * products (the codes enter the tensor cores unrounded, and so does q down to
 * 2^-29 of its row's largest element). Weights, times the ratio of their V scale
 * to a reference, are rounded to fp16 under 2^11: 11 bits of a weight down to
 * 2^-25 of the largest, 2^-36 of the largest below that. The reference is at
 * most 2^12 times the largest scale of 128 keys, or 2^-64 of the request's
 * largest. Sums and statistics are fp32. A NaN code reaches only the rows that
 * see its key. Results do not depend on the order in which blocks run. The
 * workspace may serve calls of any smaller shapes too.
 * A request whose lengths or rows of q do not fit is left out, a page index
 * outside the pages makes its keys invisible; both record
 * STAR_ERR_DEVICE_BOUNDS.
 */
star_status star_kv8_attend(const void* q, const int64_t q_stride[2], int n_tokens,
                            const int32_t* cu_new, const int32_t* kv_len, int B,
                            const int32_t* block_table, int max_pages, const void* k_pages,
                            const void* v_pages, const float* k_scale, const float* v_scale,
                            int num_pages, int page_len, int kv_type, int Hq, int Hkv, int D,
                            int max_new, int max_kv, void* o, float* lse, void* workspace,
                            size_t workspace_bytes, void* cuda_stream);

/*
 * star_device_status — synchronises `cuda_stream`, then reads the status
 * bits at the start of `workspace` (a workspace passed to any call; the bits
 * are sticky since the last read) and clears them. After a device error it
 * also clears the decode counters (the header size the last decode call
 * recorded in the status block), since an aborted call may leave them
 * non-zero. Returns STAR_OK, STAR_ERR_DEVICE_TIMEOUT or STAR_ERR_DEVICE_BOUNDS
 * (message in star_last_error), or STAR_ERR_CUDA.
 */
star_status star_device_status(void* workspace, void* cuda_stream);

/*
 * star_debug_wait_probe — checks the kernels' bounded waits and the status
 * read-back: one CTA waits, through the same bounded wait the attention and
 * decode kernels use, on a barrier nothing arrives on; after `seconds`
 * (0 < seconds <= 2) the wait gives up and records a time-out in the status
 * word at the start of `workspace` (>= 256 bytes, cleared first). A following
 * star_device_status returns STAR_ERR_DEVICE_TIMEOUT; nothing faults and the
 * context stays usable.
 */
star_status star_debug_wait_probe(void* workspace, double seconds, void* cuda_stream);

/*
 * star_debug_index — evaluates the kernels' index math on the device for
 * every context row r in [0, L): blk[r] = block id, pos[r] = position ID,
 * kv_ranges[4r..4r+3] = {anchor_lo, anchor_hi, own_lo, own_hi} (half-open;
 * block 0 reports an empty anchor range [0, 0)). Device int32 outputs.
 */
star_status star_debug_index(int L, int block_len, int anchor_len, int32_t* blk, int32_t* pos,
                             int32_t* kv_ranges, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* STAR_H_ */
