// Parameter blocks and launchers of the operators that serve a ragged batch
// from an 8-bit paged cache (internal to the library; the public surface is
// include/star.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "star_common.cuh"

namespace star {

constexpr int kMaxRequests = 4096;  // requests of one call: their offsets live in shared memory

#ifdef __CUDACC__
// atomicInc that orders the block's work before it (after a barrier) and what the
// thread does after it: one round trip to L2, where fences around it take another.
__device__ __forceinline__ unsigned inc_acq_rel(unsigned* p, unsigned limit) {
  unsigned old;
  asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(limit) : "memory");
  return old;
}
// The end of what was launched before on the stream (see launch_after).
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A bounded wait as mbar_wait, by the SM's clock: %globaltimer takes long to read, and
// a wait that is not over at once would read it first.
constexpr long long kWaitClocks = 4000000000ll;  // 2 s at 2 GHz
__device__ __forceinline__ bool mbar_wait_clocks(uint64_t* bar, uint32_t parity, volatile int* abort,
                                                 int* status, long long limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      if (clock64() - t0 > limit) {
        atomicOr(status, kDevTimeout);
        *abort = 1;
        return false;
      }
    }
  }
}

// Sums of tiles, which stop at INT32_MAX: the host bounds the tiles of offsets that ascend,
// but others may count tokens many times over. A call whose sum gets there is left out.
__device__ __forceinline__ int add_tiles(int a, int b) {
  return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), 0x7FFFFFFFu));
}
__device__ __forceinline__ int times_tiles(int heads, int tiles) {
  return static_cast<int>(min(static_cast<long long>(heads) * tiles, 0x7FFFFFFFll));
}
constexpr int kTooManyTiles = 0x7FFFFFFF;

// Where the attention kernels' reference of V scales goes when vs, the largest scale at
// hand, is above it or 2^12 below it: to vs, but no further than 2^64 below top, the
// largest so far. O is held in units of the reference: at most 2^24 for each of 2^31
// keys times 2^64, it stays finite whatever scales follow one another (star_kv8_append
// gives a page of zeros 2^-100).
__device__ __forceinline__ float next_reference(float vs, float top) {
  return fmaxf(vs, top * 5.421010862427522e-20f);
}
#endif

// Launches a kernel whose threads all begin with after_previous(): it is set up while
// the one before it ends, which takes 2 us off a call that follows another (501
// tokens of one head: 7.4 us instead of 9.4).
template <typename Params>
inline cudaError_t launch_after(void (*kernel)(const Params), dim3 grid, int threads, size_t smem,
                                cudaStream_t stream, const Params& p) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// ---- rotary with given frequencies --------------------------------------------
struct RopeScaledParams {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;
  long long xs[3], ys[3];  // element strides of (B, S, H)
  const int32_t* pos;      // nullable
  long long pos_stride_b, pos0;
  int B, S, H, D, rot;
  int tpc, hpc;            // tokens and heads of one CTA
  int copy_rest;           // 1: elements from rot on are copied (not in place)
  float mscale_abs;
  double mscale, sign;     // sign -1: transposed rotation
  double inv_freq[64];
};
cudaError_t launch_rope_scaled(const RopeScaledParams& p, bool interleaved, cudaStream_t stream);

// ---- batch plan -----------------------------------------------------------------
struct BatchPlanParams {
  const int32_t *ctx_len, *new_len, *free_pages, *free_begin;
  int32_t *table, *cu_new, *pos, *slot, *run_start, *kv_len, *free_next;
  int B, num_free, page_shift, max_pages, n_cap, run_cap;
  int* status;        // status word
  unsigned* ticket;   // finished CTAs; zero between calls
};
cudaError_t launch_batch_plan(const BatchPlanParams& p, cudaStream_t stream);

// ---- append -----------------------------------------------------------------------
struct Kv8AppendParams {
  const __nv_bfloat16 *k, *v;
  long long ks[2], vs[2];  // element strides of (token, head)
  const int32_t *slot, *run_start;
  uint8_t *k_pages, *v_pages;
  float *k_scale, *v_scale;
  int n_tokens, Hkv, run_cap, num_pages, page_shift;
  int* status;
};
cudaError_t launch_kv8_append(const Kv8AppendParams& p, int D, int kv_type, cudaStream_t stream);

// ---- attention ----------------------------------------------------------------------
struct Kv8AttendParams {
  const __nv_bfloat16* q;
  long long qs[2];  // element strides of (token, head)
  const int32_t *cu_new, *kv_len, *table;
  const uint8_t *k_pages, *v_pages;
  const float *k_scale, *v_scale;
  __nv_bfloat16* o;
  float* lse;
  int n_tokens, B, Hq, Hkv, g, max_pages, num_pages, page_shift, max_new, max_kv;
  float scale_log2;     // log2(e) / sqrt(D)
  int* status;          // status word; status[1] receives header_bytes
  int header_bytes;     // workspace bytes holding the status block and the counters
  unsigned* counters;   // [kKv8MaxCtas] finished parts of the unit that is cut at a CTA's end
  float* part_ml;       // [CTAs][2][rows][2] maximum (log2 units) and sum of a part
  float* part_o;        // [CTAs][2][rows][D] ([D / 4][rows][4] of the chunk kernel)
};
constexpr int kKv8Tile = 128;     // keys of one tile of a CTA
// Sums that are joined, of weights and of weighted values, are held times 2^-20: P is up
// to 2^15, and 2^15 times values near the largest number do not fit fp32 where their
// average does. (The weights' sum is at least 2^-20 then, and usually 2^-9.)
constexpr float kKv8JoinShift = 20.f, kKv8Join = 9.5367431640625e-07f;
constexpr int kKv8MaxCtas = 512;  // the workspace holds parts for this many (decode)
constexpr int kKv8ChunkRows = 256, kKv8ChunkMaxCtas = 160;
// Rows of a (request, KV head) tile: 8 or 16 of the decode kernel, or the chunk
// kernel's. Up to 32 rows two decode tiles read the pages twice and still win: 20
// rows over 128K keys of 8 heads take 133 us against 168, over 2000 keys 16.5 against
// 21.4. At 40 rows three tiles take 190 us against 168 (16 ragged requests up to 16K:
// 254 against 188). None of these is near its bytes, 41 us over 128K keys: 8 rows take
// 55 us, 16 rows 77.
inline int kv8_rows(int max_new, int g) {
  const long long rows = (long long)max_new * g;
  return rows <= 8 ? 8 : rows <= 32 ? 16 : kKv8ChunkRows;
}
// A call of more rows stays on the decode kernel while it has at most this many
// tiles of 16 rows by 128 keys, since the chunk kernel needs 15 us before its first
// product: 240 rows on 3000 keys of D 64 (360 tiles) 17 us against 27, 200 rows of 8
// heads on 1000 keys (832) 22 against 26; 40 rows of 16 requests, 8 heads on 500 keys
// (1536) 36 against 37, 1024 rows of 8 heads on 600 keys (2560) 48 against 36.
constexpr int kKv8FewTiles = 1024;
cudaError_t launch_kv8_decode(const Kv8AttendParams& p, int D, int kv_type, int rows, int sms,
                              cudaStream_t stream);
cudaError_t launch_kv8_chunk(const Kv8AttendParams& p, int D, int kv_type, int sms, cudaStream_t stream);

}  // namespace star
