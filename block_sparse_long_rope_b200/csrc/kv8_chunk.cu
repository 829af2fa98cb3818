// Attention of many new tokens of a request (a query chunk, a prompt's next
// piece) over its 8-bit pages, on the 5th-generation tensor cores.
//
// The mathematics is kv8_decode.cu's: s = ks_j (q . K) / sqrt(D), o = sum
// e^(s - m) vs_j V / sum e^(s - m), token t of T seeing kv - T + t + 1 keys.
// Bound: the exponential unit and the tensor cores, about equally (256 x 128
// scores are 2048 cycles of either); what it spends now is the chain of one slot,
// score products, softmax, weight products, about 5000 cycles a tile for both
// slots out of step. 256 tokens of 64 heads after 128K keys of 8 heads (1.1
// TFLOP): 1315 us, 837 TFLOP/s (1410 to 1430 where every call has new inputs); in int8
// 1330, at D 64 1395 (e4m3) and 1368 (int8). <128, e4m3> spills 118 bytes of stores and
// 184 of loads a thread, int8 40 and 120: the rest is the way out with NaN codes.
//  * The T * g (token, query head) rows of a (request, KV head) are cut into
//    tiles of 256 rows, two slots of 128: a K or V tile of 128 keys is read and
//    converted once for both.
//  * Work is cut by (row tile, key tile) as in kv8_decode.cu: CTA c of G owns an
//    equal contiguous range of the list, whatever the lengths; a row tile's key
//    tiles end with its last row's limit. Parts of cut units go to the workspace,
//    and a second kernel joins them in order.
//  * Four warps read codes with 16-byte loads, a tile ahead, and write them as
//    fp16 (exact) in the 128-byte-swizzled layout that tcgen05.mma reads; K and V
//    have the same layout. q is fp16 times a power of two per row, which keeps
//    all its bits for elements down to 2^-29 of the row's largest.
//  * Eight warps own a slot: two threads for each row (lane of tensor memory), 64
//    keys of a tile each. One warp issues a slot's products, PV(n) then S(n+1),
//    the second slot's after the first's, so that a slot's softmax runs beside
//    the other's products (in step, both slots contend for the exponential unit:
//    1600 us). P (fp16) overwrites half of its S and feeds the P V product from
//    tensor memory.
//  * The roles' code competes for the instruction caches: a second copy of the
//    softmax step for tiles whose V scales are equal, with a multiplication less,
//    cost 70 us.
//  * P is rounded to fp16 under 2^11 as in kv8_decode.cu, the running maximum
//    moves when it grows by more than 2^4, and V scales enter through P as the
//    ratio to a running reference that stays within [1, 2^12) of the tile's
//    largest, or 2^64 below the largest so far (see next_reference). Values whose
//    scale is 2^24 below the largest of their 128 keys lose bits.
#include <math.h>

#include "kv8_codes.cuh"
#include "kv8_kernels.cuh"
#include "star_kernels.cuh"

namespace star {

namespace {

// Warps 0-15: softmax (slot = warp / 8, half of the keys = warp / 4 % 2), 16-19:
// converters, 20 and 21: MMA (+ 2 idle).
constexpr int kThreads = 768;
constexpr int kJoinThreads = 256;
constexpr int kRows = kKv8ChunkRows;
constexpr int kRing = 8;       // tiles whose scales are kept: more than the stages ahead
constexpr float kShift = 11.f; // P is held as 2^11 e^(s - m)
constexpr float kSlack = 4.f;  // growth of the maximum (log2) before it moves
// s_j f - rf in one rounding may lie half a step of the maximum above what the rounded
// maximum allows, or below: 2^-9 up to here, but 16 at 2^28, where P leaves fp16. Rows
// beyond it round s_j f first, as the maximum's product was (for all rows that costs
// 80 us of 1410).
constexpr float kFar = 65536.f;

template <int D>
struct Cfg {
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kHalf = 128 * 128;         // 64 fp16 columns of 128 rows
  static constexpr int kTile = kHalf * (D / 64);
  static constexpr int kOffK = 2 * kTile;         // after the two Q tiles
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffPrefix = kOffV + kStages * kTile;
  static constexpr size_t bytes(int B) { return 1024 + kOffPrefix + (B + 1) * sizeof(int); }
};

// What the roles need of a request; a bad one has no rows.
struct Request {
  int q0, T, kv, row_tiles;
};
__device__ __forceinline__ Request request_of(const Kv8AttendParams& p, int b, bool* bad) {
  Request r;
  const int c0 = p.cu_new[b], c1 = p.cu_new[b + 1];
  r.q0 = c0;
  r.T = c1 - c0;
  r.kv = p.kv_len[b];
  *bad = c0 < 0 || c1 < c0 || c1 > p.n_tokens || r.T > p.max_new || r.kv < 0 || r.kv > p.max_kv;
  if (*bad) r.T = 0;
  r.row_tiles = ceil_div(r.T * p.g, kRows);
  return r;
}
// Row tile rt of a request: its rows, and the keys that its first and last row see.
__device__ __forceinline__ int rows_of(const Kv8AttendParams& p, const Request& r, int rt) {
  return imin(kRows, r.T * p.g - rt * kRows);
}
__device__ __forceinline__ int keys_of_row(const Kv8AttendParams& p, const Request& r, int row) {
  return r.kv - r.T + 1 + row / p.g;
}
__device__ __forceinline__ int tiles_of(const Kv8AttendParams& p, const Request& r, int rt) {
  return imax(1, ceil_div(keys_of_row(p, r, rt * kRows + rows_of(p, r, rt) - 1), kKv8Tile));
}

// The part of the tile list that a CTA walks, unit by unit.
struct Walk {
  int b, kvh, rt, tile, tiles;
  Request r;
};
__device__ __forceinline__ Walk walk_to(const Kv8AttendParams& p, const int* prefix, int at) {
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= at) lo = mid;
    else hi = mid;
  }
  Walk w;
  bool bad;
  w.b = lo;
  w.r = request_of(p, lo, &bad);
  const int per_head = (prefix[lo + 1] - prefix[lo]) / p.Hkv;
  w.kvh = (at - prefix[lo]) / per_head;
  w.tile = (at - prefix[lo]) - w.kvh * per_head;
  w.rt = 0;
  for (w.tiles = tiles_of(p, w.r, 0); w.tile >= w.tiles; w.tiles = tiles_of(p, w.r, w.rt)) {
    w.tile -= w.tiles;
    ++w.rt;
  }
  return w;
}
// To the first tile of the next unit, whose list index is next.
__device__ __forceinline__ void next_unit(const Kv8AttendParams& p, const int* prefix, Walk& w, int next) {
  w.tile = 0;
  if (++w.rt == w.r.row_tiles) {
    w.rt = 0;
    if (++w.kvh == p.Hkv) {
      w.kvh = 0;
      bool bad;
      do ++w.b;
      while (prefix[w.b + 1] <= next);  // requests without work
      w.r = request_of(p, w.b, &bad);
    }
  }
  w.tiles = tiles_of(p, w.r, w.rt);
}

// prefix[b]: tiles before request b (by all of a block's threads); true to a lane
// that met a bad request.
__device__ __forceinline__ bool tiles_before(const Kv8AttendParams& p, int* prefix, int threads) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool any_bad = false;
  for (int b = warp; b < p.B; b += threads / 32) {
    bool bad;
    const Request r = request_of(p, b, &bad);
    any_bad |= bad;
    int sum = 0;
    for (int rt = lane; rt < r.row_tiles; rt += 32) sum = add_tiles(sum, tiles_of(p, r, rt));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum = add_tiles(sum, __shfl_xor_sync(0xffffffffu, sum, d));
    if (lane == 0) prefix[b + 1] = times_tiles(p.Hkv, sum);
  }
  __syncthreads();
  if (warp == 0) {
    int base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      int v = b0 + lane < p.B ? prefix[b0 + lane + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v = add_tiles(v, up);
      }
      if (b0 + lane < p.B) prefix[b0 + lane + 1] = add_tiles(base, v);
      base = add_tiles(base, __shfl_sync(0xffffffffu, v, 31));
    }
    if (lane == 0) prefix[0] = 0;
  }
  return any_bad;
}

struct Scales {
  float k[8], v[8];  // of the 8 groups of 16 keys; k < 0: no such page
  int nan[4];        // by converter warp: a V code at the causal edge is NaN
  int flags[4];      // [0]: kFirst, kLast (tile of a segment), kTwo (both slots have rows)
};

enum { kFirst = 1, kLast = 2, kTwo = 4 };

// D[tmem] (+)= A B with A in shared memory or tensor memory: the descriptors'
// lower words differ from product to product, the upper word is one constant.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // SBO 1024, version, SWIZZLE_128B
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ void mma_ss_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHi)
      : "memory");
}

// Instruction descriptor of tcgen05.mma kind::f16 with fp16 A and B, fp32 D.
constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Arrival of a warp, its lanes' writes before it.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return mbar_wait_clocks(bar, parity, abort, status, kWaitClocks);
}
// A wait that lasts while the count moves: its limit starts again with every step seen.
__device__ __forceinline__ bool wait_moving(uint64_t* bar, uint32_t parity, volatile int* abort, volatile int* count,
                                         int* status) {
  int seen = *count;
  long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (*abort) return false;
      const int now = *count;
      if (now != seen) {
        seen = now;
        t0 = clock64();
      }
      if (clock64() - t0 > kWaitClocks) {
        atomicOr(status, kDevTimeout);
        *abort = 1;
        return false;
      }
    }
  }
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// One answer for the whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return __all_sync(0xffffffffu, wait(bar, parity, abort, status));
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 0xff in each byte of four e4m3 codes that is NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

// 32 columns of this thread's lane, there when it returns: a load that ends
// later could meet the compiler's own copies of its registers.
__device__ __forceinline__ void tmem_ld32_now(uint32_t taddr, uint32_t (&s)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3]), "=r"(s[4]), "=r"(s[5]),
        "=r"(s[6]), "=r"(s[7]), "=r"(s[8]), "=r"(s[9]), "=r"(s[10]), "=r"(s[11]),
        "=r"(s[12]), "=r"(s[13]), "=r"(s[14]), "=r"(s[15]), "=r"(s[16]), "=r"(s[17]),
        "=r"(s[18]), "=r"(s[19]), "=r"(s[20]), "=r"(s[21]), "=r"(s[22]), "=r"(s[23]),
        "=r"(s[24]), "=r"(s[25]), "=r"(s[26]), "=r"(s[27]), "=r"(s[28]), "=r"(s[29]),
        "=r"(s[30]), "=r"(s[31])
      : "r"(taddr)
      : "memory");
}

// Steps of the softmax over 32 of a row's scores s. Score j in log2 units is
// s_j f, f = fs ks for the two groups of 16 keys.
// At an edge, or beyond kFar: scaled scores, with -inf for keys from `seen` on and for
// those of missing pages (ks < 0); f is 1 from then on.
__device__ __forceinline__ void mask_32(uint32_t (&s)[32], const float* ks, float fs, int seen) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float k = ks[j >> 4], v = __uint_as_float(s[j]) * (fs * k);
    s[j] = j < seen && !(k < 0.f) ? __float_as_uint(v) : 0xFF800000u;
  }
}
__device__ __forceinline__ float max_32(const uint32_t (&s)[32], float f0, float f1) {
  float m[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const uint32_t* v = s + 16 * g;
    float a = fmax3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
    float b = fmax3(__uint_as_float(v[3]), __uint_as_float(v[4]), __uint_as_float(v[5]));
#pragma unroll
    for (int j = 6; j < 14; j += 4) {
      a = fmax3(a, __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
      b = fmax3(b, __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
    }
    m[g] = fmax3(a, b, fmaxf(__uint_as_float(v[14]), __uint_as_float(v[15])));
  }
  return fmaxf(m[0] * f0, m[1] * f1);
}
// P = 2^(s f - rf) times the ratio of the V scale to its reference, as fp16
// pairs to tensor memory; ls receives the sums of 2^(s f - rf).
__device__ __forceinline__ void p_32(const uint32_t (&s)[32], float f0, float f1, float r0, float r1,
                                     uint64_t nref, uint64_t (&ls)[2], uint32_t dst) {
  uint32_t pk[16];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const float f = g ? f1 : f0, r = g ? r1 : r0;
    const uint64_t ff = f2_pack(f, f), rr = f2_pack(r, r);
#pragma unroll
    for (int j = 8 * g; j < 8 * g + 8; ++j) {
      float x0, x1;
      f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), ff, nref), x0, x1);
      const uint64_t e = f2_pack(ex2_approx(x0), ex2_approx(x1));
      ls[j & 1] = f2_add(ls[j & 1], e);
      f2_unpack(f2_mul(e, rr), x0, x1);
      pk[j] = half2_of(x0, x1);
    }
  }
  tmem_st16(dst, pk);
}

// Bit d of the result: a NaN code in column 32 * part + d of the V rows of keys
// [key0, key1) (the rare path of a NaN at the causal edge).
template <int D>
__device__ __noinline__ uint32_t nan_columns(const Kv8AttendParams& p, int b, int kvh, int key0,
                                             int key1, int part) {
  uint32_t bits = 0;
  for (int key = key0; key < key1; ++key) {
    const int page = p.table[static_cast<size_t>(b) * p.max_pages + (key >> p.page_shift)];
    if (page < 0 || page >= p.num_pages) continue;
    const size_t row = ((static_cast<size_t>(page) * p.Hkv + kvh) << p.page_shift) +
                       (key & ((1 << p.page_shift) - 1));
    const uint32_t* v = reinterpret_cast<const uint32_t*>(p.v_pages + row * D + 32 * part);
    for (int i = 0; i < 8; ++i) {
      const uint32_t n = nan_bytes(v[i]);
      for (int c = 0; c < 4; ++c) bits |= ((n >> (8 * c)) & 1u) << (4 * i + c);
    }
  }
  return bits;
}

}  // namespace

template <int D, int kType>
__global__ void __launch_bounds__(kThreads, 1) kv8_chunk_kernel(const __grid_constant__ Kv8AttendParams p) {
  using C = Cfg<D>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  int* prefix = reinterpret_cast<int*>(sm + C::kOffPrefix);  // [B + 1] tiles before request b
  __shared__ uint64_t q_full[2], s_full[2], p_full[2], o_full[2], done[2];
  __shared__ uint64_t k_full[S], v_full[S], empty[S], sc_full[kRing], nan_full[kRing], lead[kRing];
  __shared__ __align__(16) Scales ring[kRing];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag, mma_step;  // mma_step: the second slot's MMA warp moves
  // what a row's two threads exchange
  __shared__ float row_l[2][2][128], row_m[2][2][2][128];
  __shared__ uint32_t row_q[2][2][128];
  __shared__ float v_top[512];  // largest V scale so far, by softmax thread (a register more spills)

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  after_previous();
  // the join may be launched where there is room: it waits for this kernel's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  {
    const bool any_bad = tiles_before(p, prefix, kThreads);
    if (any_bad && lane == 0 && blockIdx.x == 0) atomicOr(p.status, kDevBounds);
    if (tid == 0 && blockIdx.x == 0) p.status[1] = p.header_bytes;
    if (tid == 0) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(&q_full[x], 8);  // (by warp)
        mbar_init(&s_full[x], 1);
        mbar_init(&p_full[x], 8);
        mbar_init(&o_full[x], 1);
        mbar_init(&done[x], 1);
      }
      for (int s = 0; s < S; ++s) {
        mbar_init(&k_full[s], 4);
        mbar_init(&v_full[s], 4);
        mbar_init(&empty[s], 2);  // V of a tile and K of the next are free
      }
      for (int s = 0; s < kRing; ++s) {
        mbar_init(&sc_full[s], 4);
        mbar_init(&nan_full[s], 4);
        mbar_init(&lead[s], 1);
      }
      fence_barrier_init();
      abort_flag = mma_step = 0;
    }
    __syncthreads();
  }
  const int total = prefix[p.B];
  if (total == kTooManyTiles) {
    if (blockIdx.x == 0 && tid == 0) atomicOr(p.status, kDevBounds);
    return;
  }
  const int G = imin(static_cast<int>(gridDim.x), total);  // CTAs with work
  if (static_cast<int>(blockIdx.x) >= G) return;
  const int begin = static_cast<int>(static_cast<long long>(blockIdx.x) * total / G);
  const int end = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * total / G);
  const int N = end - begin;

  if (warp == 20) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp >= 20) {
    // ------------------------------------------------------------ MMA issuer
    // a warp for each slot: what one does between its products runs beside the other's
    regs_down<56>();
    const int x = warp - 20;
    if (x < 2 && lane == 0) {
      constexpr uint32_t idS = idesc_f16(128, 128, 0);  // S = Q K^T, both K-major
      constexpr uint32_t idO = idesc_f16(128, D, 1);    // O += P V, V is N-major
      const uint32_t q_lo = desc_lo(smem_u32(sm) + x * C::kTile, 16), k_lo = desc_lo(smem_u32(sm) + C::kOffK, 16);
      const uint32_t v_lo = desc_lo(smem_u32(sm) + C::kOffV, C::kHalf);
      const uint32_t tS = tmem + 128 * x, tO = tmem + 256 + 128 * x;
      // K-major operands: 16 columns are 32 bytes, 64 columns a half tile
      auto issue_s = [&](int st) {
        const uint32_t b = k_lo + st * (C::kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t at = ((kk >> 2) * C::kHalf + (kk & 3) * 32) >> 4;
          mma_ss_lo(tS, q_lo + at, b + at, idS, kk > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[x]);
      };
      uint32_t cnt = 0, segs = 0;  // tiles and segments of this slot so far
      int now = 0;                 // no tile before the first
      for (int n = -1; n < N; ++n) {
        if (x == 1) mma_step = n;
        // products of a step: PV(n), S(n + 1)
        int next = 0;
        if (n + 1 < N) {
          if (!wait(&k_full[(n + 1) % S], ((n + 1) / S) & 1, &abort_flag, p.status)) break;
          next = ring[(n + 1) % kRing].flags[0];
        }
        // slot 1's products come after slot 0's of the same step: one slot's softmax
        // then runs beside the other's products, and not beside its softmax
        const bool has_pv = n >= 0 && (x == 0 || (now & kTwo)), has_s = n + 1 < N && (x == 0 || (next & kTwo));
        if (has_pv) {
          if (!wait(&v_full[n % S], (n / S) & 1, &abort_flag, p.status)) break;
          if (!wait(&p_full[x], cnt & 1, &abort_flag, p.status)) break;
          ++cnt;
          if (x == 1 && !wait(&lead[(n + 1) % kRing], ((n + 1) / kRing) & 1, &abort_flag, p.status)) break;
          tc_fence_after();
          const uint32_t b = v_lo + (n % S) * (C::kTile >> 4);
          // each half's P lies in the upper half of its 64 columns of S, its second 32
          // keys first
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts_lo(tO, tS + 64 * (kk >> 2) + ((kk & 2) ? 16 : 48) + 8 * (kk & 3), b + kk * (2048 >> 4), idO,
                      (!(now & kFirst) || kk > 0) ? 1u : 0u);
          if (now & kLast) mma_commit(&o_full[x]);
        }
        if (has_s) {
          if (next & kFirst) {
            if (!wait(&q_full[x], segs & 1, &abort_flag, p.status)) break;
            ++segs;
          }
          if (x == 1 && !wait(&lead[(n + 1) % kRing], ((n + 1) / kRing) & 1, &abort_flag, p.status)) break;
          tc_fence_after();
          issue_s((n + 1) % S);
        }
        if (x == 0) mbar_arrive(&lead[(n + 1) % kRing]);
        // both slots' arrivals free V(n) and K(n + 1). (A slot without rows keeps
        // in step by its waits for K; nobody waits for the last step.)
        if (n + 1 < N) {
          if (has_pv || has_s) mma_commit(&empty[(n + 1) % S]);
          else mbar_arrive(&empty[(n + 1) % S]);
        }
        now = next;
      }
      // every MMA in flight ends before tensor memory is released
      mma_commit(&done[x]);
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(&done[x], 0))
        if (global_ns() - t0 > 100000000ull) break;
    }
    __syncwarp();
  } else if (warp >= 16) {
    // ------------------------------------------------------------ converters
    regs_up<104>();  // with the MMA warps' 56: what the block was launched with
    constexpr int kLoads = D / 16;      // 16-byte loads of a thread for a K or V tile
    constexpr int kPerRow = D / 16;     // 16-byte pieces of a row
    constexpr int kRowsPer = 32 / kPerRow;
    // At D 128 eight lanes cover a row's 128 bytes and write two 64-column halves,
    // which lie in the same banks: the second half's lanes take the next row, whose
    // chunks the swizzle puts elsewhere
    const int cw = warp - 16, ch = lane % kPerRow, rl = (lane / kPerRow) ^ (ch >> 2), r0 = 32 * cw + rl;
    const int P = 1 << p.page_shift;
    struct Tile {
      int key0, left, kvh, edge, flags, page[2];  // pages of this warp's two groups of 16 keys
    };
    Walk w = walk_to(p, prefix, begin);
    auto real = [&](int page) { return page >= 0 && page < p.num_pages; };
    auto fetch = [&](int n) {
      Tile t;
      t.flags = (n == 0 || w.tile == 0 ? kFirst : 0) | (n + 1 == N || w.tile + 1 == w.tiles ? kLast : 0) |
                (rows_of(p, w.r, w.rt) > 128 ? kTwo : 0);
      t.key0 = w.tile * kKv8Tile + 32 * cw;
      t.left = w.r.kv - t.key0;  // keys from this warp's first one on
      t.kvh = w.kvh;
      t.edge = w.tile * kKv8Tile + kKv8Tile > keys_of_row(p, w.r, w.rt * kRows);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        t.page[i] = 16 * i < t.left
                        ? p.table[static_cast<size_t>(w.b) * p.max_pages + ((t.key0 + 16 * i) >> p.page_shift)]
                        : 0;
      return t;
    };
    auto step = [&](int n) {  // to tile n of this CTA
      if (w.tile + 1 < w.tiles) ++w.tile;
      else next_unit(p, prefix, w, begin + n);
    };
    // this lane's first 16 codes of a group of 16 keys
    auto start = [&](const Tile& t, int i) -> size_t {
      const size_t row = ((static_cast<size_t>(t.page[i]) * p.Hkv + t.kvh) << p.page_shift) +
                         ((t.key0 + 16 * i) & (P - 1));
      return (row + rl) * D + 16 * ch;
    };
    auto load = [&](uint4 (&x)[kLoads], const Tile& t, const uint8_t* pages) {
      if (t.left >= 32 && real(t.page[0]) && real(t.page[1])) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4* src = reinterpret_cast<const uint4*>(pages + start(t, i));
#pragma unroll
          for (int j = 0; j < kLoads / 2; ++j) x[i * (kLoads / 2) + j] = __ldg(src + j * kRowsPer * (D / 16));
        }
        return;
      }
      // keys behind the last one, and those of missing pages, are zero codes
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int i = j / (kLoads / 2), r = rl + kRowsPer * j;
        x[j] = make_uint4(0u, 0u, 0u, 0u);
        if (r < t.left && real(t.page[i]))
          x[j] = __ldg(reinterpret_cast<const uint4*>(pages + start(t, i)) +
                       (j - i * (kLoads / 2)) * kRowsPer * (D / 16));
      }
    };
    // lanes 0, 1: K scales of the warp's groups; lanes 2, 3: V scales
    auto load_scale = [&](const Tile& t) -> float {
      if (lane >= 4) return 0.f;
      const int page = lane & 1 ? t.page[1] : t.page[0];
      if (!real(page)) {
        atomicOr(p.status, kDevBounds);
        return lane < 2 ? -1.f : 0.f;
      }
      if (16 * (lane & 1) >= t.left) return 0.f;
      return __ldg((lane < 2 ? p.k_scale : p.v_scale) + static_cast<size_t>(page) * p.Hkv + t.kvh);
    };
    // Columns 16 ch .. + 15 of a row are two chunks of a 64-column half. Rows of a
    // thread are 4 apart (8 at D 64), so the swizzle takes two values (one).
    uint32_t at[2][2];
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        at[o][c] = (ch >> 2) * C::kHalf + sw128_offset(r0 + kRowsPer * o, ((2 * ch) & 7) + c) - 128 * kRowsPer * o;
    auto convert = [&](const uint4 (&x)[kLoads], uint8_t* dst) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        uint4 a, b;
        codes_to_half2<kType>(x[j].x, a.x, a.y);
        codes_to_half2<kType>(x[j].y, a.z, a.w);
        codes_to_half2<kType>(x[j].z, b.x, b.y);
        codes_to_half2<kType>(x[j].w, b.z, b.w);
        *reinterpret_cast<uint4*>(dst + at[j & 1][0] + 128 * kRowsPer * j) = a;
        *reinterpret_cast<uint4*>(dst + at[j & 1][1] + 128 * kRowsPer * j) = b;
      }
    };
    uint4 kx[kLoads], vx[kLoads];
    Tile cur = fetch(0), nxt = cur;
    load(kx, cur, p.k_pages);
    load(vx, cur, p.v_pages);
    float sc = load_scale(cur);
    if (N > 1) {
      step(1);
      nxt = fetch(1);
    }
    for (int n = 0; n < N; ++n) {
      const int st = n % S;
      // the scales' ring is deeper than the stages ahead: no wait
      Scales& ss = ring[n % kRing];
      if (n >= S && !warp_wait(&empty[st], (n / S - 1) & 1, &abort_flag, p.status)) break;
      if (lane < 2) ss.k[2 * cw + lane] = sc;
      else if (lane < 4) ss.v[2 * cw + lane - 2] = sc;
      else if (lane == 4) ss.nan[cw] = 0;
      else if (cw == 0 && lane == 5) ss.flags[0] = cur.flags;
      warp_arrive(&sc_full[n % kRing]);
      convert(kx, sm + C::kOffK + st * C::kTile);
      fence_async_shared();
      warp_arrive(&k_full[st]);
      if (n + 1 < N) {
        load(kx, nxt, p.k_pages);
        sc = load_scale(nxt);
      }
      if (n >= S && !warp_wait(&empty[(n + 1) % S], ((n + 1) / S - 1) & 1, &abort_flag, p.status)) break;
      if (kType == STAR_KV8_E4M3 && cur.edge) {
        // a NaN must not meet the weight 0 of rows that do not see its key: it
        // goes in as 0 and the rows that see it are told
        uint32_t any = 0;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          uint32_t* v = reinterpret_cast<uint32_t*>(&vx[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t nan = nan_bytes(v[i]);
            any |= nan;
            v[i] &= ~nan;
          }
        }
        if (any) ss.nan[cw] = 1;
        warp_arrive(&nan_full[n % kRing]);
      } else if (lane == 0) {
        mbar_arrive(&nan_full[n % kRing]);
      }
      convert(vx, sm + C::kOffV + st * C::kTile);
      fence_async_shared();
      warp_arrive(&v_full[st]);
      cur = nxt;
      if (n + 1 < N) load(vx, nxt, p.v_pages);
      if (n + 2 < N) {
        step(n + 2);
        nxt = fetch(n + 2);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    // Two threads a row: each takes 64 of a tile's 128 keys and half of O. They meet
    // at a named barrier of their two warps; nobody leaves the loops early (an
    // abort only makes the waits short), so every barrier is met by both.
    const int x = warp >> 3, half = (warp >> 2) & 1, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + 128 * x + 64 * half, tO = tmem + lanes + 256 + 128 * x;
    const int pair = 1 + 4 * x + (warp & 3);
    auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory"); };
    uint32_t cnt = 0, segs = 0;
    bool ok = true;
    float next_fs = 0.f;
    // a row of q into the slot's tile, as fp16 times a power of two: half of it by
    // each of its threads
    auto load_q = [&](const Walk& w) {
      if (x == 1 && rows_of(p, w.r, w.rt) <= 128) return;
      const int r = w.rt * kRows + 128 * x + row;
      uint8_t* dst = sm + x * C::kTile;
      uint4 v[D / 16];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < w.r.T * p.g) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (w.r.q0 + r / p.g) * p.qs[0] +
                                                          (w.kvh * p.g + r % p.g) * p.qs[1]) + half * (D / 16);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) v[i] = __ldg(src + i);
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                     __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu)));
      row_q[x][half][row] = top;
      pair_sync();
      top = __vmaxu2(top, row_q[x][half ^ 1][row]);
      const int e = static_cast<int>(imax(top & 0xFFFFu, top >> 16) >> 7);  // biased exponent
      const int up = imin(237, 127 + 14 - (e - 127));  // 2^(14 - (e - 127)), at most 2^110 (kv8_decode.cu)
      const float mul = __uint_as_float(static_cast<uint32_t>(up) << 23);
      // this row's factor: 2^-e log2(e) / sqrt(D)
      next_fs = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
      auto two = [&](uint32_t u) { return half2_of(bf16_lo(u) * mul, bf16_hi(u) * mul); };
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const int i = half * (D / 16) + j;
        *reinterpret_cast<uint4*>(dst + (i >> 3) * C::kHalf + sw128_offset(row, i & 7)) =
            make_uint4(two(v[j].x), two(v[j].y), two(v[j].z), two(v[j].w));
      }
      fence_async_shared();
      warp_arrive(&q_full[x]);
    };
    Walk w = walk_to(p, prefix, begin);
    load_q(w);
    for (int n0 = 0; n0 < N;) {
      // ---- one segment: the tiles of one unit that this CTA holds
      const Walk here = w;
      const int seg = imin(here.tiles - here.tile, N - n0);
      const int rows = rows_of(p, here.r, here.rt);
      const bool active = x == 0 || rows > 128;
      const int my_row = here.rt * kRows + 128 * x + row;
      const int limit = keys_of_row(p, here.r, my_row);
      // keys that the slot's and the unit's first rows see; the former's tiles need no
      // mask (0 once a row is beyond kFar: none do without)
      int lim_lo = keys_of_row(p, here.r, here.rt * kRows + 128 * x);
      const int unit_lo = keys_of_row(p, here.r, here.rt * kRows);
      float m = -INFINITY, rf = 0.f, l = 0.f, vref = 0.f, ivref = 0.f, fs = next_fs;
      bool nan = false;
      // A slot without rows skips the tiles: nobody would hold the ring for it. Rounds of
      // the ring may have passed since its last tile, and a wait by parity takes only
      // one for its own, so a segment begins with the wait for its first scores: they
      // are there after the tile's scales, and no later round is until P answers them.
      // The skipped tiles may take longer than a wait may, so its limit starts again
      // whenever the slot's MMA warp has moved.
      if (active) ok &= __all_sync(0xffffffffu, wait_moving(&s_full[x], cnt & 1, &abort_flag, &mma_step, p.status));
      if (active)  // (a loop of its own: with the test in its condition the kernel takes 2% longer)
#pragma unroll 1
      for (int i = 0; i < seg; ++i) {
        const int n = n0 + i;
        const Scales& ss = ring[n % kRing];
        ok &= warp_wait(&sc_full[n % kRing], (n / kRing) & 1, &abort_flag, p.status);
        const int key0 = (here.tile + i) * kKv8Tile, seen = limit - key0 - 64 * half;
        float kmin = ss.k[0], vmax = ss.v[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) {
          kmin = fminf(kmin, ss.k[j]);
          vmax = fmaxf(vmax, ss.v[j]);
        }
        bool masked = key0 + kKv8Tile > lim_lo || kmin < 0.f;
        const bool new_vref = vmax > vref || (vmax < vref * 0.000244140625f && vmax > 0.f);
        const float *ks = ss.k + 4 * half, *vs = ss.v + 4 * half;
        auto factor = [&](int g) { return masked ? 1.f : fs * ks[g]; };

        ok &= warp_wait(&s_full[x], cnt & 1, &abort_flag, p.status);
        tc_fence_after();
        // ---- row maximum in log2 units, 32 scores at a time (loops that are not unrolled:
        // the roles share small instruction caches; scores that stay in registers until
        // P would spill others)
        uint32_t s[32];
        float mt = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          tmem_ld32_now(tS + 32 * q, s);
          if (masked) mask_32(s, ks + 2 * q, fs, seen - 32 * q);
          mt = fmaxf(mt, max_32(s, factor(2 * q), factor(2 * q + 1)));
        }
        row_m[cnt & 1][x][half][row] = mt;
        pair_sync();
        mt = fmaxf(mt, row_m[cnt & 1][x][half ^ 1][row]);
        ++cnt;
        if (kType == STAR_KV8_E4M3 && key0 + kKv8Tile > unit_lo) {
          ok &= warp_wait(&nan_full[n % kRing], (n / kRing) & 1, &abort_flag, p.status);
          const int4 flags = *reinterpret_cast<const int4*>(ss.nan);
          nan |= (flags.x | flags.y | flags.z | flags.w) != 0;
        }
        // ---- now and then the maximum and the V reference move; O and the sum follow
        const bool up = mt > __fadd_rd(m, kSlack);  // (rounded up, a step of 8 would pass)
        if (new_vref || __any_sync(0xffffffffu, up)) {
          float alpha = 1.f;
          if (up) {
            const bool none = m == -INFINITY;  // nothing seen so far
            m = mt;
            // P = 2^(s - rf) up to 2^15.5; where m is so large that m - 11 is rounded to
            // less than that allows, rf = m
            float nrf = m - kShift;
            if (m - nrf > kShift + 0.5f) nrf = m;
            alpha = none ? 1.f : ex2_approx(rf - nrf);
            rf = nrf;
          }
          if (__any_sync(0xffffffffu, fabsf(rf) > kFar)) {
            masked = true;
            lim_lo = 0;
          }
          l *= alpha;
          if (new_vref) {
            const float top = vref > 0.f ? fmaxf(v_top[tid], vmax) : vmax, to = next_reference(vmax, top);
            v_top[tid] = top;
            alpha *= vref / to;
            vref = to;
            ivref = 1.f / to;
          }
          if (i > 0) {
#pragma unroll 1
            for (int q = half * (D / 32); q < (half + 1) * (D / 32); ++q) {
              uint32_t r[16];
              tmem_ld16(tO + 16 * q, r);
              tmem_wait_ld();
              reg_fence16(r);
#pragma unroll
              for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * alpha);
              tmem_st16(tO + 16 * q, r);
            }
            tmem_wait_st();
          }
        }
        // ---- P over S: the upper 32 scores' into the columns that they came from, then
        // the others'
        const uint64_t nref = f2_pack(-rf, -rf);
        uint64_t ls[2] = {0ull, 0ull};
#pragma unroll 1
        for (int q = 1; q >= 0; --q) {
          tmem_ld32_now(tS + 32 * q, s);
          if (masked) mask_32(s, ks + 2 * q, fs, seen - 32 * q);
          const float f0 = factor(2 * q), f1 = factor(2 * q + 1);
          const uint32_t dst = tS + (q ? 32 : 48);
          p_32(s, f0, f1, vs[2 * q] * ivref, vs[2 * q + 1] * ivref, nref, ls, dst);
        }
        float a0, a1, b0, b1;
        f2_unpack(ls[0], a0, a1);
        f2_unpack(ls[1], b0, b1);
        l += (a0 + a1) + (b0 + b1);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&p_full[x]);
      }
      // ---- the next unit's rows of q while the last products run
      n0 += seg;
      if (n0 < N) {
        next_unit(p, prefix, w, begin + n0);
        load_q(w);
      }
      // ---- epilogue
      const bool whole = seg == here.tiles;
      // parts of a unit: a CTA's first segment goes to slot 0, a later one to 1
      const size_t part = 2 * static_cast<size_t>(blockIdx.x) + (n0 == seg ? 0 : 1);
      if (active) {
        row_l[x][half][row] = l;
        pair_sync();
        l += row_l[x][half ^ 1][row];
        ok &= warp_wait(&o_full[x], segs & 1, &abort_flag, p.status);
        ++segs;
        tc_fence_after();
        const bool valid = ok && 128 * x + row < rows;
        const int head = here.kvh * p.g + my_row % p.g;
        const size_t token = here.r.q0 + my_row / p.g;
        const float mul = whole ? (l != 0.f ? 1.f / l : 0.f) : kKv8Join;
        for (int q = half * (D / 64); q < (half + 1) * (D / 64); ++q) {
          uint32_t bits = 0;
          if (nan && valid) {  // (before the load: its registers would be saved for the call)
            const int key0 = imax(here.tile * kKv8Tile, unit_lo / kKv8Tile * kKv8Tile);
            bits = nan_columns<D>(p, here.b, here.kvh, key0, imin(limit, (here.tile + seg) * kKv8Tile), q);
          }
          uint32_t r[32];
          __syncwarp();
          tmem_ld32_now(tO + 32 * q, r);
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * mul * vref);
          if (!valid) continue;
          if (bits) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if ((bits >> j) & 1u) r[j] = 0x7FFFFFFFu;
          }
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.o + (token * p.Hq + head) * D + 32 * q);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint4 y;
              y.x = pack_bf16x2(__uint_as_float(r[8 * v]), __uint_as_float(r[8 * v + 1]));
              y.y = pack_bf16x2(__uint_as_float(r[8 * v + 2]), __uint_as_float(r[8 * v + 3]));
              y.z = pack_bf16x2(__uint_as_float(r[8 * v + 4]), __uint_as_float(r[8 * v + 5]));
              y.w = pack_bf16x2(__uint_as_float(r[8 * v + 6]), __uint_as_float(r[8 * v + 7]));
              dst[v] = y;
            }
          } else {
            // (a part is [D / 4][rows][4]: a warp's rows are neighbours)
            float4* dst = reinterpret_cast<float4*>(p.part_o + part * kRows * D) + 8 * q * kRows + 128 * x + row;
#pragma unroll
            for (int v = 0; v < 8; ++v)
              dst[v * kRows] = make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                   __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
          }
        }
        if (valid && whole && half == 0 && p.lse)
          p.lse[static_cast<size_t>(head) * p.n_tokens + token] =
              l != 0.f ? (rf + log2f(l)) * 0.6931471805599453f : -INFINITY;
        if (valid && !whole && half == 0)  // nothing seen (or only NaN): a reference of -inf
          *reinterpret_cast<float2*>(p.part_ml + 2 * (part * kRows + 128 * x + row)) =
              make_float2(m == -INFINITY ? -INFINITY : rf, l * kKv8Join);
        tc_fence_before();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 20) tmem_dealloc(tmem, 512);
}

// Joins the parts of the units that CTAs cut, in order: block (c, y) rows 32 y ..
// of the unit that CTA c began and did not finish. (One CTA joining a unit's parts
// by itself took 50 us for 24 of them.)
template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv8_join_kernel(const __grid_constant__ Kv8AttendParams p) {
  extern __shared__ int prefix[];
  // (the lengths were there before the attention let this kernel begin)
  tiles_before(p, prefix, kJoinThreads);
  __syncthreads();
  const int total = prefix[p.B], G = imin(static_cast<int>(gridDim.x), total);
  const int c0 = blockIdx.x, row0 = 32 * blockIdx.y;
  Walk w{};
  int begin = 0, first_tile = 0, rows = 0;
  long long last_tile = 0;
  if (c0 < G && total != kTooManyTiles) {
    begin = static_cast<int>(static_cast<long long>(c0) * total / G);
    const int end = static_cast<int>(static_cast<long long>(c0 + 1) * total / G);
    w = walk_to(p, prefix, end - 1);
    first_tile = end - 1 - w.tile;
    last_tile = static_cast<long long>(first_tile) + w.tiles - 1;
    if (first_tile >= begin && last_tile >= end) rows = imin(32, rows_of(p, w.r, w.rt) - row0);
  }
  // the parts are there; every block waits, so that what follows this kernel
  // also follows the attention
  after_previous();
  if (rows <= 0) return;
  // CTA of list index x: the largest c with floor(c * total / G) <= x
  const int c1 = static_cast<int>(((last_tile + 1) * G - 1) / total);
  const int slot0 = begin == first_tile ? 0 : 1;
  // a thread takes four rows' elements d .. d + 3, two parts' loads at a time
  constexpr int kVecs = D / 4;
  static_assert(kJoinThreads * 4 == 32 * 32, "32 rows of D 128");
  const int r0 = row0 + threadIdx.x % 8, v = threadIdx.x / 8;
  if (v >= kVecs) return;
  float4 sum[4];
  float M[4], L[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    M[i] = -INFINITY;
    L[i] = 0.f;
  }
  for (int c = c0; c <= c1; c += 2) {
    float2 ml[2][4];
    float4 y[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + 8 * i;
        ml[j][i] = make_float2(-INFINITY, 0.f);
        y[j][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c + j <= c1 && r - row0 < rows) {
          const size_t part = 2 * static_cast<size_t>(c + j) + (c + j == c0 ? slot0 : 0);
          ml[j][i] = *reinterpret_cast<const float2*>(p.part_ml + 2 * (part * kRows + r));
          y[j][i] = reinterpret_cast<const float4*>(p.part_o + part * kRows * D)[v * kRows + r];
        }
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float mn = fmaxf(M[i], fmaxf(ml[0][i].x, ml[1][i].x));
      const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: sums of 0 (or NaN)
      const float a = ex2_approx(M[i] - ref);
      sum[i] = make_float4(sum[i].x * a, sum[i].y * a, sum[i].z * a, sum[i].w * a);
      L[i] = M[i] == -INFINITY ? L[i] : L[i] * a;
      M[i] = mn;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float b = ex2_approx(ml[j][i].x - ref);
        sum[i] = make_float4(sum[i].x + y[j][i].x * b, sum[i].y + y[j][i].y * b, sum[i].z + y[j][i].z * b,
                             sum[i].w + y[j][i].w * b);
        L[i] += ml[j][i].x == -INFINITY ? ml[j][i].y : ml[j][i].y * b;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 8 * i;
    if (r - row0 >= rows) break;
    const int rr = w.rt * kRows + r, head = w.kvh * p.g + rr % p.g;
    const size_t token = w.r.q0 + rr / p.g;
    const float inv = L[i] != 0.f ? 1.f / L[i] : 0.f;
    uint2 y;
    y.x = pack_bf16x2(sum[i].x * inv, sum[i].y * inv);
    y.y = pack_bf16x2(sum[i].z * inv, sum[i].w * inv);
    *reinterpret_cast<uint2*>(p.o + (token * p.Hq + head) * D + 4 * v) = y;
    if (v == 0 && p.lse)
      p.lse[static_cast<size_t>(head) * p.n_tokens + token] =
          L[i] != 0.f ? (M[i] + kKv8JoinShift + log2f(L[i])) * 0.6931471805599453f : -INFINITY;
  }
}

namespace {
template <int D, int kType>
cudaError_t launch(const Kv8AttendParams& p, int slot, int sms, cudaStream_t stream) {
  int dev = 0;
  cudaGetDevice(&dev);
  const cudaError_t e = set_smem_attr_once((const void*)kv8_chunk_kernel<D, kType>, slot, dev,
                                           Cfg<D>::bytes(kMaxRequests));
  if (e != cudaSuccess) return e;
  const int grid = imin(kKv8ChunkMaxCtas, sms);
  const cudaError_t launched =
      launch_after(kv8_chunk_kernel<D, kType>, dim3(grid), kThreads, Cfg<D>::bytes(p.B), stream, p);
  if (launched != cudaSuccess) return launched;
  return launch_after(kv8_join_kernel<D>, dim3(grid, kRows / 32), kJoinThreads, (p.B + 1) * sizeof(int), stream, p);
}
}  // namespace

cudaError_t launch_kv8_chunk(const Kv8AttendParams& p, int D, int kv_type, int sms, cudaStream_t stream) {
  const bool e4m3 = kv_type == STAR_KV8_E4M3;
  if (D == 128)
    return e4m3 ? launch<128, STAR_KV8_E4M3>(p, 11, sms, stream) : launch<128, STAR_KV8_INT8>(p, 12, sms, stream);
  return e4m3 ? launch<64, STAR_KV8_E4M3>(p, 13, sms, stream) : launch<64, STAR_KV8_INT8>(p, 14, sms, stream);
}

}  // namespace star
