// Attention of many new tokens of a request (a query chunk, a prompt's next
// piece) over its 8-bit pages, on the 5th-generation tensor cores.
//
// The mathematics is kv8_decode.cu's: s = ks_j (q . K) / sqrt(D), o = sum
// e^(s - m) vs_j V / sum e^(s - m), token t of T seeing kv - T + t + 1 keys.
// Bound: the exponential unit and the tensor cores, about equally (128 x 128
// scores are 1024 cycles of either).
//  * The T * g (token, query head) rows of a (request, KV head) are cut into
//    tiles of 256 rows, two slots of 128: a K or V tile of 128 keys is read and
//    converted once for both.
//  * Work is cut by (row tile, key tile) as in kv8_decode.cu: CTA c of G owns an
//    equal contiguous range of the list, whatever the lengths; a row tile's key
//    tiles end with its last row's limit. Cut units go to the workspace and
//    are joined in order by the CTA that finishes last.
//  * Four warps read codes with 16-byte loads, a tile ahead, and write them as
//    fp16 (exact) in the 128-byte-swizzled layout that tcgen05.mma reads; K and V
//    have the same layout. q is fp16 times a power of two per row, which keeps
//    all its bits for elements down to 2^-29 of the row's largest.
//  * Warps 0-3 and 4-7 own a slot each (thread = row = lane of tensor memory).
//    MMA order per key tile: PV0(n), S0(n+1), PV1(n), S1(n+1), so that a slot's
//    softmax runs beside the other's products. P (fp16) overwrites the first
//    half of its S and feeds the P V product from tensor memory.
//  * P is rounded to fp16 under 2^11 as in kv8_decode.cu, the running maximum
//    moves when it grows by more than 2^4, and V scales enter through P as the
//    ratio to a running reference that stays within [1, 2^12) of the tile's
//    largest. Values whose scale is 2^24 below the largest of their 128 keys
//    lose bits.
#include <math.h>

#include "kv8_codes.cuh"
#include "kv8_kernels.cuh"
#include "star_kernels.cuh"

namespace star {

namespace {

constexpr int kThreads = 512;  // 2 x 4 softmax warps, 4 converter warps, 1 MMA warp (+ 3 idle)
constexpr int kRows = kKv8ChunkRows;
constexpr int kRing = 8;       // tiles whose scales are kept: more than the stages ahead
constexpr float kShift = 11.f; // P is held as 2^11 e^(s - m)
constexpr float kSlack = 4.f;  // growth of the maximum (log2) before it moves

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

struct Scales {
  float k[8], v[8];  // of the 8 groups of 16 keys; k < 0: no such page
  int nan[4];        // by converter warp: a V code at the causal edge is NaN
};

// Instruction descriptor of tcgen05.mma kind::f16 with fp16 A and B, fp32 D.
constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// A bounded wait with one answer for the whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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
  __shared__ uint64_t q_full[2], s_full[2], p_full[2], o_full[2], join, done;
  __shared__ uint64_t k_full[S], k_empty[S], v_full[S], v_empty[S], sc_full[kRing], nan_full[kRing];
  __shared__ __align__(16) Scales ring[kRing];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ int s_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- tiles before each request
  {
    bool any_bad = false;
    for (int b = warp; b < p.B; b += kThreads / 32) {
      bool bad;
      const Request r = request_of(p, b, &bad);
      any_bad |= bad;
      int sum = 0;
      for (int rt = lane; rt < r.row_tiles; rt += 32) sum += tiles_of(p, r, rt);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) prefix[b + 1] = sum * p.Hkv;
    }
    if (any_bad && lane == 0 && blockIdx.x == 0) atomicOr(p.status, kDevBounds);
    if (tid == 0 && blockIdx.x == 0) p.status[1] = p.header_bytes;
    __syncthreads();
    if (warp == 0) {
      int base = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        int v = b0 + lane < p.B ? prefix[b0 + lane + 1] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, v, d);
          if (lane >= d) v += up;
        }
        if (b0 + lane < p.B) prefix[b0 + lane + 1] = base + v;
        base += __shfl_sync(0xffffffffu, v, 31);
      }
      if (lane == 0) prefix[0] = 0;
    }
    if (tid == 0) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(&q_full[x], 128);
        mbar_init(&s_full[x], 1);
        mbar_init(&p_full[x], 128);
        mbar_init(&o_full[x], 1);
      }
      for (int s = 0; s < S; ++s) {
        mbar_init(&k_full[s], 128);
        mbar_init(&k_empty[s], 1);
        mbar_init(&v_full[s], 128);
        mbar_init(&v_empty[s], 1);
      }
      for (int s = 0; s < kRing; ++s) {
        mbar_init(&sc_full[s], 4);
        mbar_init(&nan_full[s], 4);
      }
      mbar_init(&join, 256);
      mbar_init(&done, 1);
      fence_barrier_init();
      abort_flag = 0;
    }
    __syncthreads();
  }
  const int total = prefix[p.B];
  const int G = imin(static_cast<int>(gridDim.x), total);  // CTAs with work
  if (static_cast<int>(blockIdx.x) >= G) return;
  const int begin = static_cast<int>(static_cast<long long>(blockIdx.x) * total / G);
  const int end = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * total / G);
  const int N = end - begin;

  if (warp == 12) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp >= 12) {
    // ------------------------------------------------------------ MMA issuer
    regs_down<48>();
    if (warp == 12 && lane == 0) {
      constexpr uint32_t idS = idesc_f16(128, 128, 0);  // S = Q K^T, both K-major
      constexpr uint32_t idO = idesc_f16(128, D, 1);    // O += P V, V is N-major
      const uint32_t q_base = smem_u32(sm), k_base = q_base + C::kOffK, v_base = q_base + C::kOffV;
      auto kmajor = [&](uint32_t base, int kk) {
        return sdesc_sw128(base + (kk >> 2) * C::kHalf + (kk & 3) * 32, 16, 1024);
      };
      auto issue_s = [&](int x, int st) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + 128 * x, kmajor(q_base + x * C::kTile, kk), kmajor(k_base + st * C::kTile, kk),
                 idS, kk > 0 ? 1u : 0u);
        mma_commit(&s_full[x]);
      };
      Walk w = walk_to(p, prefix, begin);
      int slots = rows_of(p, w.r, w.rt) > 128 ? 2 : 1;
      bool first = true;       // first tile of a segment: O starts anew
      uint32_t cnt[2] = {0, 0};  // tiles of a slot so far
      uint32_t segs[2] = {0, 0};
      bool ok = mbar_wait(&k_full[0], 0, &abort_flag, p.status);
      for (int x = 0; ok && x < slots; ++x) {
        ok = mbar_wait(&q_full[x], 0, &abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        issue_s(x, 0);
        segs[x] = 1;
      }
      if (ok) mma_commit(&k_empty[0]);
      for (int n = 0; ok && n < N; ++n) {
        const int st = n % S, nst = (n + 1) % S;
        const bool has_next = n + 1 < N, seg_end = w.tile + 1 == w.tiles || !has_next;
        const int now = slots;
        bool next_first = false;
        if (has_next) {
          if (seg_end) {
            next_unit(p, prefix, w, begin + n + 1);
            slots = rows_of(p, w.r, w.rt) > 128 ? 2 : 1;
            next_first = true;
          } else {
            ++w.tile;
          }
          if (!mbar_wait(&k_full[nst], ((n + 1) / S) & 1, &abort_flag, p.status)) break;
        }
        if (!mbar_wait(&v_full[st], (n / S) & 1, &abort_flag, p.status)) break;
        for (int x = 0; ok && x < 2; ++x) {
          if (x < now) {
            if (!(ok = mbar_wait(&p_full[x], cnt[x] & 1, &abort_flag, p.status))) break;
            ++cnt[x];
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(tmem + 256 + 128 * x, tmem + 128 * x + kk * 8,
                     sdesc_sw128(v_base + st * C::kTile + kk * 2048, C::kHalf, 1024), idO,
                     (!first || kk > 0) ? 1u : 0u);
            if (seg_end) mma_commit(&o_full[x]);
          }
          if (has_next && x < slots) {
            if (next_first) {
              if (!(ok = mbar_wait(&q_full[x], segs[x] & 1, &abort_flag, p.status))) break;
              ++segs[x];
            }
            tc_fence_after();
            issue_s(x, nst);
          }
        }
        if (!ok) break;
        if (has_next) mma_commit(&k_empty[nst]);
        mma_commit(&v_empty[st]);
        first = seg_end;
      }
      // every MMA in flight ends before tensor memory is released
      mma_commit(&done);
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(&done, 0))
        if (global_ns() - t0 > 100000000ull) break;
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------ converters
    regs_down<112>();
    constexpr int kLoads = D / 16;      // 16-byte loads of a thread for a K or V tile
    constexpr int kPerRow = D / 16;     // 16-byte pieces of a row
    constexpr int kRowsPer = 32 / kPerRow;
    const int cw = warp - 8, ch = lane % kPerRow, r0 = 32 * cw + lane / kPerRow;
    const int P = 1 << p.page_shift;
    struct Tile {
      int key0, kv, kvh, edge, page[2];  // pages of this warp's two groups of 16 keys
    };
    Walk w = walk_to(p, prefix, begin);
    auto fetch = [&]() {
      Tile t;
      t.key0 = w.tile * kKv8Tile;
      t.kv = w.r.kv;
      t.kvh = w.kvh;
      t.edge = t.key0 + kKv8Tile > keys_of_row(p, w.r, w.rt * kRows);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = t.key0 + 32 * cw + 16 * i;
        t.page[i] = key < t.kv ? p.table[static_cast<size_t>(w.b) * p.max_pages + (key >> p.page_shift)] : 0;
      }
      return t;
    };
    auto step = [&](int n) {  // to tile n of this CTA
      if (w.tile + 1 < w.tiles) ++w.tile;
      else next_unit(p, prefix, w, begin + n);
    };
    auto load = [&](uint4 (&x)[kLoads], const Tile& t, const uint8_t* pages) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int r = r0 + kRowsPer * j, key = t.key0 + r;
        const int page = t.page[j >= kLoads / 2];
        x[j] = make_uint4(0u, 0u, 0u, 0u);  // keys behind the last one are zero codes
        if (key < t.kv && page >= 0 && page < p.num_pages) {
          const size_t row = ((static_cast<size_t>(page) * p.Hkv + t.kvh) << p.page_shift) + (key & (P - 1));
          x[j] = __ldg(reinterpret_cast<const uint4*>(pages + row * D) + ch);
        }
      }
    };
    // lanes 0, 1: K scales of the warp's groups; lanes 2, 3: V scales
    auto load_scale = [&](const Tile& t) -> float {
      if (lane >= 4) return 0.f;
      const int page = lane & 1 ? t.page[1] : t.page[0];
      const bool real = page >= 0 && page < p.num_pages;
      if (!real) {
        atomicOr(p.status, kDevBounds);
        return lane < 2 ? -1.f : 0.f;
      }
      if (t.key0 + 32 * cw + 16 * (lane & 1) >= t.kv) return 0.f;
      return __ldg((lane < 2 ? p.k_scale : p.v_scale) + static_cast<size_t>(page) * p.Hkv + t.kvh);
    };
    auto convert = [&](const uint4 (&x)[kLoads], uint8_t* dst) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int r = r0 + kRowsPer * j;
        uint4 a, b;
        codes_to_half2<kType>(x[j].x, a.x, a.y);
        codes_to_half2<kType>(x[j].y, a.z, a.w);
        codes_to_half2<kType>(x[j].z, b.x, b.y);
        codes_to_half2<kType>(x[j].w, b.z, b.w);
        // columns 16 ch .. + 15: chunks c and c + 1 of a 64-column half. At D 128
        // eight lanes share a row and two of them a chunk position: the second
        // half's lanes write in the other order, so the banks differ
        const int c = (2 * ch) & 7;
        uint8_t* half = dst + (ch >> 2) * C::kHalf;
        const bool turn = ch >= 4;
        *reinterpret_cast<uint4*>(half + sw128_offset(r, c + (turn ? 1 : 0))) = turn ? b : a;
        *reinterpret_cast<uint4*>(half + sw128_offset(r, c + (turn ? 0 : 1))) = turn ? a : b;
      }
    };
    uint4 kx[kLoads], vx[kLoads];
    Tile cur = fetch(), nxt = cur;
    load(kx, cur, p.k_pages);
    load(vx, cur, p.v_pages);
    float sc = load_scale(cur);
    if (N > 1) {
      step(1);
      nxt = fetch();
    }
    for (int n = 0; n < N; ++n) {
      const int st = n % S;
      const uint32_t again = ((n / S) - 1) & 1;
      // the scales' ring is deeper than the stages ahead: no wait
      Scales& ss = ring[n % kRing];
      if (n >= S && !warp_wait(&k_empty[st], again, &abort_flag, p.status)) break;
      if (lane < 2) ss.k[2 * cw + lane] = sc;
      else if (lane < 4) ss.v[2 * cw + lane - 2] = sc;
      else if (lane == 4) ss.nan[cw] = 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc_full[n % kRing]);
      convert(kx, sm + C::kOffK + st * C::kTile);
      fence_async_shared();
      mbar_arrive(&k_full[st]);
      if (n + 1 < N) {
        load(kx, nxt, p.k_pages);
        sc = load_scale(nxt);
      }
      if (n >= S && !warp_wait(&v_empty[st], again, &abort_flag, p.status)) break;
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
        __syncwarp();
        if (lane == 0) mbar_arrive(&nan_full[n % kRing]);
      } else if (lane == 0) {
        mbar_arrive(&nan_full[n % kRing]);
      }
      convert(vx, sm + C::kOffV + st * C::kTile);
      fence_async_shared();
      mbar_arrive(&v_full[st]);
      cur = nxt;
      if (n + 1 < N) load(vx, nxt, p.v_pages);
      if (n + 2 < N) {
        step(n + 2);
        nxt = fetch();
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    regs_up<176>();
    const int x = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + 128 * x, tO = tmem + lanes + 256 + 128 * x;
    uint32_t cnt = 0, segs = 0, joins = 0;
    // every softmax thread has got here (bounded)
    auto softmax_sync = [&]() {
      mbar_arrive(&join);
      return warp_wait(&join, joins++ & 1, &abort_flag, p.status);
    };
    float fs = 0.f;  // this row's factor: 2^-e log2(e) / sqrt(D)
    // this thread's row of q into the slot's tile, as fp16 times a power of two
    auto load_q = [&](const Walk& w) {
      const int r = w.rt * kRows + 128 * x + row;
      uint8_t* dst = sm + x * C::kTile;
      uint4 v[D / 8];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < w.r.T * p.g) {
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (w.r.q0 + r / p.g) * p.qs[0] + (w.kvh * p.g + r % p.g) * p.qs[1]);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) v[i] = __ldg(src + i);
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                     __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu)));
      const int e = static_cast<int>(imax(top & 0xFFFFu, top >> 16) >> 7);  // biased exponent
      const int up = imin(254, imax(1, 127 + 14 - (e - 127)));  // 2^(14 - (e - 127)), a normal number
      const float mul = __uint_as_float(static_cast<uint32_t>(up) << 23);
      fs = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(imax(1, 254 - up)) << 23);
      auto two = [&](uint32_t u) { return half2_of(bf16_lo(u) * mul, bf16_hi(u) * mul); };
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<uint4*>(dst + (i >> 3) * C::kHalf + sw128_offset(row, i & 7)) =
            make_uint4(two(v[i].x), two(v[i].y), two(v[i].z), two(v[i].w));
      fence_async_shared();
      mbar_arrive(&q_full[x]);
    };
    Walk w = walk_to(p, prefix, begin);
    if (x == 0 || rows_of(p, w.r, w.rt) > 128) load_q(w);
    bool ok = true;
    for (int n0 = 0; n0 < N;) {
      // ---- one segment: the tiles of one unit that this CTA holds
      const Walk here = w;
      const int seg = imin(here.tiles - here.tile, N - n0);
      const int rows = rows_of(p, here.r, here.rt);
      const bool active = x == 0 || rows > 128;
      const int my_row = here.rt * kRows + 128 * x + row;
      const int limit = keys_of_row(p, here.r, my_row);
      // keys that the slot's and the unit's first rows see
      const int lim_lo = keys_of_row(p, here.r, here.rt * kRows + 128 * x);
      const int unit_lo = keys_of_row(p, here.r, here.rt * kRows);
      float m = -INFINITY, rf = 0.f, l = 0.f, vref = 0.f;
      bool nan = false;
      for (int i = 0; active && i < seg; ++i, ++cnt) {
        const int n = n0 + i;
        const Scales& ss = ring[n % kRing];
        if (!(ok = warp_wait(&s_full[x], cnt & 1, &abort_flag, p.status))) break;
        // (S of tile n is there, so its scales' phase is the last one completed)
        if (!(ok = warp_wait(&sc_full[n % kRing], (n / kRing) & 1, &abort_flag, p.status))) break;
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(tS + 32 * q, sr[q]);
        float kmin = ss.k[0], vmax = ss.v[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) {
          kmin = fminf(kmin, ss.k[j]);
          vmax = fmaxf(vmax, ss.v[j]);
        }
        bool scaled = false;  // the factors are applied already
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) reg_fence32(sr[q]);

        const int key0 = (here.tile + i) * kKv8Tile;
        if (key0 + kKv8Tile > lim_lo || kmin < 0.f) {
          // masked keys and keys of missing pages are -inf (after the factor, which
          // may be 0)
          const int seen = limit - key0;
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float ks = ss.k[2 * q + (j >> 4)];
              const float v = __uint_as_float(sr[q][j]) * (fs * ks);
              sr[q][j] = 32 * q + j < seen && !(ks < 0.f) ? __float_as_uint(v) : 0xFF800000u;
            }
          scaled = true;
        }
        auto factor = [&](int g) { return scaled ? 1.f : fs * ss.k[g]; };
        if (kType == STAR_KV8_E4M3 && key0 + kKv8Tile > unit_lo) {
          if (!(ok = warp_wait(&nan_full[n % kRing], (n / kRing) & 1, &abort_flag, p.status))) break;
          const int4 flags = *reinterpret_cast<const int4*>(ss.nan);
          nan |= (flags.x | flags.y | flags.z | flags.w) != 0;
        }
        // ---- row maximum in log2 units
        float mt = -INFINITY;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const uint32_t* s = &sr[g >> 1][16 * (g & 1)];
          float a = __uint_as_float(s[0]), b = __uint_as_float(s[1]);
#pragma unroll
          for (int j = 2; j < 14; j += 4) {
            a = fmax3(a, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
            b = fmax3(b, __uint_as_float(s[j + 2]), __uint_as_float(s[j + 3]));
          }
          a = fmax3(a, __uint_as_float(s[14]), __uint_as_float(s[15]));
          mt = fmaxf(mt, fmaxf(a, b) * factor(g));
        }
        // ---- move the maximum and the V reference; O and the sum follow
        float alpha = 1.f;
        if (mt > m + kSlack) {
          m = mt;
          // P = 2^(s - rf); where m is so large that m - 11 is rounded, rf = m
          float nrf = m - kShift;
          if (m - nrf > kShift) nrf = m;
          alpha = l == 0.f ? 1.f : ex2_approx(rf - nrf);
          rf = nrf;
        }
        l *= alpha;
        if (vmax > vref || (vmax < vref * 0.000244140625f && vmax > 0.f)) {
          alpha *= vref / vmax;
          vref = vmax;
        }
        if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
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
        const float ivref = vref > 0.f ? 1.f / vref : 0.f;
        // ---- P = 2^(s f - rf) times the V ratio, fp16, over the first half of S
        const uint64_t nref = f2_pack(-rf, -rf);
        uint64_t ls[2] = {0ull, 0ull};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int g = 2 * q + (j >> 3);
            const float f = factor(g), ratio = ss.v[g] * ivref;
            const uint64_t ff = f2_pack(f, f);
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[q][2 * j]), __uint_as_float(sr[q][2 * j + 1])), ff, nref),
                      x0, x1);
            const uint64_t e = f2_pack(ex2_approx(x0), ex2_approx(x1));
            ls[j & 1] = f2_add(ls[j & 1], e);
            f2_unpack(f2_mul(e, f2_pack(ratio, ratio)), x0, x1);
            pk[j] = half2_of(x0, x1);
          }
          tmem_st16(tS + 16 * q, pk);
        }
        float a0, a1, b0, b1;
        f2_unpack(ls[0], a0, a1);
        f2_unpack(ls[1], b0, b1);
        l += (a0 + a1) + (b0 + b1);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      // ---- the next unit's rows of q while the last products run
      n0 += seg;
      if (n0 < N) {
        next_unit(p, prefix, w, begin + n0);
        if (x == 0 || rows_of(p, w.r, w.rt) > 128) load_q(w);
      }
      // ---- epilogue
      const bool whole = seg == here.tiles;
      // parts of a unit: a CTA's first segment goes to slot 0, a later one to 1
      const size_t part = 2 * static_cast<size_t>(blockIdx.x) + (n0 == seg ? 0 : 1);
      if (active) {
        if (!(ok = warp_wait(&o_full[x], segs & 1, &abort_flag, p.status))) break;
        ++segs;
        tc_fence_after();
        const bool valid = 128 * x + row < rows;
        const int head = here.kvh * p.g + my_row % p.g;
        const size_t token = here.r.q0 + my_row / p.g;
        const float mul = whole ? (l != 0.f ? vref / l : 0.f) : vref;
        for (int q = 0; q < D / 32; ++q) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(tO + 32 * q, r);
          tmem_wait_ld();
          reg_fence32(r);
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * mul);
          if (!valid) continue;
          if (nan) {
            const int key0 = imax(here.tile * kKv8Tile, unit_lo / kKv8Tile * kKv8Tile);
            const uint32_t bits = nan_columns<D>(p, here.b, here.kvh, key0,
                                                 imin(limit, (here.tile + seg) * kKv8Tile), q);
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
            float4* dst = reinterpret_cast<float4*>(p.part_o + (part * kRows + 128 * x + row) * D + 32 * q);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              dst[v] = make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                   __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
          }
        }
        if (valid && whole && p.lse)
          p.lse[static_cast<size_t>(head) * p.n_tokens + token] =
              l != 0.f ? (rf + log2f(l)) * 0.6931471805599453f : -INFINITY;
        if (valid && !whole)  // nothing seen (or only NaN): a reference of -inf
          *reinterpret_cast<float2*>(p.part_ml + 2 * (part * kRows + 128 * x + row)) =
              make_float2(m == -INFINITY ? -INFINITY : rf, l);
        tc_fence_before();
      }
      if (!whole) {
        // ---- the last CTA of a cut unit joins its parts in order
        const int first_tile = begin + n0 - seg - here.tile, last_tile = first_tile + here.tiles - 1;
        const int c0 = static_cast<int>(((first_tile + 1ll) * G - 1) / total);
        const int c1 = static_cast<int>(((last_tile + 1ll) * G - 1) / total);
        if (!(ok = softmax_sync())) break;
        if (tid == 0) {
          __threadfence();
          s_last = atomicInc(p.counters + c0, c1 - c0) == static_cast<unsigned>(c1 - c0);
          __threadfence();
        }
        if (!(ok = softmax_sync())) break;
        if (s_last) {
          const int begin0 = static_cast<int>(static_cast<long long>(c0) * total / G);
          const size_t slot0 = 2 * static_cast<size_t>(c0) + (begin0 == first_tile ? 0 : 1);
          for (int e = tid; e < rows * (D / 4); e += 256) {
            const int r = e / (D / 4), d = 4 * (e % (D / 4));
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float M = -INFINITY, L = 0.f;
            for (int c = c0; c <= c1; ++c) {
              const size_t at = (c == c0 ? slot0 : 2 * static_cast<size_t>(c)) * kRows + r;
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + 2 * at));
              const float4 y = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D + d));
              const float mn = fmaxf(M, ml.x);
              if (mn == -INFINITY) {
                L += ml.y;
                continue;
              }
              const float a = ex2_approx(M - mn), b = ex2_approx(ml.x - mn);
              sum = make_float4(sum.x * a + y.x * b, sum.y * a + y.y * b, sum.z * a + y.z * b, sum.w * a + y.w * b);
              L = L * a + ml.y * b;
              M = mn;
            }
            const int rr = here.rt * kRows + r, head = here.kvh * p.g + rr % p.g;
            const size_t token = here.r.q0 + rr / p.g;
            const float inv = L != 0.f ? 1.f / L : 0.f;
            uint2 y;
            y.x = pack_bf16x2(sum.x * inv, sum.y * inv);
            y.y = pack_bf16x2(sum.z * inv, sum.w * inv);
            *reinterpret_cast<uint2*>(p.o + (token * p.Hq + head) * D + d) = y;
            if (d == 0 && p.lse)
              p.lse[static_cast<size_t>(head) * p.n_tokens + token] =
                  L != 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

namespace {
template <int D, int kType>
cudaError_t launch(const Kv8AttendParams& p, int slot, int sms, cudaStream_t stream) {
  int dev = 0;
  cudaGetDevice(&dev);
  const cudaError_t e = set_smem_attr_once((const void*)kv8_chunk_kernel<D, kType>, slot, dev,
                                           Cfg<D>::bytes(kMaxRequests));
  if (e != cudaSuccess) return e;
  kv8_chunk_kernel<D, kType><<<imin(kKv8ChunkMaxCtas, sms), kThreads, Cfg<D>::bytes(p.B), stream>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_kv8_chunk(const Kv8AttendParams& p, int D, int kv_type, int sms, cudaStream_t stream) {
  const bool e4m3 = kv_type == STAR_KV8_E4M3;
  if (D == 128)
    return e4m3 ? launch<128, STAR_KV8_E4M3>(p, 11, sms, stream) : launch<128, STAR_KV8_INT8>(p, 12, sms, stream);
  return e4m3 ? launch<64, STAR_KV8_E4M3>(p, 13, sms, stream) : launch<64, STAR_KV8_INT8>(p, 14, sms, stream);
}

}  // namespace star
