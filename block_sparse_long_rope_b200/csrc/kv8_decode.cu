// Attention of a few new tokens of each request over its 8-bit pages.
//
// With codes K, V of page j and scales ks_j, vs_j, row r of a (request, KV head)
// with query q sees
//   s = ks_j (q . K) / sqrt(D),  o = sum e^(s - m) vs_j V / sum e^(s - m).
// Bound: HBM, one byte an element of K and V: 1M tokens of 8 heads of 128 (2.15 GB)
// take 329 us, 6.5 TB/s, where a loop that only copies takes 309 (348 behind a kernel
// that leaves the L2 full of its writes, which go out meanwhile; 355 to 380 where every
// call has new inputs); 16 requests of 1K to 16K tokens (268 MB) 59 us, whose CTAs end
// between 40 and 59. A short call is latency: 501 tokens of one head 7.0 to 7.5 us, of
// which one tile alone is 4.9. The design keeps the stream going:
//  * The T * g (token, query head) rows of a (request, KV head) form one tile of
//    8 or 16 rows, so each code is read once for all of them; further rows make
//    further tiles.
//  * Work is cut by tiles of 128 keys: CTA c owns an equal contiguous range of
//    the (request, head, row tile, key tile) list, whatever the lengths. Each
//    CTA finds its range from the lengths itself. A CTA that holds a whole
//    unit writes its output; parts of a unit go to the workspace, and the CTA
//    that finishes one last joins its parts in order, once its own list is done.
//  * Each of the 8 warps takes 16 keys of a tile and streams them through its
//    own ring with cp.async, so nothing waits for other warps and pages need
//    only be 16 rows. An instruction copies 512 contiguous bytes (64-byte pieces
//    in fragment order reached 4.6 TB/s instead of 7.0) and swizzles their 16-byte
//    pieces, and the keys are assigned to matrix rows so that the fragments'
//    reads have no bank conflicts either.
//  * The products are mma.m16n8k16 with keys (then head elements) as the 16
//    rows and query rows as the 8 columns, S^T = K q^T and O^T = V^T P^T: 8 query
//    rows waste nothing, and the accumulators are a quarter of a 16-row tile's.
//    Codes become fp16 without rounding; q, scaled by a power of two to just
//    below 2^15, keeps all its bits for elements down to 2^-29 of the row's
//    largest; P^T comes from S^T by an 8x8 transposition in registers.
//  * P is rounded to fp16 under 2^11, so that a weight keeps full precision
//    down to 2^-25 of the largest, and is not flushed before 2^-35: a long flat
//    tail behind one peak still adds up. The running maximum moves only when
//    it grows by more than 2^4, so P < 2^15 stays finite.
//  * V scales enter through P as the ratio to a running reference; beyond
//    [2^-12, 1] the reference moves and O is rescaled (see next_reference).
#include <math.h>

#include <atomic>

#include "kv8_codes.cuh"
#include "kv8_kernels.cuh"
#include "star_kernels.cuh"

namespace star {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;
// 16 rows of D 128 hold 64 accumulators and 32 words of q a thread: within 128
// registers they spill throughout (16 rows over 100K keys of 8 heads: 88 us instead of
// 65). At D 64 the spills are few (28 bytes of stores and 52 of loads for e4m3) and two
// CTAs take 41 us instead of 53; 8 rows of D 128 in e4m3 spill 20 and 36.
__host__ __device__ constexpr int ctas_per_sm(int D, int NT) { return NT == 1 || D == 64 ? 2 : 1; }
constexpr float kPShift = 11.f;  // P is held as 2^11 e^(s - m)
constexpr float kSlack = 4.f;    // growth of the maximum (log2) before it moves

template <int D>
struct Cfg {
  // one warp's stage: 16 keys of K codes, then of V codes, in whole 128-byte lines;
  // the two scales of every stage come after the rings
  static constexpr int kStage = 16 * D * 2;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kScales = kWarps * kRing;
  static constexpr int kPrefix = kScales + kWarps * kStages * 8;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Offset of 16-byte piece c of row r in a stage's 16 rows of D bytes: the pieces
// of a 128-byte line trade places by the line's number.
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}
// Key of matrix row i (0..7): at D 128 neighbours are 4 apart, in other banks.
template <int D>
__device__ __forceinline__ int key_of(int i) {
  return D == 128 ? ((i & 1) << 2) | (i >> 1) : i;
}

// 0xff in each byte of four e4m3 codes that is NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

// What a CTA needs of one request.
struct Request {
  int q0, T, kv, row_tiles, tiles;  // tiles: key tiles of every row tile, at least 1
};
template <int kRows>
__device__ __forceinline__ Request request_of(const Kv8AttendParams& p, int b, bool* bad) {
  Request r;
  const int c0 = p.cu_new[b], c1 = p.cu_new[b + 1];
  r.q0 = c0;
  r.T = c1 - c0;
  r.kv = p.kv_len[b];
  *bad = c0 < 0 || c1 < c0 || c1 > p.n_tokens || r.T > p.max_new || r.kv < 0 || r.kv > p.max_kv;
  if (*bad) r.T = 0;
  r.row_tiles = ceil_div(r.T * p.g, kRows);
  r.tiles = imax(1, ceil_div(r.kv, kKv8Tile));
  return r;
}

// A unit that a CTA holds a part of.
struct Cut {
  int first_tile, row0, rows, kvh, q0, c0, c1;  // c0 .. c1: the CTAs with its parts
  int last;                                     // this CTA finished last
};

// Four elements of a joined row of a cut unit, and its lse.
__device__ __forceinline__ void finish_row(const Kv8AttendParams& p, const Cut& c, int n, int d, int D,
                                           const float4& sum, float M, float L) {
  const int r = c.row0 + n, head = c.kvh * p.g + r % p.g;
  const size_t token = c.q0 + r / p.g;
  const float inv = L != 0.f ? 1.f / L : 0.f;
  uint2 y;
  y.x = pack_bf16x2(sum.x * inv, sum.y * inv);
  y.y = pack_bf16x2(sum.z * inv, sum.w * inv);
  *reinterpret_cast<uint2*>(p.o + (token * p.Hq + head) * D + d) = y;
  if (d == 0 && p.lse)
    p.lse[static_cast<size_t>(head) * p.n_tokens + token] =
        L != 0.f ? (M + (kKv8JoinShift - kPShift) + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

template <int D, int kType, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, NT))
    kv8_decode_kernel(const __grid_constant__ Kv8AttendParams p) {
  using C = Cfg<D>;
  constexpr int kRows = 8 * NT;
  constexpr int kSteps = D / 16;  // k-steps of S^T, and 16-row tiles of O^T
  constexpr int kWords = D / 16;  // 32-bit words of a thread's share of a K row
  extern __shared__ __align__(128) uint8_t smem[];
  int* prefix = reinterpret_cast<int*>(smem + C::kPrefix);  // [B + 1] tiles before request b
  __shared__ float wm[kWarps][kRows], wl[kWarps][kRows];
  __shared__ int warp_tiles[kWarps];
  __shared__ float v_top[kWarps];  // largest V scale so far (a register more spills)
  __shared__ Cut cuts[2];
  int ncuts = 0;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, t4 = lane & 3;
  const int P = 1 << p.page_shift;

  after_previous();
  // ---- tiles before each request
  {
    const int per = ceil_div(p.B, kThreads);
    const int b0 = imin(p.B, tid * per), b1 = imin(p.B, b0 + per);
    int mine = 0;
    bool any_bad = false;
    for (int b = b0; b < b1; ++b) {
      bool bad;
      const Request r = request_of<kRows>(p, b, &bad);
      mine = add_tiles(mine, times_tiles(p.Hkv, times_tiles(r.row_tiles, r.tiles)));
      any_bad |= bad;
    }
    if (any_bad && blockIdx.x == 0) atomicOr(p.status, kDevBounds);
    if (tid == 0 && blockIdx.x == 0) p.status[1] = p.header_bytes;
    int inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc = add_tiles(inc, up);
    }
    if (lane == 31) warp_tiles[warp] = inc;
    __syncthreads();
    int at = inc - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += warp_tiles[w];
      total = add_tiles(total, warp_tiles[w]);
    }
    for (int b = b0; b < b1; ++b) {
      bool bad;
      const Request r = request_of<kRows>(p, b, &bad);
      prefix[b] = at;
      at += p.Hkv * r.row_tiles * r.tiles;
    }
    if (tid == 0) prefix[p.B] = total;
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

  // ---- this warp's ring
  uint8_t* ring = smem + warp * C::kRing;
  const uint32_t ring_u32 = smem_u32(ring);
  float* scales = reinterpret_cast<float*>(smem + C::kScales) + warp * kStages * 2;  // K and V scale by stage

  // cursors over the tile list: request, unit (head, row tile) in it, key tile
  struct Cursor {
    int b, unit, tile;
    Request r;
  };
  auto locate = [&](int at) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= at) lo = mid;
      else hi = mid;
    }
    Cursor c;
    bool bad;
    c.b = lo;
    c.r = request_of<kRows>(p, lo, &bad);
    c.unit = (at - prefix[lo]) / c.r.tiles;
    c.tile = (at - prefix[lo]) - c.unit * c.r.tiles;
    return c;
  };
  auto advance = [&](Cursor& c, int next) {  // to list index next < end
    if (++c.tile < c.r.tiles) return;
    c.tile = 0;
    if (++c.unit < p.Hkv * c.r.row_tiles) return;
    c.unit = 0;
    bool bad;
    do ++c.b;
    while (prefix[c.b + 1] <= next);  // requests without work
    c.r = request_of<kRows>(p, c.b, &bad);
  };

  // ---- the copies run kStages - 1 tiles ahead; page numbers one further
  Cursor pf = locate(begin);
  int pf_at = begin;
  auto page_of = [&](const Cursor& c) -> int {
    const int key0 = c.tile * kKv8Tile + 16 * warp;
    return key0 < c.r.kv ? p.table[static_cast<size_t>(c.b) * p.max_pages + (key0 >> p.page_shift)] : 0;
  };
  int pf_page = page_of(pf);
  auto issue = [&](int stage) {
    if (pf_at < end) {
      const int key0 = pf.tile * kKv8Tile + 16 * warp;
      const int kvh = pf.unit / pf.r.row_tiles;
      const uint32_t dst = ring_u32 + stage * C::kStage;
      if (key0 < pf.r.kv) {
        const bool ok = pf_page >= 0 && pf_page < p.num_pages;
        const size_t unit = static_cast<size_t>(ok ? pf_page : 0) * p.Hkv + kvh;
        const size_t row = (unit << p.page_shift) + (key0 & (P - 1));
        const uint8_t* kb = p.k_pages + row * D;
        const uint8_t* vb = p.v_pages + row * D;
        const int left = pf.r.kv - key0;  // rows behind the last key read as zero codes
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {  // 512 bytes: 4 rows, or 8 of D 64
          const int r = (512 / D) * i + lane / (D / 16), bytes = r < left ? 16 : 0;
          const uint32_t to = dst + piece<D>(r, lane % (D / 16));
          cp_async16(to, kb + 512 * i + 16 * lane, bytes);
          cp_async16(to + 16 * D, vb + 512 * i + 16 * lane, bytes);
        }
        float* sc = scales + 2 * stage;
        if (ok) {
          if (lane < 2) cp_async4(smem_u32(sc + lane), (lane ? p.v_scale : p.k_scale) + unit);
        } else if (lane == 0) {  // no such page: its keys are invisible
          sc[0] = -1.f;
          atomicOr(p.status, kDevBounds);
        }
      }
      if (++pf_at < end) {
        advance(pf, pf_at);
        pf_page = page_of(pf);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s);

  Cursor cur = locate(begin);
  int stage = 0, at = begin;
  while (at < end) {
    // ---- one segment: the tiles of one unit that this CTA holds
    const int kvh = cur.unit / cur.r.row_tiles, rt = cur.unit - kvh * cur.r.row_tiles;
    const int tile0 = cur.tile, seg = imin(cur.r.tiles - tile0, end - at);
    const int rows = imin(kRows, cur.r.T * p.g - rt * kRows);  // valid rows of the tile
    const Cursor here = cur;
    // rows sit at token t = r / g of the request; row r sees keys below its limit
    const int past = here.r.kv - here.r.T + 1;
    const int lim_lo = past + (rt * kRows) / p.g;              // the first row's
    const int lim_hi = past + (rt * kRows + rows - 1) / p.g;   // the last row's

    // ---- q as B fragments: column n = gq is row rt * kRows + 8 * nt + gq
    uint32_t qf[NT][kSteps][2];
    float qscale[NT];  // this lane's row (gq): 2^e log2(e) / sqrt(D)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = 8 * nt + gq, r = rt * kRows + n;
      uint32_t w[kSteps * 2];
#pragma unroll
      for (int i = 0; i < kSteps * 2; ++i) w[i] = 0u;
      if (n < rows) {
        const __nv_bfloat16* src = p.q + (here.r.q0 + r / p.g) * p.qs[0] +
                                   (kvh * p.g + r % p.g) * p.qs[1] + 16 * t4;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + 64 * c + 8 * v);
            w[8 * c + 4 * v + 0] = x.x;
            w[8 * c + 4 * v + 1] = x.y;
            w[8 * c + 4 * v + 2] = x.z;
            w[8 * c + 4 * v + 3] = x.w;
          }
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kSteps * 2; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = static_cast<int>(imax(top & 0xFFFFu, top >> 16) >> 7);  // biased exponent
      // 2^(14 - (e - 127)), at most 2^110: that makes any bf16 number fp16 (subnormal ones
      // are multiples of 2^-133), and its reciprocal times scale_log2 stays normal
      const int up = imin(237, 127 + 14 - (e - 127));
      const float mul = __uint_as_float(static_cast<uint32_t>(up) << 23);
      qscale[nt] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        qf[nt][i][0] = pack_half2(bf16_lo(w[2 * i]) * mul, bf16_hi(w[2 * i]) * mul);
        qf[nt][i][1] = pack_half2(bf16_lo(w[2 * i + 1]) * mul, bf16_hi(w[2 * i + 1]) * mul);
      }
    }
    float fs[NT][2];  // the factors of this thread's two columns, rows 2 t4 and 2 t4 + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      fs[nt][0] = __shfl_sync(0xffffffffu, qscale[nt], 8 * t4);
      fs[nt][1] = __shfl_sync(0xffffffffu, qscale[nt], 8 * t4 + 4);
    }

    float o[NT][kSteps][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < kSteps; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
    float vref = 0.f, inv_vref = 0.f;  // O is held in units of vref

    for (int i = 0; i < seg; ++i) {
      cp_wait<kStages - 2>();
      __syncwarp();
      const uint8_t* st = ring + stage * C::kStage;
      const int key0 = (tile0 + i) * kKv8Tile + 16 * warp;
      const float ks = *static_cast<const volatile float*>(scales + 2 * stage);
      if (key0 < lim_hi && !(ks < 0.f)) {
        // ---- S^T = K q^T
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
        uint32_t k0[kWords], k1[kWords];
#pragma unroll
        for (int c = 0; c < kWords / 4; ++c) {
          const uint4 a = *reinterpret_cast<const uint4*>(st + piece<D>(key_of<D>(gq), t4 + 4 * c));
          const uint4 b = *reinterpret_cast<const uint4*>(st + piece<D>(key_of<D>(gq) + 8, t4 + 4 * c));
          k0[4 * c] = a.x, k0[4 * c + 1] = a.y, k0[4 * c + 2] = a.z, k0[4 * c + 3] = a.w;
          k1[4 * c] = b.x, k1[4 * c + 1] = b.y, k1[4 * c + 2] = b.z, k1[4 * c + 3] = b.w;
        }
#pragma unroll
        for (int w = 0; w < kSteps; ++w) {
          uint32_t a0, a1, a2, a3;
          codes_to_half2<kType>(k0[w], a0, a2);
          codes_to_half2<kType>(k1[w], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(s[nt], a0, a1, a2, a3, qf[nt][w][0], qf[nt][w][1]);
        }
        // ---- scores in log2 units; masked ones are -inf
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[nt][c] *= fs[nt][c & 1] * ks;
        if (key0 + 16 > lim_lo) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int r = rt * kRows + 8 * nt + 2 * t4 + (c & 1);
              const int key = key0 + key_of<D>(gq) + 8 * (c >> 1);
              if (key >= past + r / p.g) s[nt][c] = -INFINITY;
            }
        }
        // ---- running maximum, moved only when it grows by more than kSlack (the sum
        // rounded down: near 2^26 a maximum moves in steps of 8, and up is 8)
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) grow |= s[nt][c] > __fadd_rd(m[nt][c & 1], kSlack);
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float t = fmaxf(s[nt][c], s[nt][c + 2]);
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
              const float mn = fmaxf(m[nt][c], t);
              const float a = mn == -INFINITY ? 1.f : ex2_approx(m[nt][c] - mn);
              m[nt][c] = mn;
              l[nt][c] *= a;
#pragma unroll
              for (int j = 0; j < kSteps; ++j) {
                o[nt][j][c] *= a;
                o[nt][j][c + 2] *= a;
              }
            }
        }
        // ---- the V scale as a ratio to the reference
        const float vs = *static_cast<const volatile float*>(scales + 2 * stage + 1);
        if (vs > vref || (vs < vref * 0.000244140625f && vs > 0.f)) {
          const float top = vref > 0.f ? fmaxf(v_top[warp], vs) : vs, to = next_reference(vs, top);
          __syncwarp();
          if (lane == 0) v_top[warp] = top;
          __syncwarp();
          if (to != vref) {
            const float a = vref / to;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < kSteps; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[nt][j][c] *= a;
            vref = to;
            inv_vref = 1.f / to;
          }
        }
        const float vr = vs * inv_vref;
        // ---- P^T, by columns of keys
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // (two additions: m - kPShift would be rounded where m is large)
            const float ref = m[nt][c & 1] == -INFINITY ? 0.f : m[nt][c & 1];
            e[c] = ex2_approx((s[nt][c] - ref) + kPShift);
            l[nt][c & 1] += e[c];
          }
          pb[nt][0] = transpose8x8(pack_half2(e[0] * vr, e[1] * vr));
          pb[nt][1] = transpose8x8(pack_half2(e[2] * vr, e[3] * vr));
        }
        // ---- O^T += V^T P^T: the keys of matrix columns 2 t4, 2 t4 + 1 and 8 more;
        // lanes with `turn` read each pair in the other order (for the banks)
        // (at the causal edge a NaN code must not meet the weight 0 of rows that
        // do not see it)
        constexpr int kVWords = D / 32;  // words of a thread's share of a V row
        const int turn = D == 128 ? gq & 1 : (gq >> 1) & 1;
        uint32_t v[4][kVWords];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = key_of<D>(2 * t4 + ((r & 1) ^ turn)) + 8 * (r >> 1);
          if (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(st + 16 * D + piece<D>(row, gq));
            v[r][0] = x.x, v[r][1] = x.y, v[r][kVWords - 2] = x.z, v[r][kVWords - 1] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(st + 16 * D + piece<D>(row, gq >> 1) + 8 * (gq & 1));
            v[r][0] = x.x, v[r][1] = x.y;
          }
        }
        if (kType == STAR_KV8_E4M3 && key0 + 16 > lim_lo && here.r.T > 1) {
          bool nan = false;
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int w = 0; w < kVWords; ++w) nan |= nan_bytes(v[r][w]) != 0;
          if (__any_sync(0xffffffffu, nan)) {
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {
              bool sees[NT][2];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  sees[nt][c] = key0 + key_of<D>(k & 7) + (k & 8) < past + (rt * kRows + 8 * nt + 2 * t4 + c) / p.g;
#pragma unroll
              for (int w = 0; w < kVWords; ++w) {
                // k: matrix column, held by lane (k % 8) / 2 of this lane's four
                const int second = (k & 1) ^ turn;
                const uint32_t mine = second ? ((k & 8) ? v[3][w] : v[1][w]) : ((k & 8) ? v[2][w] : v[0][w]);
                const uint32_t bytes = nan_bytes(__shfl_sync(0xffffffffu, mine, (lane & 28) + ((k & 7) >> 1)));
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                      if (((bytes >> (8 * i)) & 1u) && sees[nt][c])
                        o[nt][2 * w + (i >> 1)][c + 2 * (i & 1)] = __uint_as_float(0x7FFFFFFFu);
              }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int w = 0; w < kVWords; ++w) v[r][w] &= ~nan_bytes(v[r][w]);
          }
        }
        // two keys' bytes interleaved become a fragment's pairs
        const uint32_t even = turn ? 0x1504u : 0x5140u, odd = turn ? 0x3726u : 0x7362u;
#pragma unroll
        for (int w = 0; w < kVWords; ++w)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t sel = x ? odd : even;
            uint32_t a0, a1, a2, a3;
            codes_to_half2<kType>(__byte_perm(v[0][w], v[1][w], sel), a0, a1);
            codes_to_half2<kType>(__byte_perm(v[2][w], v[3][w], sel), a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][2 * w + x], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
          }
      }
      // refill the stage read in the previous step (every lane is past it)
      issue(stage == 0 ? kStages - 1 : stage - 1);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    // the stage of the segment's last tile is refilled after the next tile: until
    // then it holds this warp's output
    const int free_stage = stage == 0 ? kStages - 1 : stage - 1;
    at += seg;
    cur.tile += seg - 1;
    if (at < end) advance(cur, at);

    // ---- the segment's end: join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 4);
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 8);
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 16);
        if (gq == 0) {
          wm[warp][8 * nt + 2 * t4 + c] = m[nt][c];
          wl[warp][8 * nt + 2 * t4 + c] = l[nt][c];
        }
      }
    __syncthreads();
    const bool whole = seg == here.r.tiles;
    // parts of a unit: a CTA's first segment goes to slot 0, a later one to 1
    const size_t part = 2 * static_cast<size_t>(blockIdx.x) + (at - seg == begin ? 0 : 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float w[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float M = -INFINITY;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) M = fmaxf(M, wm[x][8 * nt + 2 * t4 + c]);
        w[c] = M == -INFINITY ? 0.f : ex2_approx(m[nt][c] - M) * kKv8Join;
      }
      float* mine = reinterpret_cast<float*>(ring + free_stage * C::kStage);  // [8][D]
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          *reinterpret_cast<float2*>(mine + (2 * t4 + c) * D + gq * (D / 8) + 2 * j) =
              make_float2(o[nt][j][c] * w[c] * vref, o[nt][j][c + 2] * w[c] * vref);
      __syncthreads();
      const int n = tid / (D / 4), d = 4 * (tid % (D / 4));
      if (n < 8) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) M = fmaxf(M, wm[x][8 * nt + n]);
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
          const float4 y = *reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(smem + x * C::kRing + free_stage * C::kStage) + n * D + d);
          sum = make_float4(sum.x + y.x, sum.y + y.y, sum.z + y.z, sum.w + y.w);
          // (a maximum of -inf: nothing seen, a sum of 0, or only NaN)
          L += M == -INFINITY ? wl[x][8 * nt + n] : wl[x][8 * nt + n] * kKv8Join * ex2_approx(wm[x][8 * nt + n] - M);
        }
        if (8 * nt + n < rows) {
          if (whole) {
            const int r = rt * kRows + 8 * nt + n, head = kvh * p.g + r % p.g;
            const size_t token = here.r.q0 + r / p.g;
            const float inv = L != 0.f ? 1.f / L : 0.f;
            uint2 y;
            y.x = pack_bf16x2(sum.x * inv, sum.y * inv);
            y.y = pack_bf16x2(sum.z * inv, sum.w * inv);
            *reinterpret_cast<uint2*>(p.o + (token * p.Hq + head) * D + d) = y;
            if (d == 0 && p.lse)
              p.lse[static_cast<size_t>(head) * p.n_tokens + token] =
                  L != 0.f ? (M + (kKv8JoinShift - kPShift) + log2f(L)) * 0.6931471805599453f : -INFINITY;
          } else {
            *reinterpret_cast<float4*>(p.part_o + (part * kRows + 8 * nt + n) * D + d) = sum;
            if (d == 0)
              *reinterpret_cast<float2*>(p.part_ml + 2 * (part * kRows + 8 * nt + n)) = make_float2(M, L);
          }
        }
      }
      __syncthreads();
    }

    // ---- a cut unit's parts are joined by the CTA that finishes last, once
    // its own list is done: nobody waits for the counter here
    if (!whole) {
      if (tid == 0) {
        Cut& c = cuts[ncuts];
        c.first_tile = at - seg - tile0;
        c.row0 = rt * kRows;
        c.rows = rows;
        c.kvh = kvh;
        c.q0 = here.r.q0;
        // CTA of list index x: the largest c with floor(c * total / G) <= x
        c.c0 = static_cast<int>(((c.first_tile + 1ll) * G - 1) / total);
        c.c1 = static_cast<int>(((c.first_tile + static_cast<long long>(here.r.tiles)) * G - 1) / total);
        // a unit is cut at the end of its first CTA, and a CTA's end cuts one unit
        c.last = inc_acq_rel(p.counters + c.c0, c.c1 - c.c0) == static_cast<unsigned>(c.c1 - c.c0);
      }
      ++ncuts;
    }
  }
  cp_wait<0>();

  // ---- the joins, parts in order: a thread takes four elements of a row; where
  // rows leave threads over, they share out more than eight parts (one head of 64
  // over 30K tokens has 235: 14 us instead of 24; four parts shared out cost 0.4 us)
  if (ncuts > 0) __syncthreads();
  struct Sum {
    float4 o;
    float M, L;
  };
  Sum* shared_sums = reinterpret_cast<Sum*>(smem);  // the rings are done with
  for (int i = 0; i < ncuts; ++i) {
    const Cut c = cuts[i];
    if (!c.last) continue;
    // the unit's first part is its CTA's first segment only if the CTA begins there
    const int begin0 = static_cast<int>(static_cast<long long>(c.c0) * total / G);
    const int slot0 = begin0 == c.first_tile ? 0 : 1;
    const int items = c.rows * (D / 4), parts = c.c1 - c.c0 + 1;
    const int shares = parts > 8 ? imax(1, kThreads / items) : 1;
    auto add = [&](Sum& t, const float2* ml, const float4* y, int n) {
      float mn = t.M;
      for (int j = 0; j < n; ++j) mn = fmaxf(mn, ml[j].x);
      const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: sums of 0 (or NaN)
      const float a = ex2_approx(t.M - ref);
      t.o = make_float4(t.o.x * a, t.o.y * a, t.o.z * a, t.o.w * a);
      t.L = t.M == -INFINITY ? t.L : t.L * a;
      t.M = mn;
      for (int j = 0; j < n; ++j) {
        const float w = ex2_approx(ml[j].x - ref);
        t.o = make_float4(t.o.x + y[j].x * w, t.o.y + y[j].y * w, t.o.z + y[j].z * w, t.o.w + y[j].w * w);
        t.L += ml[j].x == -INFINITY ? ml[j].y : ml[j].y * w;
      }
    };
    for (int e0 = tid; e0 < shares * items; e0 += kThreads) {
      const int share = shares > 1 ? e0 / items : 0, e = e0 - share * items;
      const int n = e / (D / 4), d = 4 * (e % (D / 4));
      auto part = [&](int x) { return (2 * static_cast<size_t>(x) + (x == c.c0 ? slot0 : 0)) * kRows + n; };
      Sum t{make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f};
      const int x1 = c.c0 + (share + 1) * parts / shares;
      for (int x0 = c.c0 + share * parts / shares; x0 < x1; x0 += 8) {  // (eight parts' loads at a time)
        float2 ml[8];
        float4 y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ml[j] = make_float2(-INFINITY, 0.f);
          y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (x0 + j < x1) {
            ml[j] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + 2 * part(x0 + j)));
            y[j] = __ldcg(reinterpret_cast<const float4*>(p.part_o + part(x0 + j) * D + d));
          }
        }
        add(t, ml, y, 8);
      }
      if (shares > 1) {
        shared_sums[e0] = t;
        continue;
      }
      finish_row(p, c, n, d, D, t.o, t.M, t.L);
    }
    if (shares > 1) {
      __syncthreads();
      if (tid < items) {
        Sum t = shared_sums[tid];
        for (int share = 1; share < shares; ++share) {
          const Sum u = shared_sums[share * items + tid];
          const float2 ml = make_float2(u.M, u.L);
          add(t, &ml, &u.o, 1);
        }
        finish_row(p, c, tid / (D / 4), 4 * (tid % (D / 4)), D, t.o, t.M, t.L);
      }
      __syncthreads();
    }
  }
}

namespace {
template <int D, int kType, int NT>
cudaError_t launch(const Kv8AttendParams& p, int sms, cudaStream_t stream) {
  const size_t smem = Cfg<D>::kPrefix + (p.B + 1) * sizeof(int);
  static std::atomic<bool> raised[64];  // this variant's shared-memory limit, by device
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !raised[dev].load(std::memory_order_acquire)) {
    cudaError_t e = cudaFuncSetAttribute(
        kv8_decode_kernel<D, kType, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        static_cast<int>(Cfg<D>::kPrefix + (kMaxRequests + 1) * sizeof(int)));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) raised[dev].store(true, std::memory_order_release);
  }
  const int grid = imin(kKv8MaxCtas, ctas_per_sm(D, NT) * sms);
  return launch_after(kv8_decode_kernel<D, kType, NT>, dim3(grid), kThreads, smem, stream, p);
}
}  // namespace

cudaError_t launch_kv8_decode(const Kv8AttendParams& p, int D, int kv_type, int rows, int sms,
                              cudaStream_t stream) {
  const bool e4m3 = kv_type == STAR_KV8_E4M3, one = rows == 8;
  if (D == 128) {
    if (e4m3) return one ? launch<128, STAR_KV8_E4M3, 1>(p, sms, stream) : launch<128, STAR_KV8_E4M3, 2>(p, sms, stream);
    return one ? launch<128, STAR_KV8_INT8, 1>(p, sms, stream) : launch<128, STAR_KV8_INT8, 2>(p, sms, stream);
  }
  if (e4m3) return one ? launch<64, STAR_KV8_E4M3, 1>(p, sms, stream) : launch<64, STAR_KV8_E4M3, 2>(p, sms, stream);
  return one ? launch<64, STAR_KV8_INT8, 1>(p, sms, stream) : launch<64, STAR_KV8_INT8, 2>(p, sms, stream);
}

}  // namespace star
