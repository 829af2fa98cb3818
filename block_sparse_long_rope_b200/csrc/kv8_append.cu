// New tokens' K and V rows into 8-bit pages, one scale per page and head.
//
// A run is a span of one request's new tokens within one page. For each head
// with amax the largest finite magnitude of the run and top the largest code
// (448 or 127):
//   s = 2^ceil(log2(amax / top)), at least 2^-100
//   s' = s for a run that starts its page, max(old, s) otherwise
//   code = nearest(x / s'); earlier rows where s' grew: nearest(code * old / s')
// Powers of two make the division exact, so a code is rounded once, and an e4m3
// row whose scale grows keeps its values down to the subnormal codes. An e4m3
// code has the same relative step at any scale: the power of two costs it
// nothing; int8 gives up at most one bit of amax / 127.
//
// Bound: HBM, 2 bytes read and 1 written an element. A CTA takes one (run,
// head, K or V): its threads hold the whole piece in registers between the
// maximum and the rounding, so each element is read once. 16K tokens of 8 heads of
// 128, K and V (101 MB): 18.9 us with other inputs each time (int8, whose conversions
// are four to e4m3's two packed ones: 23.9), 15.8 us for one graph replayed, part of
// whose inputs stay in the L2; 16 decode rows 2.5 us.
#include "kv8_codes.cuh"
#include "kv8_kernels.cuh"
#include "star_index.cuh"

namespace star {

namespace {

constexpr int kThreads = 128;

// 2^ceil(log2(amax / top)) for a finite bf16 magnitude given by its bits: with
// amax = m 2^e, top = t 2^f (m, t in [1, 2)) it is 2^(e - f), doubled if m > t.
template <int kType>
__device__ __forceinline__ float pow2_scale(uint32_t bits) {
  constexpr int f = kType == STAR_KV8_E4M3 ? 8 : 6;
  constexpr uint32_t t = kType == STAR_KV8_E4M3 ? 0x60u : 0x7Eu;  // mantissas of 1.75, 1.984375
  // a subnormal amax lies far below the floor of 2^-100
  const int e = static_cast<int>(bits >> 7) - 127 - f + ((bits & 0x7Fu) > t ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(imax(e, -100) + 127) << 23);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

template <int kType, int D, int kVec>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const __grid_constant__ Kv8AppendParams p) {
  constexpr int kRowVecs = D / 8;  // 16-byte vectors of a bf16 row
  __shared__ uint32_t red[kThreads / 32];
  after_previous();
  const int u = blockIdx.x, h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int t0 = p.run_start[u], t1 = p.run_start[u + 1];
  if (t0 >= t1) return;
  const int P = 1 << p.page_shift;
  if (t0 < 0 || t1 > p.n_tokens) {
    if (threadIdx.x == 0) atomicOr(p.status, kDevBounds);
    return;
  }
  const int slot = p.slot[t0];
  if (slot < 0) return;
  const int page = slot >> p.page_shift, row0 = slot & (P - 1);
  const int rows = t1 - t0;
  if (page >= p.num_pages || row0 + rows > P) {
    if (threadIdx.x == 0) atomicOr(p.status, kDevBounds);
    return;
  }
  const size_t unit = static_cast<size_t>(page) * p.Hkv + h;
  float* scale_at = (is_v ? p.v_scale : p.k_scale) + unit;
  const float old = row0 > 0 ? *scale_at : 0.f;
  const __nv_bfloat16* src = is_v ? p.v + h * p.vs[1] : p.k + h * p.ks[1];
  const long long stride = is_v ? p.vs[0] : p.ks[0];
  uint8_t* dst = (is_v ? p.v_pages : p.k_pages) + (unit << p.page_shift) * D;

  uint4 x[kVec];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int e = threadIdx.x + i * kThreads, r = e / kRowVecs, c = e % kRowVecs;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows)
      x[i] = *reinterpret_cast<const uint4*>(src + (t0 + static_cast<long long>(r)) * stride + 8 * c);
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const uint32_t a = max_u16x2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu);
    const uint32_t b = max_u16x2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu);
    top = max_u16x2(top, max_u16x2(a, b));
  }
  auto block_max = [&](uint32_t m) -> uint32_t {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
    __syncthreads();  // red may still be read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max_u16x2(m, red[w]);
    return imax(static_cast<int>(m & 0xFFFFu), static_cast<int>(m >> 16));
  };
  uint32_t amax = block_max(top);
  if (amax >= 0x7F80u) {  // infinities or NaN: the largest finite magnitude (rare)
    top = 0;
    auto finite = [](uint32_t w) -> uint32_t {
      uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
      if (lo >= 0x7F80u) lo = 0;
      if (hi >= 0x7F80u) hi = 0;
      return lo | (hi << 16);
    };
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      top = max_u16x2(top, max_u16x2(max_u16x2(finite(x[i].x), finite(x[i].y)),
                                     max_u16x2(finite(x[i].z), finite(x[i].w))));
    amax = block_max(top);
  }
  const float s = fmaxf(pow2_scale<kType>(amax), old);
  // a product with 1 / s is exact for a power of two; a caller's own old scale
  // may be another number and takes the division
  const float inv = 1.f / s;
  const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0;
  auto code4 = [&](uint32_t a, uint32_t b) -> uint32_t {
    const float f[4] = {bf16_lo(a), bf16_hi(a), bf16_lo(b), bf16_hi(b)};
    if (pow2) return to_codes<kType>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    return to_codes<kType>(__fdiv_rn(f[0], s), __fdiv_rn(f[1], s), __fdiv_rn(f[2], s), __fdiv_rn(f[3], s));
  };
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int e = threadIdx.x + i * kThreads, r = e / kRowVecs, c = e % kRowVecs;
    if (r >= rows) continue;
    uint2 q;
    q.x = code4(x[i].x, x[i].y);
    q.y = code4(x[i].z, x[i].w);
    *reinterpret_cast<uint2*>(dst + static_cast<size_t>(row0 + r) * D + 8 * c) = q;
  }
  if (row0 > 0 && s > old) {
    const float ratio = old > 0.f ? old / s : 0.f;
    for (int e = threadIdx.x; e < row0 * (D / 16); e += kThreads) {
      uint4 w = reinterpret_cast<uint4*>(dst)[e];
      uint32_t* v = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        codes_to_half2<kType>(v[i], lo, hi);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        v[i] = to_codes<kType>(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
      }
      reinterpret_cast<uint4*>(dst)[e] = w;
    }
  }
  if (threadIdx.x == 0) *scale_at = s;  // every thread read the old one before block_max's barrier
}

template <int kType, int D>
cudaError_t launch_type(const Kv8AppendParams& p, cudaStream_t stream) {
  const dim3 grid(p.run_cap, p.Hkv, 2);
  switch ((D << p.page_shift) / 8 / kThreads) {  // vectors of a thread for a full page
    case 1: return launch_after(kv8_append_kernel<kType, D, 1>, grid, kThreads, 0, stream, p);
    case 2: return launch_after(kv8_append_kernel<kType, D, 2>, grid, kThreads, 0, stream, p);
    case 4: return launch_after(kv8_append_kernel<kType, D, 4>, grid, kThreads, 0, stream, p);
    case 8: return launch_after(kv8_append_kernel<kType, D, 8>, grid, kThreads, 0, stream, p);
    default: return launch_after(kv8_append_kernel<kType, D, 16>, grid, kThreads, 0, stream, p);
  }
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendParams& p, int D, int kv_type, cudaStream_t stream) {
  if (p.run_cap <= 0) return cudaSuccess;
  if (kv_type == STAR_KV8_E4M3)
    return D == 128 ? launch_type<STAR_KV8_E4M3, 128>(p, stream) : launch_type<STAR_KV8_E4M3, 64>(p, stream);
  return D == 128 ? launch_type<STAR_KV8_INT8, 128>(p, stream) : launch_type<STAR_KV8_INT8, 64>(p, stream);
}

}  // namespace star
