// Rotary positions with given inverse frequencies: half or interleaved pairs,
// over all or the leading rot elements of a head, forward or transposed.
//
//   y_first  = m (a cos - b sin),  y_second = m (b cos + a sin),  angle p f_i
// with the sine's sign turned for the transpose (the gradient).
//
// Rounding is rope_math.cuh's: fp64 angles and sine/cosine, the rotation in
// fp32 with the error bound E = 2^-22 |m| (|a| + |b|), and Ziv's test; an
// element within E of a rounding boundary is recomputed in fp64 and rounded
// once. m is folded into the fp32 cosine and sine, one more rounding of 2^-25
// that the bound has room for (2^-25 for cos, 2^-25 for m cos, two of 2^-24 for
// product and sum stay below 2^-22).
//
// Bound: HBM, 4 bytes an element. A CTA covers tpc tokens of hpc heads: it
// issues its first loads, builds the (cos, sin) table of its tokens in shared
// memory while they are on the way, then streams 16-byte vectors, kBatch of
// them a thread at once.
#include <cmath>

#include "kv8_kernels.cuh"
#include "rope_math.cuh"
#include "star_index.cuh"

namespace star {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;
constexpr int kBatch = 4;  // units of a thread in flight

// The rare slow path, out of line: both outputs of a pair in fp64.
__device__ __noinline__ uint32_t scaled_pair_exact(float a, float b, long long pos, double f,
                                                   double mscale, double sign) {
  double c, s;
  rope_angle(pos, f, &c, &s);
  s *= sign;
  const double ad = a, bd = b;
  const uint32_t o0 = pack_bf16x2(f32_round_odd((ad * c - bd * s) * mscale), 0.f) & 0xFFFFu;
  const uint32_t o1 = pack_bf16x2(f32_round_odd((bd * c + ad * s) * mscale), 0.f) & 0xFFFFu;
  return o0 | (o1 << 16);
}

}  // namespace

// A unit is one thread's share of a head row: of the rotated part a 16-byte
// vector and its partner rot/2 elements on (half), or one 16-byte vector of
// four pairs (interleaved); of the rest one vector.
template <bool kInter>
__global__ void __launch_bounds__(kThreads) rope_scaled_kernel(const __grid_constant__ RopeScaledParams p) {
  __shared__ float2 tab[kMaxTok][64];  // m (cos, sin)
  const int half = p.rot / 2;
  const int tok0 = blockIdx.x * p.tpc, ntok = imin(p.tpc, p.S - tok0);
  const int h0 = blockIdx.z * p.hpc, nh = imin(p.hpc, p.H - h0);
  const int b = blockIdx.y;
  const unsigned rot_units = kInter ? p.rot / 8 : p.rot / 16;
  const unsigned per_row = rot_units + (p.copy_rest ? (p.D - p.rot) / 8 : 0);
  const unsigned per_tok = per_row * nh, units = per_tok * ntok;
  // u / per_tok and rem / per_row by one multiply-high (u * divisor < 2^32)
  const unsigned magic_t = 0xFFFFFFFFu / per_tok + 1u, magic_r = 0xFFFFFFFFu / per_row + 1u;
  const __nv_bfloat16* xb = p.x + b * p.xs[0];
  __nv_bfloat16* yb = p.y + b * p.ys[0];

  uint4 lo[kBatch], hi[kBatch];
  int tok[kBatch], row[kBatch], unit[kBatch];
  auto load = [&](unsigned u0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const unsigned u = u0 + i * kThreads;
      if (u >= units) {
        tok[i] = -1;
        continue;
      }
      const unsigned t = per_tok == 1 ? u : __umulhi(u, magic_t);
      const unsigned rem = u - t * per_tok;
      const unsigned h = per_row == 1 ? rem : __umulhi(rem, magic_r);
      tok[i] = t;
      row[i] = h0 + h;
      unit[i] = rem - h * per_row;
      const __nv_bfloat16* xr = xb + (tok0 + static_cast<long long>(t)) * p.xs[1] + row[i] * p.xs[2];
      if (unit[i] < static_cast<int>(rot_units)) {
        lo[i] = *reinterpret_cast<const uint4*>(xr + 8 * unit[i]);
        if (!kInter) hi[i] = *reinterpret_cast<const uint4*>(xr + half + 8 * unit[i]);
      } else {
        lo[i] = *reinterpret_cast<const uint4*>(xr + p.rot + 8 * (unit[i] - rot_units));
      }
    }
  };
  load(threadIdx.x);

  auto position = [&](int t) -> long long {
    return p.pos ? p.pos[b * p.pos_stride_b + tok0 + t] : p.pos0 + tok0 + t;
  };
  for (int e = threadIdx.x; e < ntok * half; e += kThreads) {
    const int t = e / half, i = e - t * half;
    double c, s;
    rope_angle(position(t), p.inv_freq[i], &c, &s);
    tab[t][i] = make_float2(static_cast<float>(c * p.mscale), static_cast<float>(s * p.sign * p.mscale));
  }
  __syncthreads();

  auto pair = [&](float a, float bb, int t, int i) -> uint32_t {
    const float2 cs = tab[t][i];
    const float e = 2.3841858e-07f * p.mscale_abs * (fabsf(a) + fabsf(bb));
    const float y0 = fmaf(a, cs.x, -(bb * cs.y)), y1 = fmaf(bb, cs.x, a * cs.y);
    const uint32_t r0 = pack_bf16x2(y0 - e, y0 + e), r1 = pack_bf16x2(y1 - e, y1 + e);
    if ((r0 & 0xFFFFu) == (r0 >> 16) && (r1 & 0xFFFFu) == (r1 >> 16))
      return __byte_perm(r0, r1, 0x5410);
    return scaled_pair_exact(a, bb, position(t), p.inv_freq[i], p.mscale, p.sign);
  };
  for (unsigned u0 = threadIdx.x; u0 < units; u0 += kBatch * kThreads) {
    if (u0 != threadIdx.x) load(u0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (tok[i] < 0) continue;
      const int t = tok[i];
      __nv_bfloat16* yr = yb + (tok0 + static_cast<long long>(t)) * p.ys[1] + row[i] * p.ys[2];
      if (unit[i] >= static_cast<int>(rot_units)) {
        *reinterpret_cast<uint4*>(yr + p.rot + 8 * (unit[i] - rot_units)) = lo[i];
        continue;
      }
      const uint32_t l[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w};
      uint32_t ol[4], oh[4];
      if (kInter) {
#pragma unroll
        for (int w = 0; w < 4; ++w) ol[w] = pair(bf16_lo(l[w]), bf16_hi(l[w]), t, 4 * unit[i] + w);
      } else {
        const uint32_t r[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int i0 = 8 * unit[i] + 2 * w;
          const uint32_t p0 = pair(bf16_lo(l[w]), bf16_lo(r[w]), t, i0);
          const uint32_t p1 = pair(bf16_hi(l[w]), bf16_hi(r[w]), t, i0 + 1);
          ol[w] = __byte_perm(p0, p1, 0x5410);  // first outputs of both pairs
          oh[w] = __byte_perm(p0, p1, 0x7632);
        }
        *reinterpret_cast<uint4*>(yr + half + 8 * unit[i]) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
      }
      *reinterpret_cast<uint4*>(yr + 8 * unit[i]) = make_uint4(ol[0], ol[1], ol[2], ol[3]);
    }
  }
}

cudaError_t launch_rope_scaled(const RopeScaledParams& p_in, bool interleaved, cudaStream_t stream) {
  RopeScaledParams p = p_in;
  // 8 tokens a CTA share one table; a short call takes fewer, then fewer heads,
  // so that its grid still covers the GPU
  p.tpc = kMaxTok;
  while (p.tpc > 1 && (long long)ceil_div(p.S, p.tpc) * p.B < 2 * 148) p.tpc /= 2;
  const int row_units = p.rot / (interleaved ? 8 : 16) + (p.copy_rest ? (p.D - p.rot) / 8 : 0);
  // the multiply-high division needs units * divisor < 2^32: 8 * 8192 * 8192
  p.hpc = imin(p.H, 8192 / row_units);
  if (p.tpc == 1 && (long long)p.S * p.B < 148) p.hpc = imax(1, kThreads / row_units);
  const dim3 grid(ceil_div(p.S, p.tpc), p.B, ceil_div(p.H, p.hpc));
  if (interleaved)
    rope_scaled_kernel<true><<<grid, kThreads, 0, stream>>>(p);
  else
    rope_scaled_kernel<false><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace star
