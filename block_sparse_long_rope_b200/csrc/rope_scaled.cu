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
// product and sum stay below 2^-22). The bound is taken as 2^-23 of 2 |m| (|a| + |b|),
// which is infinite where a product could leave fp32: such a pair goes to fp64 too.
//
// Bound: HBM, 4 bytes an element. A unit is 16 elements of a head row: 8 pairs
// (of the half layout two 16-byte vectors rot/2 apart, of the interleaved one two
// neighbours) or 16 elements to copy. A thread keeps one unit of one token and
// walks over heads, its 8 cosines and sines in registers; the CTA builds them
// once in shared memory, with their fp64 values for the slow path. The rounding
// test takes both ends of the error interval as packed bf16 pairs and branches
// once for a unit's 8 pairs. 16K tokens x 40 heads of 128 (336 MB): 62.2 us, 5.4
// TB/s, two thirds of the issue slots (interleaved 64.8; half of the head 62.2, since
// copying lanes wait for the pairs of their warp); 16 tokens 3.1 us. A CTA's rows are 8
// tokens of 4 heads (8 at D 64): with fewer heads than that threads idle, and 16K
// tokens of 5 heads take 21.8 us, of one 18.4.
#include <cmath>

#include "kv8_kernels.cuh"
#include "rope_math.cuh"
#include "star_index.cuh"

namespace star {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;
// Heads of a thread in flight; with 64 registers, four CTAs of an SM hide the rest
// (63.1 us for 16K tokens x 40 heads; the next heads' loads ahead of the
// arithmetic take 80 registers, three CTAs and 65.5 us).
constexpr int kBatch = 2;

// Both outputs of a pair in fp64 (first in the lower half), rounded once.
__device__ __noinline__ uint32_t scaled_pair_exact(float a, float b, double c, double s) {
  const double ad = a, bd = b;
  const uint32_t o0 = pack_bf16x2(f32_round_odd(ad * c - bd * s), 0.f) & 0xFFFFu;
  const uint32_t o1 = pack_bf16x2(f32_round_odd(bd * c + ad * s), 0.f) & 0xFFFFu;
  return o0 | (o1 << 16);
}

}  // namespace

template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 4) rope_scaled_kernel(const __grid_constant__ RopeScaledParams p) {
  constexpr int kUnits = D / 16;          // threads of a head row
  constexpr int kGroups = kThreads / kUnits;
  __shared__ double2 exact[kMaxTok][64];  // m (cos, sin)
  // their fp32 roundings, 8 pairs of a unit and a gap: units lie in other banks
  __shared__ float2 tab[kMaxTok][kUnits * 10];
  after_previous();
  const int half = p.rot / 2;
  const int tok0 = blockIdx.x * p.tpc, ntok = imin(p.tpc, p.S - tok0);
  const int b = blockIdx.y;
  const int u = threadIdx.x % kUnits, g = threadIdx.x / kUnits;
  const int per = kGroups / p.tpc;        // threads that share a token's heads
  const int t = g / per;
  const int h_end = imin(p.H, static_cast<int>(blockIdx.z + 1) * p.hpc);
  int h = blockIdx.z * p.hpc + g % per;
  const bool pairs = 16 * u < p.rot;
  const int first = !pairs ? 16 * u : kInter ? 16 * u : 8 * u;    // this unit's two vectors
  const int second = !pairs || kInter ? first + 8 : first + half;
  const bool mine = t < ntok && (pairs || p.copy_rest);
  const __nv_bfloat16* x = p.x + b * p.xs[0] + (tok0 + static_cast<long long>(t)) * p.xs[1] + h * p.xs[2] + first;
  __nv_bfloat16* y = p.y + b * p.ys[0] + (tok0 + static_cast<long long>(t)) * p.ys[1] + h * p.ys[2] + first;
  const long long x_step = per * p.xs[2], y_step = per * p.ys[2];  // to this thread's next head
  const int gap = second - first;

  uint4 lo[kBatch], hi[kBatch];
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < kBatch; ++i, x += x_step)
      if (mine && h + i * per < h_end) {
        lo[i] = *reinterpret_cast<const uint4*>(x);
        hi[i] = *reinterpret_cast<const uint4*>(x + gap);
      }
  };
  load();
  for (int e = threadIdx.x; e < ntok * half; e += kThreads) {
    const int tt = e / half, i = e - tt * half;
    const long long pos = p.pos ? p.pos[b * p.pos_stride_b + tok0 + tt] : p.pos0 + tok0 + tt;
    double c, s;
    rope_angle(pos, p.inv_freq[i], &c, &s);
    c *= p.mscale;
    s *= p.sign * p.mscale;
    exact[tt][i] = make_double2(c, s);
    tab[tt][i + 2 * (i / 8)] = make_float2(static_cast<float>(c), static_cast<float>(s));
  }
  __syncthreads();
  if (!mine) return;
  float c[8], s[8];
  if (pairs) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 v = *reinterpret_cast<const float4*>(&tab[t][10 * u + 2 * j]);
      c[2 * j] = v.x, s[2 * j] = v.y, c[2 * j + 1] = v.z, s[2 * j + 1] = v.w;
    }
  }
  const float reach = 2.f * p.mscale_abs;
  constexpr float kErr = 1.1920929e-07f;  // 2^-23

  // Units of a row's copied part and its pairs sit in different lanes of a warp
  while (h < h_end) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i, y += y_step) {
      if (h + i * per >= h_end) break;
      uint32_t* l = reinterpret_cast<uint32_t*>(&lo[i]);
      uint32_t* r = reinterpret_cast<uint32_t*>(&hi[i]);
      if (pairs) {
        // pair j: elements a_j, b_j and both outputs' interval ends, packed (first,
        // second); they agree unless a rounding boundary lies between
        auto elem = [&](int j, float& a, float& bb) {
          if (kInter) {
            const uint32_t w = j < 4 ? l[j] : r[j - 4];
            a = bf16_lo(w), bb = bf16_hi(w);
          } else {
            a = j & 1 ? bf16_hi(l[j >> 1]) : bf16_lo(l[j >> 1]);
            bb = j & 1 ? bf16_hi(r[j >> 1]) : bf16_lo(r[j >> 1]);
          }
        };
        uint32_t out[8], bad = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float a, bb;
          elem(j, a, bb);
          const float t = reach * (fabsf(a) + fabsf(bb));
          const float y0 = fmaf(a, c[j], -(bb * s[j])), y1 = fmaf(bb, c[j], a * s[j]);
          out[j] = pack_bf16x2(fmaf(t, -kErr, y0), fmaf(t, -kErr, y1));
          if (out[j] != pack_bf16x2(fmaf(t, kErr, y0), fmaf(t, kErr, y1))) bad |= 1u << j;
        }
        if (bad) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (!((bad >> j) & 1u)) continue;
            float a, bb;
            elem(j, a, bb);
            const double2 cs = exact[t][8 * u + j];
            out[j] = scaled_pair_exact(a, bb, cs.x, cs.y);
          }
        }
        if (kInter) {
#pragma unroll
          for (int j = 0; j < 4; ++j) l[j] = out[j], r[j] = out[4 + j];
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            l[j] = __byte_perm(out[2 * j], out[2 * j + 1], 0x5410);  // first outputs
            r[j] = __byte_perm(out[2 * j], out[2 * j + 1], 0x7632);
          }
        }
      }
      *reinterpret_cast<uint4*>(y) = lo[i];
      *reinterpret_cast<uint4*>(y + gap) = hi[i];
    }
    h += kBatch * per;
    load();
  }
}

cudaError_t launch_rope_scaled(const RopeScaledParams& p_in, bool interleaved, cudaStream_t stream) {
  RopeScaledParams p = p_in;
  const int groups = kThreads / (p.D / 16);  // (token, head) rows of a CTA at a time
  // 8 tokens a CTA share their table's cost; a short call takes fewer, then fewer
  // heads, so that its grid still covers the GPU
  p.tpc = kMaxTok;
  while (p.tpc > 1 && (long long)ceil_div(p.S, p.tpc) * p.B < 2 * 148) p.tpc /= 2;
  p.hpc = (long long)ceil_div(p.S, p.tpc) * p.B < 148 ? imin(p.H, groups / p.tpc) : p.H;
  const dim3 grid(ceil_div(p.S, p.tpc), p.B, ceil_div(p.H, p.hpc));
  if (p.D == 128)
    return interleaved ? launch_after(rope_scaled_kernel<128, true>, grid, kThreads, 0, stream, p)
                       : launch_after(rope_scaled_kernel<128, false>, grid, kThreads, 0, stream, p);
  return interleaved ? launch_after(rope_scaled_kernel<64, true>, grid, kThreads, 0, stream, p)
                     : launch_after(rope_scaled_kernel<64, false>, grid, kThreads, 0, stream, p);
}

}  // namespace star
