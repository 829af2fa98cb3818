// 8-bit codes of the paged cache: conversion of pairs to fp16 for the tensor
// cores (every code of either type is an fp16 value) and to the code range.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "star.h"
#include "star_common.cuh"

namespace star {

// Four codes of one 32-bit word as two fp16 pairs, in order.
template <int kType>
__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (kType == STAR_KV8_E4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // the byte x + 128 under the fp16 exponent of 1024 is 1152 + x
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
  }
}

// Nearest codes of four values already divided by the scale (ties to even,
// saturating; NaN: the NaN code, or 0 for int8).
template <int kType>
__device__ __forceinline__ uint32_t to_codes(float a, float b, float c, float d) {
  uint32_t r;
  if (kType == STAR_KV8_E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
  } else {
    auto one = [](float x) -> uint32_t {
      if (x != x) return 0u;
      return static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(x, -127.f), 127.f))) & 0xFFu;
    };
    r = one(a) | (one(b) << 8) | (one(c) << 16) | (one(d) << 24);
  }
  return r;
}

}  // namespace star
