// sd_kv.cuh -- the paged 8-bit cache as its kernels see it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sd_common.cuh"

namespace sdk {

// Element [page][slot][head][d] of K and V at page * st_block + slot * st_tok + head * st_head + d
// (64-bit: a long cache passes 2^32 elements); scales [num_blocks][Hkv].
struct KvCache {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  long st_block, st_tok, st_head;
  int num_blocks, log2_bs, Hkv, D;
};

constexpr float kMinScale = 7.8886090522101181e-31f;  // 2^-100, the smallest scale a page is given

// Two e4m3 values as two fp32 (exact).
__device__ __forceinline__ float2 e4m3x2_to_f32(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Two fp32 to e4m3 (lo in the low byte): to nearest even, beyond +-448 (infinities too) to +-448,
// NaN to NaN.
__device__ __forceinline__ uint16_t f32_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four fp32 to e4m3, v0 in the lowest byte, to nearest (halves away from zero), NaN to NaN. The
// instruction rounds by adding bits that it is given; 0x8001 is one half for the first of a pair and,
// read backwards, for the second. Four values take the time that two take with the instruction
// that rounds to nearest by itself (4 cycles of a warp on one scheduler, measured).
__device__ __forceinline__ uint32_t f32_to_e4m3x4(float v0, float v1, float v2, float v3) {
  uint32_t r;
  asm("cvt.rs.satfinite.e4m3x4.f32 %0, {%1, %2, %3, %4}, %5;"
      : "=r"(r)
      : "f"(v3), "f"(v2), "f"(v1), "f"(v0), "r"(0x80018001u));
  return r;
}

// Four fp32 of 3 significant bits to e5m2, exactly from 2^-14 to 57344, NaN to NaN.
__device__ __forceinline__ uint32_t f32_to_e5m2x4(float v0, float v1, float v2, float v3) {
  uint32_t r;
  asm("cvt.rs.satfinite.e5m2x4.f32 %0, {%1, %2, %3, %4}, %5;"
      : "=r"(r)
      : "f"(v3), "f"(v2), "f"(v1), "f"(v0), "r"(0x80018001u));
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace sdk
