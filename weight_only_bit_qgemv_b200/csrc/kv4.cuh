// The 4-bit cache's layout and the helpers that its kernels and the prompt attention share:
// element types, the softmax's exponential, and the sequence that a packed row belongs to.
//
// codes  [pages, kv_heads, 2 (key, value), page, dim / 2] bytes
// scales [pages, kv_heads, page, 2 (key, value), dim / 32] binary16
// A row is dim / 32 blocks of 32 codes, packed as int4 weights are (element 2j of a block in the
// low half of its byte j). Within a row the pieces are stored so that the attention kernel's
// matrix operands come out of shared memory with one wide load a row:
//   key    32-bit word t of block b at word t * blocks + b        (t 0..3: one quad lane's codes)
//   value  16-bit halfword g of block b at halfword g * blocks + b (g 0..7: one column's codes)
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "woq.h"

namespace woq {

// 2^x, within 2^-22 of it; below 2^-126 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four consecutive elements of one row, as float.
__device__ __forceinline__ float4 load4(const void *base, int64_t at, int dtype) {
  if (dtype == WOQ_F32) return *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
  const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + at);
  float2 a, b;
  if (dtype == WOQ_F16) {
    a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
    b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
  } else {
    a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w.x));
    b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w.y));
  }
  return make_float4(a.x, a.y, b.x, b.y);
}

// Two floats rounded to nearest even in a 16-bit type.
__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype) {
  if (dtype == WOQ_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void store4(void *base, int64_t at, int dtype, float4 v) {
  if (dtype == WOQ_F32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(base) + at) = v;
  } else {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + at) =
        make_uint2(pack2(v.x, v.y, dtype), pack2(v.z, v.w, dtype));
  }
}

// Row t of a packed batch is row t - cu[b] of the sequence b with cu[b] <= t < cu[b + 1]; -1 if
// no sequence has it. Any contents of cu keep the reads inside [0, batch].
__device__ __forceinline__ int sequence_of(const int32_t *cu, int batch, int64_t t) {
  int lo = 0, hi = batch;  // cu[lo] <= t (checked at the end), cu[hi] > t or hi == batch
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return cu[lo] <= t && t < cu[lo + 1] ? lo : -1;
}

}  // namespace woq
