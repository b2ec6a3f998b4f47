// Device helpers of the selective scan's kernels.
#pragma once

#include "device_common.h"
#include "kernels.h"

namespace mlstm {

__device__ __forceinline__ float scan_load(const bf16_t* p) { return bf16_to_f32(p->bits); }
__device__ __forceinline__ float scan_load(const float* p) { return *p; }
__device__ __forceinline__ uint16_t to_bf16(float x) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }
__device__ __forceinline__ void scan_store(bf16_t* p, float x) { p->bits = to_bf16(x); }
__device__ __forceinline__ void scan_store(float* p, float x) { *p = x; }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// exp(d A) with A2 = A log2(e).  The instruction is low by 1e-9 to 6e-9 of the
// value on average near exponents of zero (rounding apart, over 2^20 values), and
// a slow state multiplies thousands of these; the addend, for free in the fused
// product, takes that out.  d = 0 gives 1.
__device__ __forceinline__ float decay(float d, float A2) { return exp2_fast(fmaf(d, A2, 4e-9f)); }

// The value is formed here, not behind what follows.
__device__ __forceinline__ void formed(float& x) { asm volatile("" : "+v"(x)); }

// 1 / (1 + e^-x)
__device__ __forceinline__ float scan_sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp2_fast(-kLog2e * x));
}

// log(1 + e^x) = max(x, 0) + log(1 + e),  e = e^-|x| in (0, 1].  With s = e /
// (2 + e) <= 1/3, log(1 + e) = 2 atanh(s) = 2 s (1 + s^2/3 + s^4/5 + ...); the
// bracket is a polynomial in s^2 fitted at Chebyshev points of [0, 1/9], off by
// 4e-9.  A small e keeps its digits (log(1 + e) of a rounded 1 + e does not).
__device__ __forceinline__ float softplus(float x) {
  const float e = exp2_fast(-kLog2e * fabsf(x));
  const float s = e * __builtin_amdgcn_rcpf(2.0f + e), q = s * s;
  float p = 0.28174657f;
  p = fmaf(p, q, 0.27961419f);
  p = fmaf(p, q, 0.40024854f);
  p = fmaf(p, q, 0.66666316f);
  p = fmaf(p, q, 2.0f);
  return fmaf(s, p, fmaxf(x, 0.0f));
}

// Values as they are in memory, and how a float becomes one.
template <typename T>
struct Raw;
template <>
struct Raw<bf16_t> {
  typedef uint16_t type;
  __device__ static __forceinline__ float value(uint16_t x) { return bf16_to_f32(x); }
  __device__ static __forceinline__ uint16_t load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
  }
  __device__ static __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off, float x) {
    __builtin_amdgcn_raw_buffer_store_b16(to_bf16(x), r, off, 0, 0);
  }
};
template <>
struct Raw<float> {
  typedef uint32_t type;
  __device__ static __forceinline__ float value(uint32_t x) { return __uint_as_float(x); }
  __device__ static __forceinline__ uint32_t load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
  }
  __device__ static __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off, float x) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), r, off, 0, 0);
  }
};

// Four rows of a tensor from row t on: a lane's offset in row j is fixed, the
// base moves with t.  Rows from `end` on are outside of the resource: they read
// as zero and are not written.
constexpr uint32_t kNowhere = 0xFFFFFFF0u;  // outside of every resource
template <typename T, int ROWS>
struct RowWindow {
  const T* base;
  uint32_t stride;  // bytes; below 2^27
  uint32_t off[ROWS];
  __device__ __forceinline__ void init(const void* p, int64_t batch, int64_t token, uint32_t column, bool in) {
    base = static_cast<const T*>(p) + batch;
    stride = (uint32_t)token * sizeof(T);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) off[j] = in ? column * (uint32_t)sizeof(T) + j * stride : kNowhere;
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t at(int t, int end) const {
    // (uniform; the clamp alone would be taken for a lane's value)
    const int n = __builtin_amdgcn_readfirstlane(min(max(end - t, 0), ROWS));
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(reinterpret_cast<const char*>(base)) + (int64_t)t * stride, 0, (int)(n * stride), 0x00020000);
  }
};

}  // namespace mlstm
