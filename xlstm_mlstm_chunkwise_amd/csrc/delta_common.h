// Device helpers of the gated delta rule's kernels: operands carried in
// several bf16 parts, and the 16 x 16 x 32 products over them.
//
// A float32 value is cut into three bf16 parts of eight significant bits
// each (hi + mid + lo, exact unless a part falls below the smallest normal).
// A product of an n-part and an m-part operand runs the part pairs (i, j)
// with i + j < max(n, m): a bf16 input (one part) times a three-part operand
// takes three matrix instructions and loses nothing but the float32
// accumulation; three parts times three take six and drop terms below 2^-24.
// The state is carried from chunk to chunk in float32 and every chunk
// multiplies it, so two-part operands (2^-17 a rounding) would show in the
// float32 outputs (final state, gate gradients: 4e-6 to 9e-6 of their norm
// instead of below 1e-6); only results that are stored as bf16 use two.
#pragma once

#include "device_common.h"
#include "kernels.h"

namespace mlstm {

template <int N>
struct Parts {
  bf16x8_t p[N];
};

// Eight floats as N parts.  N = 3: each part is the leading sixteen bits of
// what the parts before it left (truncation; the remainders are exact).
// N = 2: nearest-even roundings.
template <int N>
__device__ __forceinline__ Parts<N> split_parts(const float (&x)[8]) {
  Parts<N> f;
  if constexpr (N == 1) {
    f.p[0] = Ops<bf16_t>::round(x);
  } else if constexpr (N == 2) {
    Ops<bf16_t>::split(x, f.p[0], f.p[1]);
  } else {
    uint32_t w[3][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a = x[2 * e], b = x[2 * e + 1];
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
        w[n][e] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
        if (n < 2) {
          a -= __uint_as_float(ua & 0xffff0000u);
          b -= __uint_as_float(ub & 0xffff0000u);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < 3; ++n) f.p[n] = as_bf16x8(make_uint4(w[n][0], w[n][1], w[n][2], w[n][3]));
  }
  return f;
}

// Two accumulator tiles (rows 0..15 and 16..31 of a 32-row block, one
// column per lane) as the eight values of one operand.
__device__ __forceinline__ void tiles8(const float4_t& a, const float4_t& b, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = a[e];
    x[e + 4] = b[e];
  }
}

template <int NA, int NB>
__device__ __forceinline__ float4_t mma_parts(const Parts<NA>& a, const Parts<NB>& b, float4_t c) {
  constexpr int M = NA > NB ? NA : NB;
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < M) c = mma16b(a.p[i], b.p[j], c);
  return c;
}

// Operand parts out of LDS planes (plane stride in elements).
// Row operand whose slots are 8 * (l / 16) + e: one 16-byte read a plane.
template <int N>
__device__ __forceinline__ Parts<N> lds_row8(const uint16_t* p, int plane) {
  Parts<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) f.p[n] = as_bf16x8(*reinterpret_cast<const uint4*>(p + n * plane));
  return f;
}
// Row operand in the slot order of two accumulator tiles: slots e < 4 at
// p[0..3], the others sixteen elements on.
template <int N>
__device__ __forceinline__ Parts<N> lds_row44(const uint16_t* p, int plane) {
  Parts<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint2 a = *reinterpret_cast<const uint2*>(p + n * plane);
    const uint2 b = *reinterpret_cast<const uint2*>(p + n * plane + 16);
    f.p[n] = as_bf16x8(make_uint4(a.x, a.y, b.x, b.y));
  }
  return f;
}
__device__ __forceinline__ uint2 lds_tr4(const uint16_t* p) {
  return __builtin_bit_cast(
      uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4_t*)(p)));
}
// Column operand: lane l gets column c0 + l % 16 of a row-major tile X, rows
// r0 + {0..3} (slots 0..3) and r0 + d + {0..3} (slots 4..7), r0 counted from
// the lane group's own base: 4 * (l / 16) with d = 16 for the slot order of
// two accumulator tiles, 8 * (l / 16) with d = 4 for the plain order.
template <int N>
__device__ __forceinline__ Parts<N> lds_col(const uint16_t* X, int ld, int plane, int r0, int d, int c0, int lane) {
  const int j = lane & 15;
  const uint16_t* p = X + (r0 + (j >> 2)) * ld + c0 + 4 * (j & 3);
  Parts<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint2 a = lds_tr4(p + n * plane), b = lds_tr4(p + n * plane + d * ld);
    f.p[n] = as_bf16x8(make_uint4(a.x, a.y, b.x, b.y));
  }
  return f;
}

// Storage of Q, K, V by input type: parts and tokens per chunk.  A float32
// input is itself carried in three parts, so its chunk has half the rows for
// the same LDS.
template <typename TIn>
struct DeltaIn;
template <>
struct DeltaIn<bf16_t> {
  static constexpr int kParts = 1, kChunk = kDeltaChunkBf16;
};
template <>
struct DeltaIn<float> {
  static constexpr int kParts = 3, kChunk = kDeltaChunkF32;
};

__device__ __forceinline__ float load1(const bf16_t* p) { return bf16_to_f32(p->bits); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(bf16_t* p, float x) { p->bits = f32_to_bf16(x); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store4(bf16_t* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = make_uint2(round_bf16x2(a, b), round_bf16x2(c, d));
}
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}

// Eight consecutive inputs as operand parts (global memory, 16-byte aligned).
__device__ __forceinline__ Parts<1> load_parts(const bf16_t* p) {
  Parts<1> f;
  f.p[0] = as_bf16x8(*reinterpret_cast<const uint4*>(p));
  return f;
}
__device__ __forceinline__ Parts<3> load_parts(const float* p) {
  float x[8];
  Ops<float>::load8(p, x);
  return split_parts<3>(x);
}
template <int N>
__device__ __forceinline__ Parts<N> zero_parts() {
  Parts<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) f.p[n] = as_bf16x8(make_uint4(0u, 0u, 0u, 0u));
  return f;
}
template <int N>
__device__ __forceinline__ void store_parts(uint16_t* p, int plane, const Parts<N>& f) {
#pragma unroll
  for (int n = 0; n < N; ++n) *reinterpret_cast<uint4*>(p + n * plane) = __builtin_bit_cast(uint4, f.p[n]);
}

// Rows [t0, t0 + ROWS) of a row-major input of S rows and W columns into LDS
// planes, zeros behind the last row.
template <typename TIn, int ROWS, int W>
__device__ __forceinline__ void stage_rows(uint16_t* dst, int ld, int plane, const TIn* src, int t0, int S, int tid,
                                           int threads) {
  constexpr int NP = DeltaIn<TIn>::kParts;
  for (int i = tid; i < ROWS * (W / 8); i += threads) {
    const int r = i / (W / 8), c = 8 * (i % (W / 8));
    const Parts<NP> f = t0 + r < S ? load_parts(src + (size_t)(t0 + r) * W + c) : zero_parts<NP>();
    store_parts<NP>(dst + r * ld + c, plane, f);
  }
}

// A float32 L x L matrix into three LDS planes.
template <int L>
__device__ __forceinline__ void stage_square(uint16_t* dst, int ld, int plane, const float* src, int tid, int threads) {
  for (int i = tid; i < L * (L / 8); i += threads) {
    const int r = i / (L / 8), c = 8 * (i % (L / 8));
    float x[8];
    Ops<float>::load8(src + r * L + c, x);
    store_parts<3>(dst + r * ld + c, plane, split_parts<3>(x));
  }
}

}  // namespace mlstm
