// Dropout with the residual sum, gfx950: the mask comes from a counter-based
// generator and is never stored, so the gradient forms it again.
//   word j of Philox 4x32-10(key = seed, counter = (block, offset)) decides
//   value 4 block + j: dropped below `limit`, else times `scale`.
// A round takes two 32 x 32 -> 64 bit products and four exclusive ors for four
// values.  Bound by memory: 2^28 values in bf16 with the residual 270 us for 1.6
// GB (6 TB/s, vector issue 57 % of the cycles), without 205 us for 1.07 GB (5.2).
#include "device_common.h"
#include "delta_common.h"
#include "kernels.h"

namespace mlstm {
namespace {

constexpr int kThreads = 256;

struct Words {
  uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t m0 = (uint64_t)0xD2511F53u * c0, m1 = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(m1 >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(m0 >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)m1;
    c3 = (uint32_t)m0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

__device__ __forceinline__ float ld(const bf16_t* p) { return bf16_to_f32(p->bits); }
__device__ __forceinline__ float ld(const float* p) { return *p; }
__device__ __forceinline__ void st(bf16_t* p, float x) { p->bits = f32_to_bf16(x); }
__device__ __forceinline__ void st(float* p, float x) { *p = x; }

// VEC values a thread: 16 bytes of an aligned tensor, or one block of four by
// single values.
template <typename T, int VEC, bool WIDE, bool RES>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const DropoutParams p) {
  const uint64_t seed = p.seed_dev ? (uint64_t)p.seed_dev[0] : p.seed;
  const uint64_t offset = p.seed_dev ? (uint64_t)p.seed_dev[1] : p.offset;
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.residual);
  T* y = static_cast<T*>(p.y);
  const int64_t step = (int64_t)gridDim.x * kThreads * VEC;
  for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * VEC; i < p.n; i += step) {
    float v[VEC], r[VEC];
    const bool whole = WIDE && i + VEC <= p.n;
    if (whole) {
      if constexpr (WIDE) {
        if constexpr (sizeof(T) == 2) {
          Ops<bf16_t>::load8(x + i, v);
          if (RES) Ops<bf16_t>::load8(res + i, r);
        } else {
          const float4 a = *reinterpret_cast<const float4*>(x + i);
          v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
          if (RES) {
            const float4 b = *reinterpret_cast<const float4*>(res + i);
            r[0] = b.x; r[1] = b.y; r[2] = b.z; r[3] = b.w;
          }
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[e] = i + e < p.n ? ld(x + i + e) : 0.0f;
        if (RES) r[e] = i + e < p.n ? ld(res + i + e) : 0.0f;
      }
    }
#pragma unroll
    for (int b = 0; b < VEC / 4; ++b) {
      const Words w = philox((uint64_t)i / 4 + b, offset, seed);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 4 * b + j;
        const float kept = w.w[j] >= p.limit ? v[e] * p.scale : 0.0f;
        v[e] = RES ? kept + r[e] : kept;
      }
    }
    if (whole) {
      if constexpr (WIDE) {
        if constexpr (sizeof(T) == 2)
          *reinterpret_cast<uint4*>(y + i) = make_uint4(round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3]),
                                                        round_bf16x2(v[4], v[5]), round_bf16x2(v[6], v[7]));
        else
          *reinterpret_cast<float4*>(y + i) = make_float4(v[0], v[1], v[2], v[3]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (i + e < p.n) st(y + i + e, v[e]);
    }
  }
}

template <typename T, int VEC, bool WIDE>
hipError_t launch(const DropoutParams& p, hipStream_t stream) {
  const int64_t per = (int64_t)kThreads * VEC;
  int64_t groups = (p.n + per - 1) / per;
  if (groups > (1 << 20)) groups = 1 << 20;
  if (p.residual)
    hipLaunchKernelGGL((dropout_kernel<T, VEC, WIDE, true>), dim3((unsigned)groups), dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((dropout_kernel<T, VEC, WIDE, false>), dim3((unsigned)groups), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutParams& p, hipStream_t stream) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.y) |
                       reinterpret_cast<uintptr_t>(p.residual);
  // (2^28 values, whole calls: bf16 218 us, by single values 419; float32 363 and 556)
  const bool wide = at % 16 == 0;
  if (p.bf16) return wide ? launch<bf16_t, 8, true>(p, stream) : launch<bf16_t, 4, false>(p, stream);
  return wide ? launch<float, 4, true>(p, stream) : launch<float, 4, false>(p, stream);
}

}  // namespace mlstm
