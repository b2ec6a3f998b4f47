// Gated delta rule: one token for every head (decode), gfx950.
//
// With a = sigmoid(f), b = sigmoid(i) and the state C entering the step:
//   u = b (v - a C^T k),   C' = a C + k u^T,   h = s C'^T q.
// h = s (a C^T q + u (k . q)), so one pass over C gives both C^T k and
// C^T q, and C' is written from the registers that hold C: the state is read
// once and written once, which bounds the step.  One workgroup per (head, 64
// columns): thread (row group, column quad) holds 16-byte pieces of
// every 16th row, all loads issued before anything waits on them, with
// non-temporal accesses as in the step of the plain cell (a model's other
// layers pass through the caches between two steps of one layer).  64 heads
// of 256 x 512, 67.5 MB: 13.5 us with states that no cache holds (twelve sets in
// turn, 5.0 TB/s), 11.2 us on the same set again and again; on that, 128 columns
// a workgroup took 12.1 us against 11.6.
#include "device_common.h"
#include "kernels.h"

namespace mlstm {
namespace {

typedef float nt_f4_t __attribute__((ext_vector_type(4)));

constexpr int kRowGroups = 16, kCols = 64, kThreads = kCols / 4 * kRowGroups;

__device__ __forceinline__ float ld(const void* x, size_t i, int bf16) {
  return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(x)[i]) : static_cast<const float*>(x)[i];
}

template <int DK>
__global__ __launch_bounds__(kThreads) void delta_step_kernel(const DeltaStepParams p) {
  constexpr int RPT = DK / kRowGroups, CQ = kCols / 4;
  __shared__ float s_q[DK], s_k[DK], s_kq[kThreads / 64];
  __shared__ float4 s_ck[kRowGroups][CQ], s_cq[kRowGroups][CQ];
  __shared__ float4 s_u[CQ];

  const int NS = p.DV / kCols;
  const int bh = blockIdx.x / NS, slice = blockIdx.x % NS;
  const int tid = threadIdx.x, cq = tid % CQ, rg = tid / CQ;
  const int col = slice * kCols + 4 * cq;
  const size_t base = (size_t)bh * DK * p.DV + col;

  nt_f4_t C[RPT];
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    C[r] = (nt_f4_t){0.0f, 0.0f, 0.0f, 0.0f};
    if (p.C_in)
      C[r] = __builtin_nontemporal_load(
          reinterpret_cast<const nt_f4_t*>(p.C_in + base + (size_t)(rg + kRowGroups * r) * p.DV));
  }
  const float a = expf(log_sigmoid(p.f_pre[bh]));
  const float b = 1.0f / (1.0f + expf(-p.i_pre[bh]));
  float dot = 0.0f;
  for (int i = tid; i < DK; i += kThreads) {
    const float q = ld(p.q, (size_t)bh * DK + i, p.qkv_bf16), k = ld(p.k, (size_t)bh * DK + i, p.qkv_bf16);
    s_q[i] = q;
    s_k[i] = k;
    dot += q * k;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, 64);
  if ((tid & 63) == 0) s_kq[tid >> 6] = dot;
  __syncthreads();

  nt_f4_t ck = {0.0f, 0.0f, 0.0f, 0.0f}, cqv = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const float k = s_k[rg + kRowGroups * r], q = s_q[rg + kRowGroups * r];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ck[e] += k * C[r][e];
      cqv[e] += q * C[r][e];
    }
  }
  s_ck[rg][cq] = __builtin_bit_cast(float4, ck);
  s_cq[rg][cq] = __builtin_bit_cast(float4, cqv);
  __syncthreads();

  if (rg == 0) {
    float kq = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) kq += s_kq[w];
#pragma unroll
    for (int g = 1; g < kRowGroups; ++g) {
      const nt_f4_t x = __builtin_bit_cast(nt_f4_t, s_ck[g][cq]), y = __builtin_bit_cast(nt_f4_t, s_cq[g][cq]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ck[e] += x[e];
        cqv[e] += y[e];
      }
    }
    nt_f4_t u;
    float h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[e] = b * (ld(p.v, (size_t)bh * p.DV + col + e, p.qkv_bf16) - a * ck[e]);
      h[e] = p.scale * (a * cqv[e] + u[e] * kq);
    }
    s_u[cq] = __builtin_bit_cast(float4, u);
    const size_t o = (size_t)bh * p.DV + col;
    if (p.h_bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.h) + o) =
          make_uint2(round_bf16x2(h[0], h[1]), round_bf16x2(h[2], h[3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p.h) + o) = make_float4(h[0], h[1], h[2], h[3]);
  }
  __syncthreads();

  const nt_f4_t u = __builtin_bit_cast(nt_f4_t, s_u[cq]);
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const float k = s_k[rg + kRowGroups * r];
#pragma unroll
    for (int e = 0; e < 4; ++e) C[r][e] = a * C[r][e] + k * u[e];
    __builtin_nontemporal_store(C[r],
                                reinterpret_cast<nt_f4_t*>(p.C_out + base + (size_t)(rg + kRowGroups * r) * p.DV));
  }
}

template <int DK>
hipError_t launch_dk(const DeltaStepParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)((long long)p.BH * (p.DV / kCols))), block(kThreads);
  hipLaunchKernelGGL((delta_step_kernel<DK>), grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_step(const DeltaStepParams& p, hipStream_t stream) {
  if (p.DV <= 0 || p.DV % 64 != 0) return hipErrorInvalidValue;
  switch (p.DK) {
    case 64: return launch_dk<64>(p, stream);
    case 128: return launch_dk<128>(p, stream);
    case 256: return launch_dk<256>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mlstm
