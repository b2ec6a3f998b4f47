// Gated delta rule: what a chunk needs before the states are known, gfx950.
//
// Per head, with a_t = sigmoid(f_t), b_t = sigmoid(i_t) and the state C:
//   u_t = b_t (v_t - a_t C_{t-1}^T k_t),  C_t = a_t C_{t-1} + k_t u_t^T,
//   h_t = s C_t^T q_t.
// Over a chunk of L rows entered with state C0, with B_t = sum_{r <= t} log a_r,
// e_t = e^{B_t} and D_tj = e^{B_t - B_j} for j <= t (0 above the diagonal):
//   U = T (V - diag(e) K C0),  T = (I + diag(b) (K K^T o D)_strict)^-1 diag(b),
//   H = s (diag(e) Q C0 + P U),  P = Q K^T o D.
// This kernel forms T, P and the decays of every chunk, one workgroup each,
// all chunks at once.
//
// B is summed in double: a gate that closes the state for good (f = -inf, a
// document's end) enters as log a = -200, whose e^ is zero in float32, and
// the differences B_t - B_j of the tokens behind it keep their digits.  T
// comes by forward substitution, one column a lane with the column in
// registers: the recurrence itself, so it is as stable as running the tokens
// one by one, also for keys that repeat.
#include "delta_common.h"
#include "kernels.h"

namespace mlstm {
namespace {

template <typename TIn>
__global__ __launch_bounds__(4 * DeltaIn<TIn>::kChunk) void delta_prep_kernel(const DeltaParams p) {
  constexpr int L = DeltaIn<TIn>::kChunk, NP = DeltaIn<TIn>::kParts, RT = L / 16;
  constexpr int LDA = L + 4;
  __shared__ double s_b[L];
  __shared__ float s_beta[L];
  __shared__ float s_A[L * LDA];

  const int bh = blockIdx.x / p.Nc, c = blockIdx.x % p.Nc;
  const int t0 = c * L;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const size_t at = (size_t)bh * p.Nc + c;

  if (wave == 0) {
    const int t = t0 + lane;
    const bool in = lane < L && t < p.S;
    double b = in ? (double)fmaxf(log_sigmoid(p.f_pre[(size_t)bh * p.S + t]), kMinLogDecay) : 0.0;
    const float ip = in ? p.i_pre[(size_t)bh * p.S + t] : -INFINITY;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double y = __shfl_up(b, off, 64);
      if (lane >= off) b += y;
    }
    const double last = __shfl(b, L - 1, 64);
    if (lane < L) {
      s_b[lane] = b;
      s_beta[lane] = 1.0f / (1.0f + expf(-ip));
      p.bsum[at * L + lane] = b;
      p.e[at * L + lane] = expf((float)b);
      p.w[at * L + lane] = expf((float)(last - b));
    }
  }
  __syncthreads();

  // K K^T and Q K^T: this wave's 16 rows against the column tiles up to its own
  const TIn* K = static_cast<const TIn*>(p.K) + (size_t)bh * p.S * p.DK;
  const TIn* Q = static_cast<const TIn*>(p.Q) + (size_t)bh * p.S * p.DK;
  float4_t kk[RT], qk[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) kk[j] = qk[j] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  const int ta = t0 + 16 * wave + row;
  for (int d = 8 * grp; d < p.DK; d += 32) {
    const bool in = ta < p.S;
    const Parts<NP> ka = in ? load_parts(K + (size_t)ta * p.DK + d) : zero_parts<NP>();
    const Parts<NP> qa = in ? load_parts(Q + (size_t)ta * p.DK + d) : zero_parts<NP>();
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      if (j > wave) continue;
      const int tb = t0 + 16 * j + row;
      const Parts<NP> kb = tb < p.S ? load_parts(K + (size_t)tb * p.DK + d) : zero_parts<NP>();
      kk[j] = mma_parts<NP, NP>(ka, kb, kk[j]);
      qk[j] = mma_parts<NP, NP>(qa, kb, qk[j]);
    }
  }
  float* P = p.P + at * L * L;
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int cc = 16 * j + row;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * wave + 4 * grp + r;
      const float D = cc <= t ? expf((float)(s_b[t] - s_b[cc])) : 0.0f;
      s_A[t * LDA + cc] = cc < t ? s_beta[t] * D * kk[j][r] : 0.0f;
      P[t * L + cc] = cc <= t ? D * qk[j][r] : 0.0f;
    }
  }
  __syncthreads();

  // (I + A)^-1, column `lane`: x_t = [t = lane] - sum_{m < t} A_tm x_m
  if (wave == 0 && lane < L) {
    float x[L];
    const float beta = s_beta[lane];
    float* T = p.T + at * L * L + lane;
#pragma unroll
    for (int t = 0; t < L; ++t) {
      float a[4] = {t == lane ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int m = 0; m < t; m += 4) {
        const float4 r = *reinterpret_cast<const float4*>(&s_A[t * LDA + m]);
        a[0] -= r.x * x[m];
        if (m + 1 < t) a[1] -= r.y * x[m + 1];
        if (m + 2 < t) a[2] -= r.z * x[m + 2];
        if (m + 3 < t) a[3] -= r.w * x[m + 3];
      }
      x[t] = (a[0] + a[1]) + (a[2] + a[3]);
      T[t * L] = x[t] * beta;
    }
  }
}

}  // namespace

hipError_t launch_delta_prep(const DeltaParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)((long long)p.BH * p.Nc));
  if (p.qkv_bf16)
    hipLaunchKernelGGL((delta_prep_kernel<bf16_t>), grid, dim3(4 * DeltaIn<bf16_t>::kChunk), 0, stream, p);
  else
    hipLaunchKernelGGL((delta_prep_kernel<float>), grid, dim3(4 * DeltaIn<float>::kChunk), 0, stream, p);
  return hipGetLastError();
}

}  // namespace mlstm
