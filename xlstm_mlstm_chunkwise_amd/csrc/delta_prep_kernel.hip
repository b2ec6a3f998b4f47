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
// all chunks at once.  T and P leave it cut into bf16 parts and in operand
// order (delta_common.h), so that the walks, which read them once per slice of
// the value columns, move them to LDS as they are; for the backward walk the
// same of T^T and P^T.
//
// B is summed in double: a gate that closes the state for good (f = -inf, a
// document's end) enters as log a = -200, whose e^ is zero in float32, and
// the differences B_t - B_j of the tokens behind it keep their digits.
//
// T is the inverse by blocks of sixteen rows.  Diagonal blocks come by forward
// substitution, a column a lane; a block d rows of blocks below the diagonal is
// T_ij = -T_ii sum_{j <= m < i} A_im T_mj, on the float32 matrix cores.  It is
// the recurrence itself in another order, without the powers of A that would
// grow for keys that repeat.
//
// 64 heads of 128 x 128 at 2048 tokens (2048 chunks): 40 us, 43 us with T^T;
// 64 heads of 256 x 512 at 8192 tokens: 170 and 197 us, 0.82 and 0.97 GB moved.
// It is bound by its chain of dependent steps (the waves wait 59 % of their
// time, the vector units are busy half of it): a row of scans, the inverse's four
// diagonal blocks and three rounds of products below them.  Four workgroups a
// CU hide part of that; whole rows of K and Q in LDS leave room for two (250
// against 181 us at 256 columns), and forward substitution over all 64 rows
// instead of sixteen took 268 us.
#include "delta_common.h"
#include "kernels.h"

namespace mlstm {
namespace {

template <typename TIn, int DK, bool BACK>
__global__ __launch_bounds__(4 * DeltaIn<TIn>::kChunk) void delta_prep_kernel(const DeltaParams p) {
  constexpr int L = DeltaIn<TIn>::kChunk, NP = DeltaIn<TIn>::kParts, RT = L / 16, THREADS = 4 * L;
  constexpr int LDA = L + 4;
  constexpr int W = DK < 128 ? DK : 128;  // columns of K and Q at a time: four workgroups fit a CU
  constexpr int kTiles = 2 * NP * L * W * 2, kSquares = 2 * L * LDA * 4;
  __shared__ double s_b[L];
  __shared__ __align__(16) float s_beta[L];
  __shared__ uint4 smem[(kTiles > kSquares ? kTiles : kSquares) / 16];
  uint16_t* s_K = reinterpret_cast<uint16_t*>(smem);  // first K and Q,
  uint16_t* s_Q = s_K + NP * L * W;
  float* s_A = reinterpret_cast<float*>(smem);        // then the squares
  float* s_T = s_A + L * LDA;

  const int bh = blockIdx.x / p.Nc, c = blockIdx.x % p.Nc;
  const int t0 = c * L;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const size_t at = (size_t)bh * p.Nc + c;

  PartStage<TIn, DK, W, THREADS> gk, gq;
  const int rows = p.S - t0 < L ? p.S - t0 : L;
  const TIn* K = static_cast<const TIn*>(p.K) + ((size_t)bh * p.S + t0) * DK;
  const TIn* Q = static_cast<const TIn*>(p.Q) + ((size_t)bh * p.S + t0) * DK;
  gk.load(K, 0, rows, tid);
  gq.load(Q, 0, rows, tid);
  if (wave == 0) {
    const int t = t0 + lane;
    const bool in = lane < L && t < p.S;
    const float lf = in ? log_sigmoid(p.f_pre[(size_t)bh * p.S + t]) : 0.0f;
    double b = (double)(lf < kMinLogDecay ? kMinLogDecay : lf);  // a NaN stays one; fmaxf would close the gate
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

  // K K^T and Q K^T: this wave's 16 rows against the column tiles up to its own
  float4_t kk[RT], qk[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) kk[j] = qk[j] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  const int seed = tile_row_seed<W>(row, grp);
#pragma unroll
  for (int c0 = 0; c0 < DK; c0 += W) {
    if (c0) __syncthreads();
    gk.store(s_K, L * W, tid);
    gq.store(s_Q, L * W, tid);
    __syncthreads();
    if (c0 + W < DK) {
      gk.load(K + c0 + W, c0 + W, rows, tid);
      gq.load(Q + c0 + W, c0 + W, rows, tid);
    }
#pragma unroll
    for (int ks = 0; ks < W / 32; ++ks) {
      const Parts<NP> ka = tile_row<NP, W>(s_K, L * W, seed, wave, ks);
      const Parts<NP> qa = tile_row<NP, W>(s_Q, L * W, seed, wave, ks);
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        if (j > wave) continue;
        const Parts<NP> kb = tile_row<NP, W>(s_K, L * W, seed, j, ks);
        kk[j] = mma_parts<NP, NP>(ka, kb, kk[j]);
        qk[j] = mma_parts<NP, NP>(qa, kb, qk[j]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    if (j > wave) continue;
    const int cc = 16 * j + row;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * wave + 4 * grp + r;
      const float D = cc <= t ? expf((float)(s_b[t] - s_b[cc])) : 0.0f;
      s_A[t * LDA + cc] = cc < t ? s_beta[t] * D * kk[j][r] : 0.0f;
      qk[j][r] = cc <= t ? D * qk[j][r] : 0.0f;
    }
  }
  __syncthreads();
  // diagonal blocks: column `lane` of (I + A_ii)^-1
  if (lane < 16) {
    float x[16];
    const float* A = &s_A[16 * wave * LDA + 16 * wave];
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      float a = t == lane ? 1.0f : 0.0f;
#pragma unroll
      for (int m = 0; m < t; ++m) a -= A[t * LDA + m] * x[m];
      x[t] = a;
      s_T[(16 * wave + t) * LDA + 16 * wave + lane] = a;
    }
  }
#pragma unroll
  for (int d = 1; d < RT; ++d) {
    __syncthreads();
    if (wave >= d) {
      const int j = wave - d;
      float4_t g = {0.0f, 0.0f, 0.0f, 0.0f}, x = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int m = j; m < wave; ++m)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          g = __builtin_amdgcn_mfma_f32_16x16x4f32(s_A[(16 * wave + row) * LDA + 16 * m + 4 * s + grp],
                                                   s_T[(16 * m + 4 * s + grp) * LDA + 16 * j + row], g, 0, 0, 0);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        x = __builtin_amdgcn_mfma_f32_16x16x4f32(s_T[(16 * wave + row) * LDA + 16 * wave + 4 * grp + s], g[s], x, 0, 0,
                                                 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) s_T[(16 * wave + 4 * grp + r) * LDA + 16 * j + row] = -x[r];
    }
  }
  __syncthreads();
  // P takes A's place
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    if (j > wave) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) s_A[(16 * wave + 4 * grp + r) * LDA + 16 * j + row] = qk[j][r];
  }
  __syncthreads();

  constexpr int NF = square_frags<L>();
  const size_t frag_at = at * NF * 3 * kFragElems;
  auto put = [&](const float* M, bool up, bool beta, int planes, uint16_t* dst) {
    for (int i = tid; i < NF * 64; i += THREADS) {
      const int f = i >> 6, l = i & 63, o = 4 * (l >> 4);
      int rt = f, ts = 0;
      if (L == 64) {
        rt = up ? (f < 4 ? f >> 1 : f - 2) : (f < 2 ? f : 2 + ((f - 2) >> 1));
        ts = up ? (f < 4 ? f & 1 : 1) : (f < 2 ? 0 : (f - 2) & 1);
      }
      const int a = 16 * rt + (l & 15);
      // read whole, then cut at the diagonal: what is above it is in range, but
      // nobody has written it
      float x[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int b = 32 * ts + o + 16 * half;
        float4_t m, scale = {1.0f, 1.0f, 1.0f, 1.0f};
        if (up) {
#pragma unroll
          for (int e = 0; e < 4; ++e) m[e] = M[(b + e) * LDA + a];
        } else {
          m = *reinterpret_cast<const float4_t*>(M + a * LDA + b);
          if (beta) scale = *reinterpret_cast<const float4_t*>(s_beta + b);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool low = up ? a <= b + e : b + e <= a;
          x[4 * half + e] = low ? m[e] * (beta ? up ? s_beta[a] : scale[e] : 1.0f) : 0.0f;
        }
      }
      const Parts<3> y = planes == 3 ? split_parts<3>(x) : widen_parts(split_parts<2>(x));
      for (int n = 0; n < planes; ++n)
        *reinterpret_cast<uint4*>(dst + frag_at + (size_t)(f * planes + n) * kFragElems + 8 * l) =
            __builtin_bit_cast(uint4, n == 0 ? y.p[0] : n == 1 ? y.p[1] : y.p[2]);
    }
  };
  put(s_T, false, true, 3, p.T);
  put(s_A, BACK, false, !BACK && p.h_bf16 ? 2 : 3, p.P);
  if constexpr (BACK) put(s_T, true, true, 3, p.Tt);
}

template <typename TIn, int DK>
hipError_t launch_dk(const DeltaParams& p, bool back, hipStream_t stream) {
  const dim3 grid((unsigned)((long long)p.BH * p.Nc)), block(4 * DeltaIn<TIn>::kChunk);
  if (back) hipLaunchKernelGGL((delta_prep_kernel<TIn, DK, true>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((delta_prep_kernel<TIn, DK, false>), grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_prep(const DeltaParams& p, bool back, hipStream_t stream) {
  switch (p.DK) {
    case 64: return p.qkv_bf16 ? launch_dk<bf16_t, 64>(p, back, stream) : launch_dk<float, 64>(p, back, stream);
    case 128: return p.qkv_bf16 ? launch_dk<bf16_t, 128>(p, back, stream) : launch_dk<float, 128>(p, back, stream);
    case 256: return p.qkv_bf16 ? launch_dk<bf16_t, 256>(p, back, stream) : launch_dk<float, 256>(p, back, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mlstm
