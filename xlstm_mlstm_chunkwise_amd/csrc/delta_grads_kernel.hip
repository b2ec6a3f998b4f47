// Gated delta rule: dQ, dK and the gate gradients of every chunk, gfx950.
//
// With C the state entering the chunk, G the gradient of the state behind
// it, U and dV as the two walks left them and e, w, D as in
// delta_prep_kernel.hip:
//   dP = s D o (dH U^T),   dA = -(D o (dV U^T))_strict,
//   dQ = s e dH C^T + dP K,
//   dK = dP^T Q + (dA + dA^T) K - e dV C^T + w U G^T,
//   d log a_t = sum_{r >= t} (q_r . dq_r - v_r . dv_r) + <C behind, G>,
//   d b_t = dV_t . U_t / b_t^2,
// with the sum over the chunk's own rows only and <C behind, G> = g <C, G> +
// sum_t w_t u_t . (K G)_t formed afresh for every chunk: one running sum over
// the whole sequence would add up the roundings of all tokens behind t.
//
// One workgroup per chunk, DHQK / 32 waves: wave i owns rows 32 i .. 32 i + 31
// of C and G, which it reads from memory straight into its operands, and
// forms dQ^T and dK^T for them; the 64 x 64 products are spread over the
// waves.  dH, U and dV go through LDS in steps of 32 value columns.
#include "delta_common.h"
#include "kernels.h"

namespace mlstm {
namespace {

// The i-th tile (row tile, column tile) on or below the diagonal.
__device__ __forceinline__ void lower_tile(int i, int& rt, int& ct) {
  rt = 0;
  while (i > rt) i -= ++rt;
  ct = i;
}

template <typename TIn, typename TH, int DK>
struct GradLds {
  static constexpr int L = DeltaIn<TIn>::kChunk, NP = DeltaIn<TIn>::kParts, NH = DeltaIn<TH>::kParts;
  static constexpr int kLdT = 40, kPlaneT = L * kLdT;   // 32 value columns of dH, U, dV
  static constexpr int kLd = DK + 8, kPlane = L * kLd;  // K, Q (in the same space afterwards)
  static constexpr int kLdS = L + 8, kPlaneS = L * kLdS;  // dP and dA + dA^T
  static constexpr int kStage = (NH + 6) * kPlaneT > 2 * NP * kPlane ? (NH + 6) * kPlaneT : 2 * NP * kPlane;
  static constexpr int kBytes = 2 * (kStage + 2 * 3 * kPlaneS);
};

template <typename TIn, typename TH, int DK>
__global__ __launch_bounds__(2 * DK) void delta_grads_kernel(const DeltaParams p) {
  typedef GradLds<TIn, TH, DK> W;
  constexpr int L = W::L, NP = W::NP, NH = W::NH, NW = DK / 32, THREADS = 64 * NW;
  constexpr int RT = L / 16, NT = RT * (RT + 1) / 2, TPW = (NT + NW - 1) / NW;
  constexpr int NB = NP == 1 ? 2 : 3;  // parts of the terms of dK alone, which is stored as TIn
  constexpr int ROWS = (4 * L + THREADS - 1) / THREADS;
  __shared__ uint4 smem[W::kBytes / 16];
  __shared__ float s_red[NW][L];
  __shared__ float s_dvu[L], s_vdv[L], s_cg[NW];
  __shared__ double s_b[L];
  uint16_t* s_H = reinterpret_cast<uint16_t*>(smem);
  uint16_t* s_U = s_H + NH * W::kPlaneT;
  uint16_t* s_R = s_U + 3 * W::kPlaneT;
  uint16_t* s_K = reinterpret_cast<uint16_t*>(smem);
  uint16_t* s_Q = s_K + NP * W::kPlane;
  uint16_t* s_dP = reinterpret_cast<uint16_t*>(smem) + W::kStage;
  uint16_t* s_dA = s_dP + 3 * W::kPlaneS;

  const int bh = blockIdx.x / p.Nc, c = blockIdx.x % p.Nc, t0 = c * L;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const size_t at = (size_t)bh * p.Nc + c;
  const int DV = p.DV;
  if (tid < L) s_b[tid] = p.bsum[at * L + tid];

  float4_t dq[2][RT], dkc[2][RT], dkg[2][RT], hu[TPW], ru[TPW];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) dq[i][j] = dkc[i][j] = dkg[i][j] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < TPW; ++i) hu[i] = ru[i] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  float cg = 0.0f, dvu[ROWS], vdv[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) dvu[i] = vdv[i] = 0.0f;

  const float* Cs = p.C_states + (at * DK + 32 * wave + row) * DV + 8 * grp;
  const float* Gs = p.G_states + (at * DK + 32 * wave + row) * DV + 8 * grp;
  for (int v0 = 0; v0 < DV; v0 += 32) {
    float xc[2][8], xg[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      Ops<float>::load8(Cs + (size_t)16 * i * DV + v0, xc[i]);
      Ops<float>::load8(Gs + (size_t)16 * i * DV + v0, xg[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int piece = tid + i * THREADS;
      if (piece >= 4 * L) break;
      const int t = piece >> 2, cc = v0 + 8 * (piece & 3), o = t * W::kLdT + 8 * (piece & 3);
      float xu[8], xr[8];
      Ops<float>::load8(p.U + (at * L + t) * DV + cc, xu);
      Ops<float>::load8(p.R + (at * L + t) * DV + cc, xr);
      store_parts<3>(s_U + o, W::kPlaneT, split_parts<3>(xu));
      store_parts<3>(s_R + o, W::kPlaneT, split_parts<3>(xr));
      const size_t g = ((size_t)bh * p.S + t0 + t) * DV + cc;
      const bool in = t0 + t < p.S;
      store_parts<NH>(s_H + o, W::kPlaneT, in ? load_parts(static_cast<const TH*>(p.dH) + g) : zero_parts<NH>());
      float xv[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (in) Ops<TIn>::load8(static_cast<const TIn*>(p.V) + g, xv);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dvu[i] += xr[e] * xu[e];
        vdv[i] += xv[e] * xr[e];
      }
    }
    __syncthreads();

    // the products with the states: rows of C and G, columns t
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) cg += xc[i][e] * xg[i][e];
      const Parts<3> cp = split_parts<3>(xc[i]);
      Parts<NB> cb;
#pragma unroll
      for (int n = 0; n < NB; ++n) cb.p[n] = cp.p[n];
      const Parts<NB> gp = split_parts<NB>(xg[i]);
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int o = (16 * j + row) * W::kLdT + 8 * grp;
        dq[i][j] = mma_parts<3, NH>(cp, lds_row8<NH>(s_H + o, W::kPlaneT), dq[i][j]);
        dkc[i][j] = mma_parts<NB, NB>(cb, lds_row8<NB>(s_R + o, W::kPlaneT), dkc[i][j]);
        dkg[i][j] = mma_parts<NB, NB>(gp, lds_row8<NB>(s_U + o, W::kPlaneT), dkg[i][j]);
      }
    }
    // dH U^T and dV U^T
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int tile = wave + i * NW;
      if (tile >= NT) break;
      int rt, ct;
      lower_tile(tile, rt, ct);
      const int oa = (16 * rt + row) * W::kLdT + 8 * grp, ob = (16 * ct + row) * W::kLdT + 8 * grp;
      const Parts<3> up = lds_row8<3>(s_U + ob, W::kPlaneT);
      hu[i] = mma_parts<NH, 3>(lds_row8<NH>(s_H + oa, W::kPlaneT), up, hu[i]);
      Parts<NB> ub;
#pragma unroll
      for (int n = 0; n < NB; ++n) ub.p[n] = up.p[n];
      ru[i] = mma_parts<NB, NB>(lds_row8<NB>(s_R + oa, W::kPlaneT), ub, ru[i]);
    }
  }
  __syncthreads();  // the staged columns are read out: K and Q take their place

  // row sums of the staged pieces, four lanes a row
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int piece = tid + i * THREADS;
    float a = dvu[i], b = vdv[i];
    a += __shfl_xor(a, 1, 64);
    b += __shfl_xor(b, 1, 64);
    a += __shfl_xor(a, 2, 64);
    b += __shfl_xor(b, 2, 64);
    if (piece < 4 * L && (piece & 3) == 0) {
      s_dvu[piece >> 2] = a;
      s_vdv[piece >> 2] = b;
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) cg += __shfl_xor(cg, o, 64);
  if (lane == 0) s_cg[wave] = cg;

  // dP and dA + dA^T as parts (zero above dP's diagonal)
  for (int i = tid; i < 3 * W::kPlaneS / 8; i += THREADS) reinterpret_cast<uint4*>(s_dP)[i] = make_uint4(0u, 0u, 0u, 0u);
  const TIn* K = static_cast<const TIn*>(p.K) + (size_t)bh * p.S * DK;
  const TIn* Q = static_cast<const TIn*>(p.Q) + (size_t)bh * p.S * DK;
  stage_rows<TIn, L, DK>(s_K, W::kLd, W::kPlane, K, t0, p.S, tid, THREADS);
  stage_rows<TIn, L, DK>(s_Q, W::kLd, W::kPlane, Q, t0, p.S, tid, THREADS);
  __syncthreads();
  auto put = [&](uint16_t* dst, float x) {
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      const uint32_t u = __float_as_uint(x);
      dst[n * W::kPlaneS] = (uint16_t)(u >> 16);
      x -= __uint_as_float(u & 0xffff0000u);
    }
  };
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    const int tile = wave + i * NW;
    if (tile >= NT) break;
    int rt, ct;
    lower_tile(tile, rt, ct);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * rt + 4 * grp + r, j = 16 * ct + row;
      if (j <= t) {
        const float D = expf((float)(s_b[t] - s_b[j]));
        put(s_dP + t * W::kLdS + j, p.scale * D * hu[i][r]);
        const float a = j < t ? -D * ru[i][r] : 0.0f;
        put(s_dA + t * W::kLdS + j, a);
        if (j < t) put(s_dA + j * W::kLdS + t, a);
      }
    }
  }
  __syncthreads();

  // scale by rows, then the products within the chunk
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int t = 16 * j + row;
    const float e = p.e[at * L + t], w = p.w[at * L + t], se = p.scale * e;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        dq[i][j][r] *= se;
        dkc[i][j][r] = w * dkg[i][j][r] - e * dkc[i][j][r];
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k0 = 32 * wave + 16 * i;
#pragma unroll
    for (int s = 0; s < L / 32; ++s) {
      const Parts<NP> kt = lds_col<NP>(s_K, W::kLd, W::kPlane, 32 * s + 8 * grp, 4, k0, lane);
      const Parts<NP> qt = lds_col<NP>(s_Q, W::kLd, W::kPlane, 32 * s + 8 * grp, 4, k0, lane);
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int o = (16 * j + row) * W::kLdS + 32 * s + 8 * grp;
        if (s <= j / 2) dq[i][j] = mma_parts<NP, 3>(kt, lds_row8<3>(s_dP + o, W::kPlaneS), dq[i][j]);
        if (s >= j / 2)
          dkc[i][j] = mma_parts<NP, NB>(qt, lds_col<NB>(s_dP, W::kLdS, W::kPlaneS, 32 * s + 8 * grp, 4, 16 * j, lane),
                                        dkc[i][j]);
        dkc[i][j] = mma_parts<NP, NB>(kt, lds_row8<NB>(s_dA + o, W::kPlaneS), dkc[i][j]);
      }
    }
  }

  // store, and q . dq by rows
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int t = 16 * j + row;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k0 = 32 * wave + 16 * i + 4 * grp;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float q = 0.0f;
#pragma unroll
        for (int n = NP - 1; n >= 0; --n) q += bf16_to_f32(s_Q[n * W::kPlane + t * W::kLd + k0 + r]);
        dot += q * dq[i][j][r];
      }
      if (t0 + t < p.S) {
        const size_t o = ((size_t)bh * p.S + t0 + t) * DK + k0;
        store4(static_cast<TIn*>(p.dQ) + o, dq[i][j][0], dq[i][j][1], dq[i][j][2], dq[i][j][3]);
        store4(static_cast<TIn*>(p.dK) + o, dkc[i][j][0], dkc[i][j][1], dkc[i][j][2], dkc[i][j][3]);
      }
    }
    dot += __shfl_xor(dot, 16, 64);
    dot += __shfl_xor(dot, 32, 64);
    if (grp == 0) s_red[wave][t] = dot;
  }
  __syncthreads();

  // gate gradients: one lane a row
  if (wave == 0) {
    const int t = lane < L ? lane : L - 1;
    float d = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) d += s_red[w][t];
    d -= s_vdv[t];
    if (lane >= L) d = 0.0f;
    if (lane == L - 1) {
      float a = 0.0f, x = 0.0f;
      for (int i = 0; i < DV / 16; ++i) a += p.anchor[at * (DV / 16) + i];
#pragma unroll
      for (int w = 0; w < NW; ++w) x += s_cg[w];
      d += a + p.e[at * L + L - 1] * x;
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const float y = __shfl_down(d, off, 64);
      if (lane + off < 64) d += y;
    }
    if (lane < L && t0 + t < p.S) {
      const size_t o = (size_t)bh * p.S + t0 + t;
      const float f = p.f_pre[o], ip = p.i_pre[o];
      // a gate that passes nothing has no gradient: its e^ is zero in float32,
      // or it is the first and there is no state to pass
      const bool closed = expf(log_sigmoid(f)) == 0.0f || (t0 + t == 0 && !p.C0);
      p.d_f[o] = closed ? 0.0f : d / (1.0f + expf(f));
      const float beta = 1.0f / (1.0f + expf(-ip));
      p.d_i[o] = beta > 0.0f ? s_dvu[t] / beta * (1.0f - beta) : 0.0f;
    }
  }
}

template <typename TIn, typename TH>
hipError_t launch_types(const DeltaParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)((long long)p.BH * p.Nc)), block(2 * p.DK);
  switch (p.DK) {
    case 64: hipLaunchKernelGGL((delta_grads_kernel<TIn, TH, 64>), grid, block, 0, stream, p); break;
    case 128: hipLaunchKernelGGL((delta_grads_kernel<TIn, TH, 128>), grid, block, 0, stream, p); break;
    case 256: hipLaunchKernelGGL((delta_grads_kernel<TIn, TH, 256>), grid, block, 0, stream, p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grads(const DeltaParams& p, hipStream_t stream) {
  if (p.qkv_bf16)
    return p.h_bf16 ? launch_types<bf16_t, bf16_t>(p, stream) : launch_types<bf16_t, float>(p, stream);
  return p.h_bf16 ? launch_types<float, bf16_t>(p, stream) : launch_types<float, float>(p, stream);
}

}  // namespace mlstm
