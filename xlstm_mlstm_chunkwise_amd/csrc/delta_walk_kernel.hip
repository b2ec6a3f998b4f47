// Gated delta rule: the chunks of a head in order, gfx950.
//
// One workgroup walks the chunks of one head for a slice of the value
// columns.  The columns of the state are independent of each other, so each
// wave carries all DHQK rows of sixteen columns in accumulator registers and
// no wave waits for another's result; the waves of a workgroup share the
// chunk's K, Q, T and P in LDS.  Per chunk (delta_prep_kernel.hip has T, P
// and the decays e, w; g = e of the chunk's last row):
//   U = T (V - e K C),   H = s (e Q C + P U),   C <- g C + K^T (w U).
// The accumulator tiles of C, of V - e K C and of U feed straight back as
// the right operand of the next product: the slot order of two accumulator
// tiles is matched by how the left operands are read from LDS.
#include "delta_common.h"
#include "kernels.h"

namespace mlstm {
namespace {

// LDS of a workgroup: two input tiles (K, Q) and two squares (T, P), as parts.
template <typename TIn, int DK>
struct WalkLds {
  static constexpr int L = DeltaIn<TIn>::kChunk, NP = DeltaIn<TIn>::kParts;
  static constexpr int kLd = DK + 8, kPlane = L * kLd;
  static constexpr int kLdS = L + 8, kPlaneS = L * kLdS;
  static constexpr int kBytes = 2 * (2 * NP * kPlane + 2 * 3 * kPlaneS) + 4 * 2 * L;
};

// acc[rt] += M[rows 16 rt ..][all L] . X for a lower triangular L x L matrix
// M (LDS planes) and X in parts of 32 rows.
template <int L, int NX>
__device__ __forceinline__ void lower_times(const uint16_t* M, int ld, int plane, const Parts<NX> (&x)[L / 32],
                                            float4_t (&acc)[L / 16], int row, int grp) {
#pragma unroll
  for (int rt = 0; rt < L / 16; ++rt)
#pragma unroll
    for (int ts = 0; ts <= rt / 2; ++ts)
      acc[rt] = mma_parts<3, NX>(lds_row44<3>(M + (16 * rt + row) * ld + 32 * ts + 4 * grp, plane), x[ts], acc[rt]);
}

// acc[rt] += (M^T)[rows 16 rt ..] . X, M lower triangular.
template <int L, int NX>
__device__ __forceinline__ void upper_times(const uint16_t* M, int ld, int plane, const Parts<NX> (&x)[L / 32],
                                            float4_t (&acc)[L / 16], int lane, int grp) {
#pragma unroll
  for (int rt = 0; rt < L / 16; ++rt)
#pragma unroll
    for (int ts = rt / 2; ts < L / 32; ++ts)
      acc[rt] = mma_parts<3, NX>(lds_col<3>(M, ld, plane, 32 * ts + 4 * grp, 16, 16 * rt, lane), x[ts], acc[rt]);
}

// FWD: H and the final state.  STATES: the state entering every chunk and U,
// for the backward pass.
template <typename TIn, int DK, int NW, bool FWD, bool STATES>
__global__ __launch_bounds__(64 * NW) void delta_walk_kernel(const DeltaParams p) {
  typedef WalkLds<TIn, DK> W;
  constexpr int L = W::L, NP = W::NP, RT = L / 16, TS = L / 32, KT = DK / 16, THREADS = 64 * NW;
  __shared__ uint4 smem[W::kBytes / 16];
  uint16_t* s_K = reinterpret_cast<uint16_t*>(smem);
  uint16_t* s_Q = s_K + NP * W::kPlane;
  uint16_t* s_T = s_Q + NP * W::kPlane;
  uint16_t* s_P = s_T + 3 * W::kPlaneS;
  float* s_e = reinterpret_cast<float*>(s_P + 3 * W::kPlaneS);
  float* s_w = s_e + L;

  // slices of one head share an XCD's L2 where the head count is a multiple of 8
  const int bh = blockIdx.x % p.BH, slice = blockIdx.x / p.BH;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const int col = (slice * NW + wave) * 16 + row;
  const TIn* K = static_cast<const TIn*>(p.K) + (size_t)bh * p.S * DK;
  const TIn* Q = static_cast<const TIn*>(p.Q) + (size_t)bh * p.S * DK;
  const TIn* V = static_cast<const TIn*>(p.V) + (size_t)bh * p.S * p.DV + col;

  float4_t C[KT];
#pragma unroll
  for (int k = 0; k < KT; ++k)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      C[k][r] = p.C0 ? p.C0[((size_t)bh * DK + 16 * k + 4 * grp + r) * p.DV + col] : 0.0f;

  for (int c = 0; c < p.Nc; ++c) {
    const int t0 = c * L;
    const size_t at = (size_t)bh * p.Nc + c;
    // this lane's values of V: rows 16 rt + 4 grp + r of its column
    float4_t v[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = t0 + 16 * rt + 4 * grp + r;
        v[rt][r] = t < p.S ? load1(V + (size_t)t * p.DV) : 0.0f;
      }
    __syncthreads();  // the chunk before is read out
    stage_rows<TIn, L, DK>(s_K, W::kLd, W::kPlane, K, t0, p.S, tid, THREADS);
    if constexpr (FWD) stage_rows<TIn, L, DK>(s_Q, W::kLd, W::kPlane, Q, t0, p.S, tid, THREADS);
    stage_square<L>(s_T, W::kLdS, W::kPlaneS, p.T + at * L * L, tid, THREADS);
    if constexpr (FWD) stage_square<L>(s_P, W::kLdS, W::kPlaneS, p.P + at * L * L, tid, THREADS);
    if (tid < L) {
      s_e[tid] = p.e[at * L + tid];
      s_w[tid] = p.w[at * L + tid];
    }
    __syncthreads();

    if constexpr (STATES) {
      float* Cs = p.C_states + at * DK * p.DV + col;
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r) Cs[(size_t)(16 * k + 4 * grp + r) * p.DV] = C[k][r];
    }

    // K C and Q C
    float4_t kc[RT], qc[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) kc[rt] = qc[rt] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) {
      float x[8];
      tiles8(C[2 * ks], C[2 * ks + 1], x);
      const Parts<3> cp = split_parts<3>(x);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int off = (16 * rt + row) * W::kLd + 32 * ks + 4 * grp;
        kc[rt] = mma_parts<NP, 3>(lds_row44<NP>(s_K + off, W::kPlane), cp, kc[rt]);
        if constexpr (FWD) qc[rt] = mma_parts<NP, 3>(lds_row44<NP>(s_Q + off, W::kPlane), cp, qc[rt]);
      }
    }

    // U = T (V - e K C)
    float4_t u[RT];
    {
      Parts<3> xp[TS];
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        float x[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 e = *reinterpret_cast<const float4*>(s_e + 32 * ts + 16 * h + 4 * grp);
          const float ev[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
          for (int r = 0; r < 4; ++r) x[4 * h + r] = v[2 * ts + h][r] - ev[r] * kc[2 * ts + h][r];
        }
        xp[ts] = split_parts<3>(x);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) u[rt] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
      lower_times<L, 3>(s_T, W::kLdS, W::kPlaneS, xp, u, row, grp);
    }
    if constexpr (STATES) {
      float* U = p.U + at * L * p.DV + col;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int r = 0; r < 4; ++r) U[(size_t)(16 * rt + 4 * grp + r) * p.DV] = u[rt][r];
    }

    // H = s (e Q C + P U)
    if constexpr (FWD) {
      Parts<3> up[TS];
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        float x[8];
        tiles8(u[2 * ts], u[2 * ts + 1], x);
        up[ts] = split_parts<3>(x);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float4 e = *reinterpret_cast<const float4*>(s_e + 16 * rt + 4 * grp);
        qc[rt][0] *= e.x;
        qc[rt][1] *= e.y;
        qc[rt][2] *= e.z;
        qc[rt][3] *= e.w;
      }
      lower_times<L, 3>(s_P, W::kLdS, W::kPlaneS, up, qc, row, grp);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = t0 + 16 * rt + 4 * grp + r;
          if (t < p.S) {
            const size_t o = ((size_t)bh * p.S + t) * p.DV + col;
            if (p.h_bf16) store1(static_cast<bf16_t*>(p.H) + o, p.scale * qc[rt][r]);
            else store1(static_cast<float*>(p.H) + o, p.scale * qc[rt][r]);
          }
        }
    }

    // C <- g C + K^T (w U)
    {
      Parts<3> wp[TS];
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        float x[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 w = *reinterpret_cast<const float4*>(s_w + 32 * ts + 16 * h + 4 * grp);
          const float wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int r = 0; r < 4; ++r) x[4 * h + r] = wv[r] * u[2 * ts + h][r];
        }
        wp[ts] = split_parts<3>(x);
      }
      const float g = s_e[L - 1];
#pragma unroll
      for (int k = 0; k < KT; ++k) {
#pragma unroll
        for (int r = 0; r < 4; ++r) C[k][r] *= g;
#pragma unroll
        for (int ts = 0; ts < TS; ++ts)
          C[k] = mma_parts<NP, 3>(lds_col<NP>(s_K, W::kLd, W::kPlane, 32 * ts + 4 * grp, 16, 16 * k, lane), wp[ts],
                                  C[k]);
      }
    }
  }

  if (p.C_out) {
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        p.C_out[((size_t)bh * DK + 16 * k + 4 * grp + r) * p.DV + col] = C[k][r];
  }
}

// The backward walk, last chunk first.  G is the gradient of the state
// behind the chunk:
//   dU = s P^T dH + w K G,   dV = T^T dU,
//   G <- g G + Q^T (s e dH) - K^T (e dV).
// It writes G of every chunk and dV for the gradient kernel, and per column
// slice the chunk's sum of w_t u_t . (K G)_t, one half of <C, G> behind the
// chunk that the gate gradient needs.
template <typename TIn, int DK, int NW>
__global__ __launch_bounds__(64 * NW) void delta_walk_back_kernel(const DeltaParams p) {
  typedef WalkLds<TIn, DK> W;
  constexpr int L = W::L, NP = W::NP, RT = L / 16, TS = L / 32, KT = DK / 16, THREADS = 64 * NW;
  __shared__ uint4 smem[W::kBytes / 16];
  uint16_t* s_K = reinterpret_cast<uint16_t*>(smem);
  uint16_t* s_Q = s_K + NP * W::kPlane;
  uint16_t* s_T = s_Q + NP * W::kPlane;
  uint16_t* s_P = s_T + 3 * W::kPlaneS;
  float* s_e = reinterpret_cast<float*>(s_P + 3 * W::kPlaneS);
  float* s_w = s_e + L;

  const int bh = blockIdx.x % p.BH, slice = blockIdx.x / p.BH;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const int col = (slice * NW + wave) * 16 + row;
  const TIn* K = static_cast<const TIn*>(p.K) + (size_t)bh * p.S * DK;
  const TIn* Q = static_cast<const TIn*>(p.Q) + (size_t)bh * p.S * DK;

  float4_t G[KT];
#pragma unroll
  for (int k = 0; k < KT; ++k)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      G[k][r] = p.dC_out ? p.dC_out[((size_t)bh * DK + 16 * k + 4 * grp + r) * p.DV + col] : 0.0f;

  for (int c = p.Nc - 1; c >= 0; --c) {
    const int t0 = c * L;
    const size_t at = (size_t)bh * p.Nc + c;
    float4_t dh[RT], u[RT];
    const float* U = p.U + at * L * p.DV + col;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * rt + 4 * grp + r;
        float x = 0.0f;
        if (t0 + t < p.S) {
          const size_t o = ((size_t)bh * p.S + t0 + t) * p.DV + col;
          x = p.h_bf16 ? load1(static_cast<const bf16_t*>(p.dH) + o) : load1(static_cast<const float*>(p.dH) + o);
        }
        dh[rt][r] = x;
        u[rt][r] = U[(size_t)t * p.DV];
      }
    __syncthreads();
    stage_rows<TIn, L, DK>(s_K, W::kLd, W::kPlane, K, t0, p.S, tid, THREADS);
    stage_rows<TIn, L, DK>(s_Q, W::kLd, W::kPlane, Q, t0, p.S, tid, THREADS);
    stage_square<L>(s_T, W::kLdS, W::kPlaneS, p.T + at * L * L, tid, THREADS);
    stage_square<L>(s_P, W::kLdS, W::kPlaneS, p.P + at * L * L, tid, THREADS);
    if (tid < L) {
      s_e[tid] = p.e[at * L + tid];
      s_w[tid] = p.w[at * L + tid];
    }
    __syncthreads();

    float* Gs = p.G_states + at * DK * p.DV + col;
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) Gs[(size_t)(16 * k + 4 * grp + r) * p.DV] = G[k][r];

    // K G
    float4_t kg[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) kg[rt] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ks = 0; ks < DK / 32; ++ks) {
      float x[8];
      tiles8(G[2 * ks], G[2 * ks + 1], x);
      const Parts<3> gp = split_parts<3>(x);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        kg[rt] = mma_parts<NP, 3>(lds_row44<NP>(s_K + (16 * rt + row) * W::kLd + 32 * ks + 4 * grp, W::kPlane), gp,
                                  kg[rt]);
    }

    // w K G, its product with u, and s dH as parts
    float anchor = 0.0f;
    Parts<3> hp[TS];
#pragma unroll
    for (int ts = 0; ts < TS; ++ts) {
      float x[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 w = *reinterpret_cast<const float4*>(s_w + 32 * ts + 16 * h + 4 * grp);
        const float wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float4_t& k4 = kg[2 * ts + h];
          k4[r] *= wv[r];
          anchor += k4[r] * u[2 * ts + h][r];
          x[4 * h + r] = p.scale * dh[2 * ts + h][r];
        }
      }
      hp[ts] = split_parts<3>(x);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) anchor += __shfl_xor(anchor, o, 64);
    if (lane == 0) p.anchor[at * (p.DV / 16) + slice * NW + wave] = anchor;
    upper_times<L, 3>(s_P, W::kLdS, W::kPlaneS, hp, kg, lane, grp);  // dU

    // dV = T^T dU
    float4_t dv[RT];
    {
      Parts<3> xp[TS];
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        float x[8];
        tiles8(kg[2 * ts], kg[2 * ts + 1], x);
        xp[ts] = split_parts<3>(x);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) dv[rt] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
      upper_times<L, 3>(s_T, W::kLdS, W::kPlaneS, xp, dv, lane, grp);
    }
    float* R = p.R + at * L * p.DV + col;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * rt + 4 * grp + r;
        R[(size_t)t * p.DV] = dv[rt][r];
        if (t0 + t < p.S) store1(static_cast<TIn*>(p.dV) + ((size_t)bh * p.S + t0 + t) * p.DV + col, dv[rt][r]);
      }

    // G <- g G + Q^T (s e dH) - K^T (e dV)
    {
      Parts<3> hq[TS], vk[TS];
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        float x[8], y[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 e = *reinterpret_cast<const float4*>(s_e + 32 * ts + 16 * h + 4 * grp);
          const float ev[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[4 * h + r] = p.scale * ev[r] * dh[2 * ts + h][r];
            y[4 * h + r] = -ev[r] * dv[2 * ts + h][r];
          }
        }
        hq[ts] = split_parts<3>(x);
        vk[ts] = split_parts<3>(y);
      }
      const float g = s_e[L - 1];
#pragma unroll
      for (int k = 0; k < KT; ++k) {
#pragma unroll
        for (int r = 0; r < 4; ++r) G[k][r] *= g;
#pragma unroll
        for (int ts = 0; ts < TS; ++ts) {
          G[k] = mma_parts<NP, 3>(lds_col<NP>(s_Q, W::kLd, W::kPlane, 32 * ts + 4 * grp, 16, 16 * k, lane), hq[ts],
                                  G[k]);
          G[k] = mma_parts<NP, 3>(lds_col<NP>(s_K, W::kLd, W::kPlane, 32 * ts + 4 * grp, 16, 16 * k, lane), vk[ts],
                                  G[k]);
        }
      }
    }
  }

  if (p.dC0) {
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        p.dC0[((size_t)bh * DK + 16 * k + 4 * grp + r) * p.DV + col] = G[k][r];
  }
}

// Waves a workgroup, sixteen columns each: as many as still leave a
// workgroup for every CU, since they share the staging of K, Q, T and P.
int walk_waves(int BH, int DV) {
  if (DV % 128 == 0 && (long long)BH * (DV / 128) >= 256) return 8;
  if ((long long)BH * (DV / 64) >= 256) return 4;
  return 2;
}

template <typename TIn, int DK, int NW>
hipError_t launch_nw(const DeltaParams& p, DeltaWalk what, hipStream_t stream) {
  const dim3 grid((unsigned)((long long)p.BH * (p.DV / (16 * NW)))), block(64 * NW);
  switch (what) {
    case DeltaWalk::kForward:
      hipLaunchKernelGGL((delta_walk_kernel<TIn, DK, NW, true, false>), grid, block, 0, stream, p);
      break;
    case DeltaWalk::kStates:
      hipLaunchKernelGGL((delta_walk_kernel<TIn, DK, NW, false, true>), grid, block, 0, stream, p);
      break;
    case DeltaWalk::kBack:
      hipLaunchKernelGGL((delta_walk_back_kernel<TIn, DK, NW>), grid, block, 0, stream, p);
      break;
  }
  return hipGetLastError();
}

template <typename TIn, int DK>
hipError_t launch_dk(const DeltaParams& p, DeltaWalk what, hipStream_t stream) {
  switch (walk_waves(p.BH, p.DV)) {
    case 8: return launch_nw<TIn, DK, 8>(p, what, stream);
    case 4: return launch_nw<TIn, DK, 4>(p, what, stream);
    default: return launch_nw<TIn, DK, 2>(p, what, stream);
  }
}

}  // namespace

hipError_t launch_delta_walk(const DeltaParams& p, DeltaWalk what, hipStream_t stream) {
  if (p.DV <= 0 || p.DV % 64 != 0) return hipErrorInvalidValue;
  switch (p.DK) {
    case 64: return p.qkv_bf16 ? launch_dk<bf16_t, 64>(p, what, stream) : launch_dk<float, 64>(p, what, stream);
    case 128: return p.qkv_bf16 ? launch_dk<bf16_t, 128>(p, what, stream) : launch_dk<float, 128>(p, what, stream);
    case 256: return p.qkv_bf16 ? launch_dk<bf16_t, 256>(p, what, stream) : launch_dk<float, 256>(p, what, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mlstm
