// Gated delta rule: dQ, dK and the gate gradients of every chunk, gfx950.
//
// With C the state entering the chunk, G the gradient of the state behind
// it, U and dV as the two walks left them and e, w, D as in
// delta_prep_kernel.hip:
//   dP = s D o (dH U^T),   dA = -(D o (dV U^T))_strict,
//   dQ = s e dH C^T + dP K,
//   dK = dP^T Q + (dA + dA^T) K - e dV C^T + w U G^T,
//   d log a_t = sum_{r >= t} (q_r . dq_r - v_r . dv_r) + <C behind, G>,
//   d i_t = (1 - b_t) dV_t . (U_t / b_t),
// with the sum over the chunk's own rows only and <C behind, G> = g <C, G> +
// sum_t w_t u_t . (K G)_t formed afresh for every chunk: one running sum over
// the whole sequence would add up the roundings of all tokens behind t.
//
// One workgroup per chunk, four or eight waves: each owns one or two row tiles
// of C and G, which it reads from memory straight into its operands, and
// forms dQ^T and dK^T for them; the 64 x 64 products are spread over the
// waves.  dH, U and dV go through LDS in steps of 32 value columns, two
// buffers deep, with w U and -e dV cut into parts beside them, so that both
// terms of dK add into one accumulator.  Every load is issued a step ahead:
// without that the step took the latency of memory three times over.
//
// 64 heads of 256 x 512 at 8192 tokens: 2.85 ms for 12.4 GB (4.4 TB/s; a
// large copy reaches 5.1), two thirds of them the states.  64 heads of 128 x 128 at
// 2048 tokens: 170 us; 15 of 64 x 192 at 1777 tokens: 34 us.  (1 / b in every
// term of d i: 1.4 % of the first, nothing of the others.)
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
  static constexpr int NB = NP == 1 ? 2 : 3;  // parts of the terms of dK alone, which is stored as TIn
  // Row tiles of the states a wave, waves, and buffers of a step.  At 256 rows
  // a workgroup of eight waves fills a CU's registers, and a second buffer
  // takes a barrier out of the step.  Smaller heads leave room for two
  // workgroups, which hide each other's waits better than a second buffer (64
  // heads of 128 x 128, 2048 tokens: 164 us against 205 with one workgroup and
  // two buffers, and 203 with two row tiles a wave and so half the waves).
  static constexpr int KPW = DK == 256 ? 2 : 1, NW = DK / (16 * KPW), BUFS = DK == 256 ? 2 : 1;
  static constexpr int kLdT = 40, kPlaneT = L * kLdT;  // 32 value columns
  // planes of a step: dH, U, dV, w U, -e dV
  static constexpr int kU = NH * kPlaneT, kR = kU + 3 * kPlaneT, kUw = kR + NB * kPlaneT, kRe = kUw + NB * kPlaneT;
  static constexpr int kStage = kRe + NB * kPlaneT;
  // behind the last step, in the same space: K, then Q, dP and dA + dA^T
  static constexpr int kLd = DK + 8, kPlane = L * kLd, kLdS = L + 8, kPlaneS = L * kLdS;
  static constexpr int kAfter = NP * kPlane + (3 + NB) * kPlaneS;
  static constexpr int kBytes = 2 * (BUFS * kStage > kAfter ? BUFS * kStage : kAfter);
};

// This lane's part of 32 value columns of sixteen rows of C or G: eight
// consecutive values.
template <int KPW>
struct StateRows {
  words4_t x[KPW][2];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int lane_off, int row16, int v0) {
#pragma unroll
    for (int i = 0; i < KPW; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        x[i][h] = __builtin_bit_cast(
            words4_t, __builtin_amdgcn_raw_buffer_load_b128(r, lane_off + 16 * h, i * row16 + 4 * v0, 0));
  }
  __device__ __forceinline__ void values(int i, float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(x[i][e >> 2][e & 3]);
  }
};

// Four values of a row: element `off` of a resource over the chunk's rows
// (zeros behind them), from column v0 on.
template <typename T>
struct Quad {
  words4_t x;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int off, int v0) {
    if constexpr (sizeof(T) == 2) {
      const v2i32_t w = __builtin_amdgcn_raw_buffer_load_b64(r, 2 * off, 2 * v0, 0);
      x[0] = (uint32_t)w[0];
      x[1] = (uint32_t)w[1];
    } else {
      x = __builtin_bit_cast(words4_t, __builtin_amdgcn_raw_buffer_load_b128(r, 4 * off, 4 * v0, 0));
    }
  }
  __device__ __forceinline__ float4_t values() const {
    if constexpr (sizeof(T) == 2)
      return (float4_t){__uint_as_float(x[0] << 16), __uint_as_float(x[0] & 0xffff0000u), __uint_as_float(x[1] << 16),
                        __uint_as_float(x[1] & 0xffff0000u)};
    else
      return __builtin_bit_cast(float4_t, x);
  }
};

template <int N>
__device__ __forceinline__ void store_quads(uint16_t* p, int plane, const float4_t& x) {
  words2_t w[N];
  split4<N>(x, w);
#pragma unroll
  for (int n = 0; n < N; ++n) *reinterpret_cast<words2_t*>(p + n * plane) = w[n];
}

template <typename TIn, typename TH, int DK>
__global__ __launch_bounds__((64 * GradLds<TIn, TH, DK>::NW)) __attribute__((amdgpu_waves_per_eu(2 * GradLds<TIn, TH, DK>::NW / (DK == 256 ? 8 : 4)))) void
delta_grads_kernel(const DeltaParams p) {
  typedef GradLds<TIn, TH, DK> W;
  constexpr int L = W::L, NP = W::NP, NH = W::NH, NB = W::NB, KPW = W::KPW, NW = W::NW, THREADS = 64 * NW;
  constexpr int RT = L / 16, NT = RT * (RT + 1) / 2, TPW = (NT + NW - 1) / NW;
  constexpr int QUADS = 8 * L, ROWS = (QUADS + THREADS - 1) / THREADS;
  __shared__ uint4 smem[W::kBytes / 16];
  __shared__ float s_red[NW][L];
  __shared__ float s_dvu[L], s_vdv[L], s_cg[NW];
  __shared__ double s_b[L];
  uint16_t* s_K = reinterpret_cast<uint16_t*>(smem);  // and Q
  uint16_t* s_dP = s_K + NP * W::kPlane;
  uint16_t* s_dA = s_dP + 3 * W::kPlaneS;

  const int bh = blockIdx.x / p.Nc, c = blockIdx.x % p.Nc, t0 = c * L;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const size_t at = (size_t)bh * p.Nc + c;
  const int DV = p.DV;
  if (tid < L) s_b[tid] = p.bsum[at * L + tid];

  float4_t dq[KPW][RT], dk[KPW][RT], hu[TPW], ru[TPW];
#pragma unroll
  for (int i = 0; i < KPW; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) dq[i][j] = dk[i][j] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < TPW; ++i) hu[i] = ru[i] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  float cg = 0.0f, dvu[ROWS], vdv[ROWS], qe[ROWS], qw[ROWS], qb[ROWS];

  // this wave's rows of the states, this thread's quads of the rest
  const uint32_t rows_bytes = 16u * KPW * (uint32_t)DV * 4u;
  const size_t first = (at * DK + 16 * KPW * __builtin_amdgcn_readfirstlane(wave)) * DV;
  const __amdgpu_buffer_rsrc_t r_c = make_rsrc(p.C_states + first, rows_bytes);
  const __amdgpu_buffer_rsrc_t r_g = make_rsrc(p.G_states + first, rows_bytes);
  const int state_off = 4 * (row * DV + 8 * grp), row16 = 64 * DV;
  StateRows<KPW> xc, xg;
  Quad<float> qu[ROWS], qr[ROWS];
  Quad<TH> qh[ROWS];
  Quad<TIn> qv[ROWS];
  const uint32_t in_seq = (uint32_t)DV * min(L, p.S - t0);
  const __amdgpu_buffer_rsrc_t r_u = make_rsrc(p.U + at * L * DV, 4u * L * DV);
  const __amdgpu_buffer_rsrc_t r_dv = make_rsrc(p.R + at * L * DV, 4u * L * DV);
  const size_t seq0 = ((size_t)bh * p.S + t0) * DV;
  const __amdgpu_buffer_rsrc_t r_dh = make_rsrc(static_cast<const TH*>(p.dH) + seq0, (uint32_t)sizeof(TH) * in_seq);
  const __amdgpu_buffer_rsrc_t r_v = make_rsrc(static_cast<const TIn*>(p.V) + seq0, (uint32_t)sizeof(TIn) * in_seq);
  // rows behind the chunk (float32 inputs: there are more threads than quads)
  // read as zeros and are not staged
  auto fetch = [&](int v0) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int quad = tid + i * THREADS, off = (quad >> 3) * DV + 4 * (quad & 7);
      qu[i].load(r_u, off, v0);
      qr[i].load(r_dv, off, v0);
      qh[i].load(r_dh, off, v0);
      qv[i].load(r_v, off, v0);
    }
  };
  auto stage = [&](uint16_t* s) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int quad = tid + i * THREADS, o = (quad >> 3) * W::kLdT + 4 * (quad & 7);
      const float4_t u = qu[i].values(), r = qr[i].values(), v = qv[i].values();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dvu[i] += r[e] * (qb[i] * u[e]);
        vdv[i] += v[e] * r[e];
      }
      if (QUADS % THREADS != 0 && quad >= QUADS) continue;
      if constexpr (NH == 1)
        *reinterpret_cast<words2_t*>(s + o) = (words2_t){qh[i].x[0], qh[i].x[1]};
      else
        store_quads<3>(s + o, W::kPlaneT, qh[i].values());
      store_quads<3>(s + W::kU + o, W::kPlaneT, u);
      store_quads<NB>(s + W::kR + o, W::kPlaneT, r);
      store_quads<NB>(s + W::kUw + o, W::kPlaneT, qw[i] * u);
      store_quads<NB>(s + W::kRe + o, W::kPlaneT, qe[i] * r);
    }
  };
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int quad = tid + i * THREADS, t = quad < QUADS ? quad >> 3 : 0;
    dvu[i] = vdv[i] = 0.0f;
    qe[i] = -p.e[at * L + t];
    qw[i] = p.w[at * L + t];
    // 1 / b, for rows with a b: both dV and U carry it, and b^2 is below the
    // smallest float32 value from i = -44 down
    const float inv = t0 + t < p.S ? 1.0f + expf(-p.i_pre[(size_t)bh * p.S + t0 + t]) : 0.0f;
    qb[i] = inv == INFINITY ? 0.0f : inv;
  }
  fetch(0);
  xc.load(r_c, state_off, row16, 0);
  xg.load(r_g, state_off, row16, 0);
  stage(s_K);
  if (DV > 32) fetch(32);

  for (int v0 = 0; v0 < DV; v0 += 32) {
    const uint16_t* s = s_K + (W::BUFS == 2 ? ((v0 >> 5) & 1) * W::kStage : 0);
    __syncthreads();  // this step is staged (and with two buffers the one before read out)
    // the products with the states: rows of C and G, columns t
    Parts<3> cp[KPW];
    Parts<NB> gp[KPW];
#pragma unroll
    for (int i = 0; i < KPW; ++i) {
      float a[8], b[8];
      xc.values(i, a);
      xg.values(i, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) cg += a[e] * b[e];
      cp[i] = split_parts<3>(a);
      gp[i] = split_parts<NB>(b);
    }
    if (v0 + 32 < DV) {
      xc.load(r_c, state_off, row16, v0 + 32);
      xg.load(r_g, state_off, row16, v0 + 32);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const uint16_t* o = s + (16 * j + row) * W::kLdT + 8 * grp;
      const Parts<NH> h = lds_row8<NH>(o, W::kPlaneT);
      const Parts<NB> r = lds_row8<NB>(o + W::kRe, W::kPlaneT), u = lds_row8<NB>(o + W::kUw, W::kPlaneT);
#pragma unroll
      for (int i = 0; i < KPW; ++i) {
        dq[i][j] = mma_parts<3, NH>(cp[i], h, dq[i][j]);
        dk[i][j] = mma_parts<NB, NB>(first_parts<NB>(cp[i]), r, dk[i][j]);
        dk[i][j] = mma_parts<NB, NB>(gp[i], u, dk[i][j]);
      }
    }
    // dH U^T and dV U^T
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int tile = wave + i * NW;
      if (tile >= NT) break;
      int rt, ct;
      lower_tile(tile, rt, ct);
      const uint16_t* a = s + (16 * rt + row) * W::kLdT + 8 * grp;
      const Parts<3> up = lds_row8<3>(s + W::kU + (16 * ct + row) * W::kLdT + 8 * grp, W::kPlaneT);
      hu[i] = mma_parts<NH, 3>(lds_row8<NH>(a, W::kPlaneT), up, hu[i]);
      ru[i] = mma_parts<NB, NB>(lds_row8<NB>(a + W::kR, W::kPlaneT), first_parts<NB>(up), ru[i]);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (v0 + 32 < DV) {
      if (W::BUFS == 1) __syncthreads();  // read out
      stage(s_K + (W::BUFS == 2 ? (((v0 >> 5) + 1) & 1) * W::kStage : 0));
      if (v0 + 64 < DV) fetch(v0 + 64);
    }
  }
  __syncthreads();  // the staged columns are read out: K takes their place

  // row sums of the staged quads, eight lanes a row
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int quad = tid + i * THREADS;
    float a = dvu[i], b = vdv[i];
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      a += __shfl_xor(a, o, 64);
      b += __shfl_xor(b, o, 64);
    }
    if (quad < QUADS && (quad & 7) == 0) {
      s_dvu[quad >> 3] = a;
      s_vdv[quad >> 3] = b;
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
  __syncthreads();
  auto put = [&](uint16_t* dst, float x, int parts) {
#pragma unroll
    for (int n = 0; n < parts; ++n) {
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
        put(s_dP + t * W::kLdS + j, p.scale * D * hu[i][r], 3);
        const float a = j < t ? -D * ru[i][r] : 0.0f;
        put(s_dA + t * W::kLdS + j, a, NB);
        if (j < t) put(s_dA + j * W::kLdS + t, a, NB);
      }
    }
  }
  __syncthreads();

  // scale by rows, then the products within the chunk
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int t = 16 * j + row;
    const float se = p.scale * p.e[at * L + t];
#pragma unroll
    for (int i = 0; i < KPW; ++i) dq[i][j] *= se;
  }
#pragma unroll
  for (int i = 0; i < KPW; ++i)
#pragma unroll
    for (int s = 0; s < L / 32; ++s) {
      const Parts<NP> kt = lds_col<NP>(s_K, W::kLd, W::kPlane, 32 * s + 8 * grp, 4, 16 * (KPW * wave + i), lane);
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int o = (16 * j + row) * W::kLdS + 32 * s + 8 * grp;
        if (s <= j / 2) dq[i][j] = mma_parts<NP, 3>(kt, lds_row8<3>(s_dP + o, W::kPlaneS), dq[i][j]);
        dk[i][j] = mma_parts<NP, NB>(kt, lds_row8<NB>(s_dA + o, W::kPlaneS), dk[i][j]);
      }
    }
  __syncthreads();
  stage_rows<TIn, L, DK>(s_K, W::kLd, W::kPlane, Q, t0, p.S, tid, THREADS);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < KPW; ++i)
#pragma unroll
    for (int s = 0; s < L / 32; ++s) {
      const Parts<NP> qt = lds_col<NP>(s_K, W::kLd, W::kPlane, 32 * s + 8 * grp, 4, 16 * (KPW * wave + i), lane);
#pragma unroll
      for (int j = 0; j < RT; ++j)
        if (s >= j / 2)
          dk[i][j] = mma_parts<NP, NB>(qt, lds_col<NB>(s_dP, W::kLdS, W::kPlaneS, 32 * s + 8 * grp, 4, 16 * j, lane),
                                       dk[i][j]);
    }

  // store, and q . dq by rows
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int t = 16 * j + row;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < KPW; ++i) {
      const int k0 = 16 * (KPW * wave + i) + 4 * grp;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float q = 0.0f;
#pragma unroll
        for (int n = NP - 1; n >= 0; --n) q += bf16_to_f32(s_K[n * W::kPlane + t * W::kLd + k0 + r]);
        dot += q * dq[i][j][r];
      }
      if (t0 + t < p.S) {
        const size_t o = ((size_t)bh * p.S + t0 + t) * DK + k0;
        store4(static_cast<TIn*>(p.dQ) + o, dq[i][j][0], dq[i][j][1], dq[i][j][2], dq[i][j][3]);
        store4(static_cast<TIn*>(p.dK) + o, dk[i][j][0], dk[i][j][1], dk[i][j][2], dk[i][j][3]);
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
      // or it is the first and there is no state to pass (a NaN passes NaN)
      const bool closed = expf(log_sigmoid(f)) == 0.0f || (t0 + t == 0 && !p.C0 && f == f);
      p.d_f[o] = closed ? 0.0f : d / (1.0f + expf(f));
      const float beta = 1.0f / (1.0f + expf(-ip));
      // 1 - b as sigmoid(-i): subtracted from one it would keep no digits near b = 1
      p.d_i[o] = beta == 0.0f ? 0.0f : s_dvu[t] / (1.0f + expf(ip));
    }
  }
}

template <typename TIn, typename TH>
hipError_t launch_types(const DeltaParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)((long long)p.BH * p.Nc));
  switch (p.DK) {
    case 64: hipLaunchKernelGGL((delta_grads_kernel<TIn, TH, 64>), grid, dim3(64 * GradLds<TIn, TH, 64>::NW), 0, stream, p); break;
    case 128: hipLaunchKernelGGL((delta_grads_kernel<TIn, TH, 128>), grid, dim3(64 * GradLds<TIn, TH, 128>::NW), 0, stream, p); break;
    case 256: hipLaunchKernelGGL((delta_grads_kernel<TIn, TH, 256>), grid, dim3(64 * GradLds<TIn, TH, 256>::NW), 0, stream, p); break;
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
