// Selective scan, gradients, gfx950.  With dr = dy z sigmoid(z) and the state
// gradient g walked from the last token to the first:
//   g_t = C_t dr_t + a_{t+1} g_{t+1},   a = exp(d A),   w_t = a_t g_t h_{t-1}
//   dC_t = sum_c dr h_t,   dB_t = sum_c u g_t,   s = sum_n g B
//   dx = d s + D dr,   d_d = x s + sum_n A w,   ddt = d_d sigmoid(dt + bias)
//   dz = dy r (d silu / dz),   dA = sum_t d w,   dD = sum dr x
//
// The forward walk has left the state in front of every eight tokens.  A block
// of eight tokens forms its states and decays again and keeps them in registers
// while it walks back.  A wave has 32 channels and sixteen states of each: lane l
// holds channels l % 16 and l % 16 + 16 and four states 4 (l / 16) ..., so that
// the sums over states run over four lanes and those over channels over sixteen,
// after two or four values in the lane.  N / 16 waves have the same channels and
// add their sums over states in LDS; waves with the same states add their parts
// of dB and dC there and leave one part for the workgroup's 2048 / N channels.
// Kernels behind this one add those, and the parts of dA, dD and dbias that each
// span of tokens leaves, in a fixed order.
//
// Bound by vector issue: per state and token five slots form h again, nine walk
// back, two to three are sums over lanes, and about 55 a token and channel stand
// around them.  8 sequences of 8192 tokens, 4096 channels of 16 states, bf16: 2.84
// ms in two spans (two waves a SIMD), 87 % of the cycles; in one span 4.0 ms.  The
// sums over channels on the matrix cores, by products with selectors, took 4.85 ms
// against 3.40.
#include "scan_common.h"

namespace mlstm {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves, T = kScanBlock;

__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Lanes 0..31: a summed over lanes l and l + 32; lanes 32..63: b.
__device__ __forceinline__ float halves(float a, float b) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
// Even rows of sixteen lanes: a summed over the row and the next; odd rows: b.
__device__ __forceinline__ float rows(float a, float b) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
// Eight values summed over sixteen lanes: lane l of a row gets value l % 16 / 2.
// Each step adds a lane's partner and, in the half of the lanes that a bank mask
// names, puts the sum of another value in its place: sixteen additions, where
// selecting in front of them takes 22 instructions and waits between them.  A
// lane move reads a register two instructions after its write at the earliest;
// the order below keeps that, with the s_nop where it cannot.
__device__ __forceinline__ float row_sums(float (&v)[8], uint64_t lanes_with_bit_1) {
  float s;
  asm("s_nop 1\n\t"
      "v_add_f32_dpp %1, %1, %1 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %2, %2, %2 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %3, %3, %3 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %4, %4, %4 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %1, %5, %5 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %2, %6, %6 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %3, %7, %7 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %4, %8, %8 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %1, %1, %1 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %2, %2, %2 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %1, %3, %3 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %2, %4, %4 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
      "s_nop 1\n\t"
      "v_add_f32_dpp %1, %1, %1 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %2, %2, %2 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_e64 %0, %1, %2, %9\n\t"
      "s_nop 1\n\t"
      "v_add_f32_dpp %0, %0, %0 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf"
      : "=&v"(s), "+&v"(v[0]), "+&v"(v[1]), "+&v"(v[2]), "+&v"(v[3])
      : "v"(v[4]), "v"(v[5]), "v"(v[6]), "v"(v[7]), "s"(lanes_with_bit_1));
  return s;
}

// The state gradient behind span `c`: the spans behind it, last to first.
__device__ __forceinline__ void enter(const ScanParams& p, int b, int c, const int (&d)[2], int n0,
                                      const float (&A2)[8], float (&ag)[8]) {
  for (int k = p.spans - 1; k > c; k -= 4) {
    float sum[4][2];
    float4_t g[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const size_t at = ((size_t)b * p.spans + max(k - j, c)) * p.D + d[e];
        sum[j][e] = p.span_sums[at];
        g[j][e] = *reinterpret_cast<const float4_t*>(p.grads + at * p.N + n0);
      }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k - j > c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ag[i] = fmaf(decay(sum[j][i / 4], A2[i]), ag[i], g[j][i / 4][i % 4]);
  }
}

template <typename IO, int N, bool GATED>
__global__ __launch_bounds__(kThreads, 2) void scan_back_kernel(const ScanParams p) {
  constexpr int NT = N / 16;                        // waves that share channels, sixteen states each
  constexpr int GROUPS = kWaves / NT, CH = 32 * GROUPS;
  constexpr int R = 4 / NT;                         // items of a lane: a token and a channel each
  constexpr int PER = 2 * N * T / kThreads;         // values of B and C of a block for a thread
  typedef typename Raw<IO>::type raw_t;
  __shared__ float2 s_d[GROUPS][T][16], s_u[GROUPS][T][16], s_dr[GROUPS][T][16];  // both channels of a lane
  __shared__ float4_t s_bc[2][T][2][N / 4];
  __shared__ float s_part[2][GROUPS][T][2 * N];
  __shared__ float s_red[kWaves][T][4][16];
  __shared__ float s_r[GATED ? kWaves : 1][T / 2][4][16];
  __shared__ float4_t s_item[R][kThreads];          // x, sigmoid(dt), dy silu'(z), dy silu(z)
  // What a lane needs once a block stays in LDS: a register more would spill, and
  // a spilled one comes back behind the loads of the next block.
  __shared__ float4_t s_dA[2][kThreads], s_dD[2][kThreads];  // dD and dbias of both channels, in two steps
  __shared__ float4_t s_scalar[kThreads];                    // dt_bias and D of both channels
  __shared__ uint4 s_off[2][kThreads];                       // offsets of x, dt; z, dy of both channels

  const int nd = (p.D + CH - 1) / CH;
  const int db = blockIdx.x % nd, bc = blockIdx.x / nd, c = bc % p.spans, b = bc / p.spans;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nt = w % NT, grp = w / NT;
  const int dl = lane & 15, g = lane >> 4, n0 = 16 * nt + 4 * g;
  const int d0 = db * CH + 32 * grp + dl;
  const bool in[2] = {d0 < p.D, d0 + 16 < p.D};
  const int dch[2] = {in[0] ? d0 : p.D - 1, in[1] ? d0 + 16 : p.D - 1};
  const int t0 = c * p.span, t1 = min(t0 + p.span, p.S);
  const int first = t0 / T, last = (t1 + T - 1) / T;  // blocks

  // i = 4 (channel) + state of four
  float A2[8], ag[8], dA[8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    A2[i] = kLog2e * p.A[(size_t)dch[i / 4] * N + n0 + i % 4];
    ag[i] = p.dh_out && in[i / 4] ? p.dh_out[((size_t)b * p.D + dch[i / 4]) * N + n0 + i % 4] : 0.0f;
  }
  if (c + 1 < p.spans) enter(p, b, c, dch, n0, A2, ag);
  s_dA[0][tid] = s_dA[1][tid] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};

  // Item r of a lane: tokens 2 g and 2 g + 1 of the block with both channels each,
  // which the NT waves of a group share out.
  auto odd = [&](int r) { return NT == 1 ? r / 2 : NT == 2 ? nt : nt / 2; };
  auto ch = [&](int r) { return NT == 4 ? nt % 2 : r % 2; };
  // Rows 2 g, and by another base 2 g + 1, of a block; the end of the span is the end of the resource.
  auto offset = [&](int64_t stride, int k) {
    return in[k] ? (uint32_t)((2 * g * stride + d0 + 16 * k) * (int)sizeof(IO)) : kNowhere;
  };
  auto rows_at = [&](const void* base, int64_t batch, int64_t stride, int blk, int odd) {
    const int t = blk * T + odd, n = __builtin_amdgcn_readfirstlane(min(max(t1 - t, 0), T));
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(base)) + (b * batch + t * stride) * (int64_t)sizeof(IO), 0,
        n * (int)stride * (int)sizeof(IO), 0x00020000);
  };
  s_off[0][tid] = make_uint4(offset(p.x.token, 0), offset(p.x.token, 1), offset(p.dt.token, 0), offset(p.dt.token, 1));
  s_off[1][tid] = make_uint4(GATED ? offset(p.z.token, 0) : 0, GATED ? offset(p.z.token, 1) : 0, offset(p.D, 0), offset(p.D, 1));
  s_scalar[tid] = (float4_t){p.bias ? p.bias[dch[0]] : 0.0f, p.bias ? p.bias[dch[1]] : 0.0f,
                             p.Dskip ? p.Dskip[dch[0]] : 0.0f, p.Dskip ? p.Dskip[dch[1]] : 0.0f};
  s_dD[0][tid] = s_dD[1][tid] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t batch = (int64_t)p.S * p.D;
  raw_t rx[R], rdt[R], rdy[R], rz[R];
  float rbc[PER];
  auto fetch = [&](int blk) {
    const uint4 oa = s_off[0][tid], ob = s_off[1][tid];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int o = odd(r), k = ch(r);
      rx[r] = Raw<IO>::load(rows_at(p.x.p, p.x.batch, p.x.token, blk, o), k ? oa.y : oa.x);
      rdt[r] = Raw<IO>::load(rows_at(p.dt.p, p.dt.batch, p.dt.token, blk, o), k ? oa.w : oa.z);
      rdy[r] = Raw<IO>::load(rows_at(p.dy, batch, p.D, blk, o), k ? ob.w : ob.z);
      if (GATED) rz[r] = Raw<IO>::load(rows_at(p.z.p, p.z.batch, p.z.token, blk, o), k ? ob.y : ob.x);
    }
    const float* from = p.bc + ((size_t)b * p.rows + blk * T) * 2 * N;
#pragma unroll
    for (int i = 0; i < PER; ++i) rbc[i] = from[tid + i * kThreads];
  };
  float2 rh[4];
  auto fetch_state = [&](int blk) {
    const float2* from = reinterpret_cast<const float2*>(p.kept) +
                         (((size_t)b * (p.rows / T) + blk) * (N / 2) + n0 / 2) * p.D;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) rh[2 * k + j] = from[(size_t)j * p.D + dch[k]];
  };
  auto add_parts = [&](int buf, int blk) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + i * kThreads, t = e / (2 * N), col = e % (2 * N);
      float s = s_part[buf][0][t][col];
#pragma unroll
      for (int k = 1; k < GROUPS; ++k) s += s_part[buf][k][t][col];
      if (blk * T + t < t1) p.part_bc[(((size_t)db * p.B + b) * p.S + blk * T + t) * 2 * N + col] = s;
    }
  };
  // the waves of a group have written what they read of each other
  auto group_sync = [] {
    if constexpr (NT > 1)
      __syncthreads();
    else
      wave_sync();
  };
  if (first < last) {
    fetch(last - 1);
    fetch_state(last - 1);
  }
  int buf = 0;
  for (int blk = last - 1; blk >= first; --blk, buf ^= 1) {
    const float4_t bias = s_scalar[tid];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int k = ch(r), q = 2 * g + odd(r);
      const bool ok = (k ? in[1] : in[0]) && blk * T + q < t1;
      const float pre = Raw<IO>::value(rdt[r]) + (k ? bias[1] : bias[0]);
      const float x = Raw<IO>::value(rx[r]), dy = Raw<IO>::value(rdy[r]), dlt = ok ? softplus(pre) : 0.0f;
      float dr = dy, dz = 0.0f;
      if (GATED) {
        const float z = Raw<IO>::value(rz[r]), sz = scan_sigmoid(z);
        dr = dy * (z * sz);
        dz = dy * (sz * fmaf(z, 1.0f - sz, 1.0f));
      }
      reinterpret_cast<float*>(&s_d[grp][q][dl])[k] = dlt;
      reinterpret_cast<float*>(&s_u[grp][q][dl])[k] = dlt * x;
      reinterpret_cast<float*>(&s_dr[grp][q][dl])[k] = dr;
      // (rows behind the last token have a gradient of d too, the one through A)
      s_item[r][tid] = (float4_t){x, ok ? scan_sigmoid(pre) : 0.0f, dz, dr};
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const ScanColumn col = scan_column(tid + i * kThreads, N);
      reinterpret_cast<float*>(s_bc[buf])[(col.token * 2 + col.which) * N + col.state] = rbc[i];
    }
    __syncthreads();
    if (blk < last - 1) add_parts(buf ^ 1, blk + 1);
    float h0[8], a[T][8], h[T][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h0[2 * i] = in[i / 2] ? rh[i].x : 0.0f;
      h0[2 * i + 1] = in[i / 2] ? rh[i].y : 0.0f;
    }
    // h0 is there before the next loads go out: a wait for it behind them would be for them too.  In front of the
    // first block, the first again: a branch would make the waits behind it the longer ones of both ways.
#pragma unroll
    for (int i = 0; i < 8; ++i) formed(h0[i]);
    fetch(max(blk - 1, first));
    fetch_state(max(blk - 1, first));
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const float2 d2 = s_d[grp][t][dl], u2 = s_u[grp][t][dl];
      const float4_t B = s_bc[buf][t][0][4 * nt + g];
      const float de[2] = {d2.x, d2.y}, u[2] = {u2.x, u2.y};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[t][i] = decay(de[i / 4], A2[i]);
        h[t][i] = fmaf(a[t][i], t ? h[t ? t - 1 : 0][i] : h0[i], u[i / 4] * B[i % 4]);
      }
    }
    float y[2];
#pragma unroll
    for (int t = T - 1; t >= 0; --t) {
      const float4_t B = s_bc[buf][t][0][4 * nt + g], C = s_bc[buf][t][1][4 * nt + g];
      const float2 d2 = s_d[grp][t][dl], u2 = s_u[grp][t][dl], r2 = s_dr[grp][t][dl];
      const float de[2] = {d2.x, d2.y}, u[2] = {u2.x, u2.y}, r[2] = {r2.x, r2.y};
      float v[8], s[2], wa[2], yt[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = i / 4, n = i % 4;
        const float gi = fmaf(C[n], r[k], ag[i]);
        v[n] = k ? fmaf(gi, u[k], v[n]) : gi * u[k];
        v[4 + n] = k ? fmaf(h[t][i], r[k], v[4 + n]) : h[t][i] * r[k];
        s[k] = n ? fmaf(gi, B[n], s[k]) : gi * B[n];
        if (GATED) yt[k] = n ? fmaf(C[n], h[t][i], yt[k]) : C[n] * h[t][i];
        ag[i] = a[t][i] * gi;
        const float wi = ag[i] * (t ? h[t ? t - 1 : 0][i] : h0[i]);
        dA[i] = fmaf(de[k], wi, dA[i]);
        wa[k] = n ? fmaf(A2[i], wi, wa[k]) : A2[i] * wi;
      }
      const float v1 = row_sums(v, 0xCCCCCCCCCCCCCCCCull);
      if (lane % 2 == 0) s_part[buf][grp][t][(dl / 8) * N + n0 + dl / 2 % 4] = v1;
      s_red[w][t][g][dl] = rows(halves(s[0], s[1]), halves(wa[0], wa[1]));
      if (GATED) {
        y[t % 2] = halves(yt[0], yt[1]);
        if (t % 2 == 0) s_r[w][t / 2][g][dl] = rows(y[0], y[1]);
      }
    }
    // long sums in two steps: 32 blocks, then those
    const bool flush = blk % 32 == 0 || blk == first;
    if (flush) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        s_dA[k][tid] += (float4_t){dA[4 * k], dA[4 * k + 1], dA[4 * k + 2], dA[4 * k + 3]};
#pragma unroll
        for (int n = 0; n < 4; ++n) dA[4 * k + n] = 0.0f;
      }
    }
    group_sync();
    const float4_t scalar = s_scalar[tid];
    float4_t sums = s_dD[0][tid];
    const uint4 ob = s_off[1][tid];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int k = ch(r), o = odd(r), q = 2 * g + o;
      float s = 0.0f, wa = 0.0f, y1 = 0.0f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        s += s_red[grp * NT + j][q][2 * k][dl];
        wa += s_red[grp * NT + j][q][2 * k + 1][dl];
        if (GATED) y1 += s_r[grp * NT + j][g][o + 2 * k][dl];
      }
      const float4_t item = s_item[r][tid];  // x, sigmoid(dt), dy silu'(z), dr
      const float sk = k ? scalar[3] : scalar[2], dlt = reinterpret_cast<const float*>(&s_d[grp][q][dl])[k];
      const float dx = fmaf(dlt, s, sk * item[3]), ddt = fmaf(item[0], s, kLn2 * wa) * item[1];
      const int sum = NT == 4 ? 0 : r % 2;  // one channel a wave, or both
      sums[sum] = fmaf(item[3], item[0], sums[sum]);
      sums[2 + sum] += ddt;
      const uint32_t off = k ? ob.w : ob.z;
      Raw<IO>::store(rows_at(p.dx, batch, p.D, blk, o), off, dx);
      Raw<IO>::store(rows_at(p.ddt, batch, p.D, blk, o), off, ddt);
      if (GATED) Raw<IO>::store(rows_at(p.dz, batch, p.D, blk, o), off, item[2] * fmaf(sk, item[0], y1));
    }
    if (flush) {
      s_dD[1][tid] += sums;
      sums = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
    }
    s_dD[0][tid] = sums;
    group_sync();
  }
  __syncthreads();
  if (first < last) add_parts(buf ^ 1, first);

  const size_t part = (size_t)b * p.spans + c;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (in[k]) {
      *reinterpret_cast<float4_t*>(p.part_a + (part * p.D + dch[k]) * N + n0) = s_dA[k][tid];
      if (c == 0 && p.dh0)
        *reinterpret_cast<float4*>(p.dh0 + ((size_t)b * p.D + dch[k]) * N + n0) =
            make_float4(ag[4 * k], ag[4 * k + 1], ag[4 * k + 2], ag[4 * k + 3]);
    }
  // dD and dbias of a channel: over the lanes that have it, then over the waves of the group
  float4_t sums = s_dD[1][tid];
  if (NT == 4) sums = nt % 2 ? (float4_t){0.0f, sums[0], 0.0f, sums[2]} : (float4_t){sums[0], 0.0f, sums[2], 0.0f};
  s_red[w][0][g][dl] = rows(halves(sums[0], sums[1]), halves(sums[2], sums[3]));
  group_sync();
  if (nt == 0) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NT; ++j) s += s_red[w + j][0][g][dl];
    const int k = g >> 1;
    if (k ? in[1] : in[0]) p.part_d[(part * 2 + (g & 1)) * p.D + (k ? dch[1] : dch[0])] = s;
  }
}

// dBm, dCm: the parts of the channel groups, in order.
template <typename IO>
__global__ __launch_bounds__(kThreads) void scan_back_columns_kernel(const ScanParams p) {
  const int64_t n = (int64_t)p.B * p.S * 2 * p.N;
  const int groups = (p.D + scan_back_channels(p.N) - 1) / scan_back_channels(p.N);
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    float s = 0.0f;
    for (int k = 0; k < groups; k += 8) {  // the loads of eight go out together
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = p.part_bc[min(k + j, groups - 1) * n + i];
#pragma unroll
      for (int j = 0; j < 8; ++j) s += k + j < groups ? x[j] : 0.0f;
    }
    const int64_t row = i / (2 * p.N);
    const int col = (int)(i - row * 2 * p.N);
    IO* out = static_cast<IO*>(col < p.N ? p.dBm : p.dCm);
    scan_store(out + row * p.N + (col < p.N ? col : col - p.N), s);
  }
}

// dA, dD and dbias: the parts of the chunks, in order.
__global__ __launch_bounds__(kThreads) void scan_back_sums_kernel(const ScanParams p) {
  const int64_t na = (int64_t)p.D * p.N, n = na + 2 * p.D;
  const int parts = p.S > 0 ? p.B * p.spans : 0;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    float s = 0.0f;
    const float* from = i < na ? p.part_a + i : p.part_d + (i - na);
    const int64_t step = i < na ? na : 2 * p.D;
    for (int k = 0; k < parts; k += 8) {  // the loads of eight go out together
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = from[min(k + j, parts - 1) * step];
#pragma unroll
      for (int j = 0; j < 8; ++j) s += k + j < parts ? x[j] : 0.0f;
    }
    if (i < na)
      p.dA[i] = s;
    else if (i < na + p.D) {
      if (p.dDskip) p.dDskip[i - na] = s;
    } else if (p.dbias) {
      p.dbias[i - na - p.D] = s;
    }
  }
}

// No tokens: the state's gradient passes through.
__global__ __launch_bounds__(kThreads) void scan_back_copy_kernel(const ScanParams p) {
  const int64_t n = (int64_t)p.B * p.D * p.N;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads)
    p.dh0[i] = p.dh_out ? p.dh_out[i] : 0.0f;
}

unsigned groups_for(int64_t threads) {
  const int64_t g = (threads + kThreads - 1) / kThreads;
  return (unsigned)(g < 1 ? 1 : g < (1 << 20) ? g : 1 << 20);
}

template <typename IO, int N>
hipError_t launch_gated(const ScanParams& p, hipStream_t stream) {
  const unsigned nd = (unsigned)((p.D + scan_back_channels(N) - 1) / scan_back_channels(N));
  const dim3 grid(nd * (unsigned)p.spans * (unsigned)p.B);
  if (p.z.p)
    hipLaunchKernelGGL((scan_back_kernel<IO, N, true>), grid, dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((scan_back_kernel<IO, N, false>), grid, dim3(kThreads), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((scan_back_columns_kernel<IO>), dim3(groups_for((int64_t)p.B * p.S * 2 * N)), dim3(kThreads), 0,
                     stream, p);
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_states(const ScanParams& p, hipStream_t stream) {
  switch (p.N) {
    case 16: return launch_gated<IO, 16>(p, stream);
    case 32: return launch_gated<IO, 32>(p, stream);
    case 64: return launch_gated<IO, 64>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_scan_back(const ScanParams& p, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (p.S > 0) {
    e = launch_scan_states(p, stream);
    if (e == hipSuccess) e = p.bf16 ? launch_states<bf16_t>(p, stream) : launch_states<float>(p, stream);
  } else if (p.dh0) {
    hipLaunchKernelGGL(scan_back_copy_kernel, dim3(groups_for((int64_t)p.B * p.D * p.N)), dim3(kThreads), 0, stream, p);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(scan_back_sums_kernel, dim3(groups_for((int64_t)p.D * (p.N + 2))), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace mlstm
