// Selective scan, forward walk, gfx950.
//   d = softplus(dt + bias),  u = d x
//   h = exp(d A) h + u B,  y = (C . h + D x) z sigmoid(z)
//
// A workgroup has 64 channels, one a lane, and four waves, which have a quarter
// of the N states each: h stays in registers.  B and C are the same for a whole
// wave; they are taken from a float32 copy by scalar loads and are scalar
// operands.  Tiles of sixteen tokens: a wave turns x and dt of four of them into
// d and u for all waves through LDS, walks the sixteen tokens with its states,
// and leaves its part of C . h in LDS, where the waves add four tokens each.
//
// Few channels leave compute units idle: the sequence is then cut into chunks
// that are walked side by side, first each from a zero state (what it leaves,
// and the sum of d, whose product with A is the log of the chunk's decay), then
// from the state that the chunks before it leave.
#include "scan_common.h"

namespace mlstm {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves, kQuad = 4;
static_assert(kScanTile == kWaves * kQuad, "a wave prepares four tokens of a tile");

// Read-only memory at an address that a whole wave shares.
typedef const float __attribute__((address_space(4)))* uniform_t;
typedef const float4_t __attribute__((address_space(4)))* uniform4_t;

// The value is waited for here.
__device__ __forceinline__ void arrived(float x) { asm volatile("" ::"s"(x)); }
__device__ __forceinline__ void arrived_lane(float x) { asm volatile("" ::"v"(x)); }
// The value is formed here, not behind what follows.
__device__ __forceinline__ void formed(float& x) { asm volatile("" : "+v"(x)); }

enum class Mode {
  kOutput,  // y and the final state
  kEnds,    // what a chunk leaves of a zero state, and its sum of d
  kKept,    // the state in front of every eight tokens
  kBoth     // kEnds, and the state gradient that a chunk hands on by itself
};

template <typename T>
__device__ __forceinline__ float at(const View& v, int b, int t, int d) {
  return scan_load(static_cast<const T*>(v.p) + (size_t)b * v.batch + (size_t)t * v.token + d);
}

// The state in front of chunk c: the chunks before it, in order.
template <int NPW>
__device__ __forceinline__ void enter(const ScanParams& p, int b, int c, int d, int n0, const float (&A2)[NPW],
                                      float (&h)[NPW]) {
  const size_t row = ((size_t)b * p.D + d) * p.N + n0;
#pragma unroll
  for (int r = 0; r < NPW; ++r) h[r] = p.h0 ? p.h0[row + r] : 0.0f;
  for (int k = 0; k < c; ++k) {
    const size_t i = ((size_t)b * p.chunks + k) * p.D + d;
    const float s = p.sums[i];
#pragma unroll
    for (int r = 0; r < NPW; ++r) h[r] = fmaf(exp2_fast(s * A2[r]), h[r], p.ends[i * p.N + n0 + r]);
  }
}

template <typename T, int N, Mode MODE, bool GATED>
__global__ __launch_bounds__(kThreads) void scan_kernel(const ScanParams p) {
  constexpr int NPW = N / kWaves;
  constexpr bool OUT = MODE == Mode::kOutput, BACK = MODE == Mode::kBoth, ENTER = OUT || MODE == Mode::kKept;
  constexpr bool COLS = OUT || BACK;      // C is read
  // tokens whose B and C are held at a time: sixteen scalar registers, and sixteen on their way
  constexpr int GROUP = (COLS ? 8 : 16) > NPW ? (COLS ? 8 : 16) / NPW : 1;
  constexpr int GROUPS = kScanTile / GROUP, PER_QUAD = kQuad / GROUP;
  __shared__ float4_t s_d[2][kWaves][64], s_u[2][kWaves][64];
  __shared__ float4_t s_g[BACK ? 2 : 1][kWaves][64];
  __shared__ float4_t s_y[OUT ? 2 : 1][kWaves][kWaves][64];

  const int nd = (p.D + kScanChannels - 1) / kScanChannels;
  const int db = blockIdx.x % nd, bc = blockIdx.x / nd, c = bc % p.chunks, b = bc / p.chunks;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = w * NPW;
  const bool in = db * kScanChannels + lane < p.D;
  // lanes behind the last channel walk along with it and store nothing
  const uint32_t d = in ? db * kScanChannels + lane : p.D - 1;
  const int t0 = c * p.chunk, t1 = min(t0 + p.chunk, p.S);
  const float bias = p.bias ? p.bias[d] : 0.0f, skip = OUT && p.Dskip ? p.Dskip[d] : 0.0f;

  float A2[NPW], h[NPW], W[NPW], G[NPW];
#pragma unroll
  for (int r = 0; r < NPW; ++r) A2[r] = kLog2e * p.A[(size_t)d * N + n0 + r];
  if (ENTER) {
    enter<NPW>(p, b, c, d, n0, A2, h);
  } else {
#pragma unroll
    for (int r = 0; r < NPW; ++r) {
      h[r] = G[r] = 0.0f;
      W[r] = 1.0f;
    }
  }

  typedef typename Raw<T>::type raw_t;
  RowWindow<T, kQuad> vx, vdt, vz, vdy, vy;
  vx.init(p.x.p, b * p.x.batch, p.x.token, d, true);
  vdt.init(p.dt.p, b * p.dt.batch, p.dt.token, d, true);
  if (GATED) vz.init(p.z.p, b * p.z.batch, p.z.token, d, true);
  if (BACK) vdy.init(p.dy, (int64_t)b * p.S * p.D, p.D, d, true);
  if (OUT) vy.init(p.y, (int64_t)b * p.S * p.D, p.D, d, in);

  raw_t rx[kQuad], rdt[kQuad], rz[kQuad], rdy[kQuad];
  float x[kQuad], sum = 0.0f;
  auto fetch = [&](int t) {
    const int tq = t + kQuad * w;
    const auto ax = vx.at(tq, t1), adt = vdt.at(tq, t1);
#pragma unroll
    for (int j = 0; j < kQuad; ++j) rx[j] = Raw<T>::load(ax, vx.off[j]);
#pragma unroll
    for (int j = 0; j < kQuad; ++j) rdt[j] = Raw<T>::load(adt, vdt.off[j]);
    if (BACK) {
      const auto ady = vdy.at(tq, t1);
#pragma unroll
      for (int j = 0; j < kQuad; ++j) rdy[j] = Raw<T>::load(ady, vdy.off[j]);
      if (GATED) {
        const auto az = vz.at(tq, t1);
#pragma unroll
        for (int j = 0; j < kQuad; ++j) rz[j] = Raw<T>::load(az, vz.off[j]);
      }
    }
  };
  // Tokens behind the chunk's end have d = u = 0 and leave the state.
  auto prepare = [&](int buf, int t) {
    float4_t dl, u, g;
#pragma unroll
    for (int j = 0; j < kQuad; ++j) {
      const float step = softplus(Raw<T>::value(rdt[j]) + bias);
      dl[j] = t + kQuad * w + j < t1 ? step : 0.0f;
      x[j] = Raw<T>::value(rx[j]);
      u[j] = dl[j] * x[j];
      if (BACK) {
        g[j] = Raw<T>::value(rdy[j]);
        const float z = GATED ? Raw<T>::value(rz[j]) : 0.0f;
        if (GATED) g[j] *= z * scan_sigmoid(z);
      }
    }
    s_d[buf][w][lane] = dl;
    s_u[buf][w][lane] = u;
    if (BACK) s_g[buf][w][lane] = g;
  };

  // B and C of a group of tokens, and d, u (and dr) of four, are asked for while
  // the group before is worked on.  Scalar loads come back in any order, so the
  // one wait for them is for all: it stands before the next are asked for.
  const uniform_t cols = (uniform_t)(uintptr_t)(p.bc + (size_t)b * p.rows * 2 * N + n0);
  float4_t nB[GROUP][NPW / 4], nC[GROUP][NPW / 4], B[GROUP][NPW / 4], C[GROUP][NPW / 4];
  float4_t nd4, nu4, ng4, d4, u4, g4;
  auto ask = [&](int t) {
#pragma unroll
    for (int j = 0; j < GROUP; ++j)
#pragma unroll
      for (int r = 0; r < NPW / 4; ++r) {
        const uniform_t at = cols + (size_t)t * 2 * N + j * 2 * N + 4 * r;
        nB[j][r] = *(uniform4_t)at;
        if (COLS) nC[j][r] = *(uniform4_t)(at + N);
      }
  };
  auto ask_quad = [&](int buf, int q) {
    nd4 = s_d[buf][q][lane];
    nu4 = s_u[buf][q][lane];
    if (BACK) ng4 = s_g[buf][q][lane];
  };

  if (t0 < t1) {
    fetch(t0);
    ask(t0);
    prepare(0, t0);
    fetch(t0 + kScanTile);
  }
  __syncthreads();
  if (t0 < t1) ask_quad(0, 0);
  int buf = 0;
  for (int t = t0; t < t1; t += kScanTile, buf ^= 1) {
    float xk[kQuad];
    float4_t y;
#pragma unroll
    for (int j = 0; j < kQuad; ++j) xk[j] = x[j];
    if (OUT && GATED) {
      const auto az = vz.at(t + kQuad * w, t1);
#pragma unroll
      for (int j = 0; j < kQuad; ++j) rz[j] = Raw<T>::load(az, vz.off[j]);
    }
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      const int q = i / PER_QUAD, j0 = i % PER_QUAD * GROUP;
#pragma unroll
      for (int j = 0; j < GROUP; ++j)
#pragma unroll
        for (int r = 0; r < NPW / 4; ++r) {
          B[j][r] = nB[j][r];
          if (COLS) C[j][r] = nC[j][r];
          arrived(B[j][r][0]);
        }
      if (j0 == 0) {
        d4 = nd4;
        u4 = nu4;
        if (BACK) g4 = ng4;
        arrived_lane(d4[0]);
        arrived_lane(u4[0]);
        if (BACK) arrived_lane(g4[0]);
        if (q + 1 < kWaves) ask_quad(buf, q + 1);
      }
      // behind the last tile, the same tile again
      ask(i + 1 < GROUPS ? t + (i + 1) * GROUP : t + kScanTile < t1 ? t + kScanTile : t);
      __builtin_amdgcn_sched_barrier(0);
      if (MODE == Mode::kKept && i % (GROUPS / 2) == 0 && in) {
        float* to = p.kept + (((size_t)b * (p.rows / kScanBlock) + t / kScanBlock + q / 2) * p.D + d) * N + n0;
#pragma unroll
        for (int r = 0; r < NPW; r += 4) *reinterpret_cast<float4*>(to + r) = make_float4(h[r], h[r + 1], h[r + 2], h[r + 3]);
      }
#pragma unroll
      for (int j = 0; j < GROUP; ++j) {
        const int k = j0 + j;
        float yk = 0.0f;
        if (!ENTER) sum += d4[k];
#pragma unroll
        for (int r = 0; r < NPW; ++r) {
          const float a = exp2_fast(d4[k] * A2[r]);
          h[r] = fmaf(a, h[r], u4[k] * B[j][r / 4][r % 4]);
          if (OUT) yk = fmaf(C[j][r / 4][r % 4], h[r], yk);
          if (BACK) {
            W[r] *= a;
            G[r] = fmaf(C[j][r / 4][r % 4], W[r] * g4[k], G[r]);
          }
        }
        y[k] = yk;
      }
#pragma unroll
      for (int r = 0; r < NPW; ++r) {
        formed(h[r]);
        if (BACK) formed(G[r]);
      }
      if (OUT && j0 + GROUP == kQuad) s_y[buf][w][q][lane] = y;
      __builtin_amdgcn_sched_barrier(0);
    }
    const bool more = t + kScanTile < t1;
    if (more) {
      prepare(buf ^ 1, t + kScanTile);
      fetch(t + 2 * kScanTile);
    }
    __syncthreads();
    if (more) ask_quad(buf ^ 1, 0);
    if (OUT) {
      float4_t s = s_y[buf][0][w][lane];
#pragma unroll
      for (int k = 1; k < kWaves; ++k) s += s_y[buf][k][w][lane];
      const auto ay = vy.at(t + kQuad * w, t1);
#pragma unroll
      for (int j = 0; j < kQuad; ++j) {
        float v = fmaf(skip, xk[j], s[j]);
        const float z = GATED ? Raw<T>::value(rz[j]) : 0.0f;
        if (GATED) v *= z * scan_sigmoid(z);
        Raw<T>::store(ay, vy.off[j], v);
      }
    }
  }
  if (!in) return;
  if (OUT) {
    if (c == p.chunks - 1 && p.h_out)
#pragma unroll
      for (int r = 0; r < NPW; ++r) p.h_out[((size_t)b * p.D + d) * N + n0 + r] = h[r];
  } else if (!ENTER) {
    const size_t i = ((size_t)b * p.chunks + c) * p.D + d;
#pragma unroll
    for (int r = 0; r < NPW; ++r) {
      p.ends[i * N + n0 + r] = h[r];
      if (BACK) p.grads[i * N + n0 + r] = G[r];
    }
    if (w == 0) p.sums[i] = sum;
  }
}

// Bm and Cm in float32, token after token, zeros behind the sequence.
template <typename T>
__global__ __launch_bounds__(kThreads) void scan_columns_kernel(const ScanParams p) {
  const int64_t n = (int64_t)p.B * p.rows * 2 * p.N;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    const int col = (int)(i % (2 * p.N));
    const int64_t row = i / (2 * p.N);
    const int b = (int)(row / p.rows), t = (int)(row - (int64_t)b * p.rows);
    float v = 0.0f;
    if (t < p.S) v = col < p.N ? at<T>(p.Bm, b, t, col) : at<T>(p.Cm, b, t, col - p.N);
    p.bc[i] = v;
  }
}

template <typename T, int N, Mode MODE>
hipError_t launch_gated(const ScanParams& p, hipStream_t stream) {
  const unsigned nd = (unsigned)((p.D + kScanChannels - 1) / kScanChannels);
  const dim3 grid(nd * (unsigned)p.chunks * (unsigned)p.B);
  if (p.z.p)
    hipLaunchKernelGGL((scan_kernel<T, N, MODE, true>), grid, dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((scan_kernel<T, N, MODE, false>), grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

template <typename T, Mode MODE>
hipError_t launch_states(const ScanParams& p, hipStream_t stream) {
  switch (p.N) {
    case 16: return launch_gated<T, 16, MODE>(p, stream);
    case 32: return launch_gated<T, 32, MODE>(p, stream);
    case 64: return launch_gated<T, 64, MODE>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

template <Mode MODE>
hipError_t launch(const ScanParams& p, hipStream_t stream) {
  return p.bf16 ? launch_states<bf16_t, MODE>(p, stream) : launch_states<float, MODE>(p, stream);
}

hipError_t launch_columns(const ScanParams& p, hipStream_t stream) {
  const int64_t n = ((int64_t)p.B * p.rows * 2 * p.N + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)(n < (1 << 16) ? n : 1 << 16));
  if (p.bf16)
    hipLaunchKernelGGL(scan_columns_kernel<bf16_t>, grid, dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL(scan_columns_kernel<float>, grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

int scan_chunks(int B, int S, int D, int N, bool back) {
  const int width = back ? scan_back_channels(N) : kScanChannels;
  const int64_t groups = (int64_t)B * ((D + width - 1) / width), tiles = ((int64_t)S + kScanTile - 1) / kScanTile;
  const int64_t most = back ? 256 : 768;
  int64_t n = groups > most / 3 ? 1 : most / groups;
  if (n > tiles / 4) n = tiles / 4;
  if (n > 64) n = 64;
  return (int)(n < 1 ? 1 : n);
}

hipError_t launch_scan(const ScanParams& p, hipStream_t stream) {
  hipError_t e = p.S > 0 ? launch_columns(p, stream) : hipSuccess;
  if (e == hipSuccess && p.chunks > 1) e = launch<Mode::kEnds>(p, stream);
  if (e == hipSuccess) e = launch<Mode::kOutput>(p, stream);
  return e;
}

hipError_t launch_scan_states(const ScanParams& p, hipStream_t stream) {
  hipError_t e = launch_columns(p, stream);
  if (e == hipSuccess && p.chunks > 1) e = launch<Mode::kBoth>(p, stream);
  if (e == hipSuccess) e = launch<Mode::kKept>(p, stream);
  return e;
}

}  // namespace mlstm
