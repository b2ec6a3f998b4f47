// Selective scan, forward walk, gfx950.
//   d = softplus(dt + bias),  u = d x
//   h = exp(d A) h + u B,  y = (C . h + D x) z sigmoid(z)
//
// A workgroup has 64 channels, one a lane, and eight waves, which have an eighth
// of the N states each: h stays in registers.  B and C are the same for a whole
// wave; they are taken from a float32 copy by scalar loads and are scalar
// operands.  Tiles of sixteen tokens: a wave turns x and dt of two of them into d
// and u for all waves through LDS, walks the sixteen tokens with its states, and
// leaves its part of C . h in LDS, where the waves add two tokens each.
//
// Bound by vector issue: six slots a state and token (the exponential takes two),
// 33 a token and channel around them.  8 sequences of 8192 tokens, 4096 channels
// of 16 states, bf16: 1.10 ms, 87 % of the cycles (2.2 GB: 0.45 ms at a copy's
// rate).  Four waves of four states each take a tenth fewer instructions but
// leave two waves a SIMD there, and 65 % of the cycles: 1.28 against 1.15 ms.
//
// Few channels leave compute units idle: the sequence is then cut into chunks
// that are walked side by side, first each from a zero state (what it leaves,
// and the sum of d, whose product with A is the log of the chunk's decay), then
// from the state that the chunks before it leave.  One sequence of 65536 tokens,
// 12 chunks: 0.81 and 1.13 ms.
#include <type_traits>

#include "scan_common.h"

namespace mlstm {
namespace {

constexpr int kWaves = kScanWaves, kThreads = 64 * kWaves;
constexpr int kQuads = kScanTile / 4;           // LDS holds four tokens of a channel together
constexpr int kOwn = kScanTile / kWaves;        // tokens of a tile that a wave prepares and finishes
typedef float own_t __attribute__((ext_vector_type(kOwn)));

// Read-only memory at an address that a whole wave shares.
typedef const float __attribute__((address_space(4)))* uniform_t;
typedef float float16_t __attribute__((ext_vector_type(16)));
typedef const float16_t __attribute__((address_space(4)))* uniform16_t;

// The value is waited for here.
__device__ __forceinline__ void arrived(float x) { asm volatile("" ::"s"(x)); }
__device__ __forceinline__ void arrived_lane(float x) { asm volatile("" ::"v"(x)); }

enum class Mode {
  kOutput,  // y and the final state
  kEnds,    // what a chunk leaves of a zero state, and its sum of d
  kKept,    // the state in front of every eight tokens
  kSpans    // kKept, and for every span its sum of d and the state gradient that it hands on by itself
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
    for (int r = 0; r < NPW; ++r) h[r] = fmaf(decay(s, A2[r]), h[r], p.ends[i * p.N + n0 + r]);
  }
}

template <typename T, int N, Mode MODE, bool GATED>
__global__ __launch_bounds__(kThreads) void scan_kernel(const ScanParams p) {
  constexpr int NPW = N / kWaves;          // states of a wave
  constexpr bool OUT = MODE == Mode::kOutput, BACK = MODE == Mode::kSpans, KEEP = MODE == Mode::kKept || BACK;
  constexpr bool ENTER = MODE != Mode::kEnds;
  constexpr bool COLS = OUT || BACK;      // C is read
  constexpr int GROUP = 16 / NPW;         // tokens whose B, or C, one scalar load of 64 bytes brings
  constexpr int GROUPS = kScanTile / GROUP;
  __shared__ float4_t s_d[2][kQuads][64], s_u[2][kQuads][64];
  __shared__ float4_t s_g[BACK ? 2 : 1][kQuads][64];
  __shared__ float4_t s_y[OUT ? 2 : 1][kWaves][kQuads][64];

  const int nd = (p.D + kScanChannels - 1) / kScanChannels;
  const int db = blockIdx.x % nd, bc = blockIdx.x / nd, c = bc % p.chunks, b = bc / p.chunks;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = w * NPW;
  const bool in = db * kScanChannels + lane < p.D;
  // lanes behind the last channel walk along with it and store nothing
  const uint32_t d = in ? db * kScanChannels + lane : p.D - 1;
  const int t0 = c * p.chunk, t1 = min(t0 + p.chunk, p.S);
  const int grads = t0 ? t0 : p.span;  // kSpans: the first token whose gradient counts
  const float bias = p.bias ? p.bias[d] : 0.0f, skip = OUT && p.Dskip ? p.Dskip[d] : 0.0f;

  float A2[NPW], h[NPW], W[NPW], G[NPW];
#pragma unroll
  for (int r = 0; r < NPW; ++r) A2[r] = kLog2e * p.A[(size_t)d * N + n0 + r];
#pragma unroll
  for (int r = 0; r < NPW; ++r) {
    h[r] = G[r] = 0.0f;
    W[r] = 1.0f;
  }
  if (ENTER) enter<NPW>(p, b, c, d, n0, A2, h);

  typedef typename Raw<T>::type raw_t;
  RowWindow<T, kOwn> vx, vdt, vz, vdy, vy;
  vx.init(p.x.p, b * p.x.batch, p.x.token, d, true);
  vdt.init(p.dt.p, b * p.dt.batch, p.dt.token, d, true);
  if (GATED) vz.init(p.z.p, b * p.z.batch, p.z.token, d, true);
  if (BACK) vdy.init(p.dy, (int64_t)b * p.S * p.D, p.D, d, true);
  if (OUT) vy.init(p.y, (int64_t)b * p.S * p.D, p.D, d, in);

  raw_t rx[kOwn], rdt[kOwn], rz[kOwn], rdy[kOwn];
  float sum = 0.0f;
  // this wave's tokens among a tile's, four of a channel together
  auto own = [&](float4_t* tile) -> own_t& {
    return *reinterpret_cast<own_t*>(reinterpret_cast<float*>(&tile[kOwn * w / 4 * 64 + lane]) + kOwn * w % 4);
  };
  auto fetch = [&](int t) {
    const int tq = t + kOwn * w;
    const auto ax = vx.at(tq, t1), adt = vdt.at(tq, t1);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) rx[j] = Raw<T>::load(ax, vx.off[j]);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) rdt[j] = Raw<T>::load(adt, vdt.off[j]);
    if (BACK) {
      // (not for tiles whose gradient is not asked for: no row is inside)
      const int end = t >= grads ? t1 : t;
      const auto ady = vdy.at(tq, end);
#pragma unroll
      for (int j = 0; j < kOwn; ++j) rdy[j] = Raw<T>::load(ady, vdy.off[j]);
      if (GATED) {
        const auto az = vz.at(tq, end);
#pragma unroll
        for (int j = 0; j < kOwn; ++j) rz[j] = Raw<T>::load(az, vz.off[j]);
      }
    }
  };
  // Tokens behind the chunk's end have d = u = 0 and leave the state.
  auto prepare = [&](auto back, int buf, int t, own_t& x) {
    constexpr bool GRAD = decltype(back)::value;
    own_t dl, u, g;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const float step = softplus(Raw<T>::value(rdt[j]) + bias);
      dl[j] = t + kOwn * w + j < t1 ? step : 0.0f;
      x[j] = Raw<T>::value(rx[j]);
      u[j] = dl[j] * x[j];
      if (GRAD) {
        g[j] = Raw<T>::value(rdy[j]);
        const float z = GATED ? Raw<T>::value(rz[j]) : 0.0f;
        if (GATED) g[j] *= z * scan_sigmoid(z);
      }
    }
    own(s_d[buf][0]) = dl;
    own(s_u[buf][0]) = u;
    if (GRAD) own(s_g[buf][0]) = g;
  };

  // B and C of a group of tokens, and d, u (and dr) of the next four or eight, are
  // asked for while the group before is worked on.  Scalar loads come back in any
  // order, so the one wait for them is for all: it stands before the next are
  // asked for.
  const uniform_t cols = (uniform_t)(uintptr_t)(p.bc + (size_t)b * p.rows * 2 * N + w * 32);
  constexpr int QG = GROUP > 4 ? GROUP / 4 : 1;  // quads a group has
  float16_t nB, nC;
  float4_t d4[2][QG], u4[2][QG], g4[2][QG];  // two sets in turn
  auto ask = [&](auto both, int t, int i) {  // group i of the tile from t on
    const uniform_t at = cols + (size_t)t * 2 * N + i * (32 * kWaves);
    nB = *(uniform16_t)at;
    if (decltype(both)::value) nC = *(uniform16_t)(at + 16);
  };
  auto ask_quads = [&](auto back, int buf, int q, int set) {
#pragma unroll
    for (int k = 0; k < QG; ++k) {
      d4[set][k] = s_d[buf][q + k][lane];
      u4[set][k] = s_u[buf][q + k][lane];
      if (decltype(back)::value) g4[set][k] = s_g[buf][q + k][lane];
    }
  };

  // y of a tile whose parts of C . h are in LDS
  auto finish = [&](int buf, int t, int end, const own_t& x) {
    own_t s = own(s_y[buf][0][0]);
#pragma unroll
    for (int k = 1; k < kWaves; ++k) s += own(s_y[buf][k][0]);
    const auto ay = vy.at(t + kOwn * w, end);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      float v = fmaf(skip, x[j], s[j]);
      const float z = GATED ? Raw<T>::value(rz[j]) : 0.0f;
      if (GATED) v *= z * scan_sigmoid(z);
      Raw<T>::store(ay, vy.off[j], v);
    }
  };

  own_t x[2];  // of the tiles in the two buffers
  // A tile: its d and u are in buffer BUF, B and C of its first group on their way.
  // GRAD: it adds to the state gradient of its span.
  auto tile = [&](auto which, auto back, int t) {
    constexpr int BUF = decltype(which)::value;
    constexpr bool GRAD = decltype(back)::value;
    // the tile behind an odd one may be the first whose gradient is asked for
    constexpr bool NEXT = GRAD || (BACK && BUF == 1), READS = OUT || GRAD;
    const bool more = t + kScanTile < t1;
    float4_t y;
    float steps = 0.0f;  // a tile's, then the chunk's: long sums in two steps
    ask_quads(back, BUF, 0, 0);
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      const int q = i * GROUP / 4, j0 = i * GROUP % 4, set = q / QG % 2;
      const float16_t B = nB, C = nC;
      arrived(B[0]);
      if (READS) arrived(C[0]);
      if (j0 == 0) {
#pragma unroll
        for (int k = 0; k < QG; ++k) {
          arrived_lane(d4[set][k][0]);
          arrived_lane(u4[set][k][0]);
          if (GRAD) arrived_lane(g4[set][k][0]);
        }
        if (q + QG < kQuads) ask_quads(back, BUF, q + QG, set ^ 1);
      }
      // behind the last tile, the same tile again
      if (i + 1 < GROUPS)
        ask(std::bool_constant<READS>{}, t, i + 1);
      else
        ask(std::bool_constant<OUT || NEXT>{}, more ? t + kScanTile : t, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (KEEP && i * GROUP % kScanBlock == 0 && in) {
        const size_t block = (size_t)b * (p.rows / kScanBlock) + (t + i * GROUP) / kScanBlock;
        float2* to = reinterpret_cast<float2*>(p.kept) + (block * (N / 2) + n0 / 2) * p.D + d;
#pragma unroll
        for (int r = 0; r < NPW / 2; ++r) to[(size_t)r * p.D] = make_float2(h[2 * r], h[2 * r + 1]);
      }
#pragma unroll
      for (int j = 0; j < GROUP; ++j) {
        const int k = j0 + j;
        const float dk = d4[set][k / 4][k % 4], uk = u4[set][k / 4][k % 4];
        float yk = 0.0f;
        if (!ENTER || GRAD) steps += dk;
#pragma unroll
        for (int r = 0; r < NPW; ++r) {
          const float a = decay(dk, A2[r]);
          h[r] = fmaf(a, h[r], uk * B[j * NPW + r]);
          if (OUT) yk = r ? fmaf(C[j * NPW + r], h[r], yk) : C[j * NPW + r] * h[r];
          if (GRAD) {
            W[r] *= a;
            G[r] = fmaf(C[j * NPW + r], W[r] * g4[set][k / 4][k % 4], G[r]);
          }
        }
        y[k % 4] = yk;
        if (OUT && k % 4 == 3) s_y[BUF][w][q + k / 4][lane] = y;
      }
#pragma unroll
      for (int r = 0; r < NPW; ++r) {
        formed(h[r]);
        if (GRAD) formed(G[r]);
      }
      // the tile before, while the next group's operands come
      if (OUT && i == 0) {
        // (in front of the first tile no row is inside)
        finish(BUF ^ 1, t - kScanTile, t > t0 ? t1 : t - kScanTile, x[BUF ^ 1]);
        if (GATED) {
          const auto az = vz.at(t + kOwn * w, t1);
#pragma unroll
          for (int j = 0; j < kOwn; ++j) rz[j] = Raw<T>::load(az, vz.off[j]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    sum += steps;
    if (BACK && (!more || (t + kScanTile) % p.span == 0)) {
      const size_t i = ((size_t)b * p.spans + t / p.span) * p.D + d;
#pragma unroll
      for (int r = 0; r < NPW; ++r) {
        if (in) p.grads[i * N + n0 + r] = G[r];
        G[r] = 0.0f;
        W[r] = 1.0f;
      }
      if (in && w == 0) p.span_sums[i] = sum;
      sum = 0.0f;
    }
    // behind the last tile too: a branch would make the waits behind it the longer ones of both ways
    prepare(std::bool_constant<NEXT>{}, BUF ^ 1, t + kScanTile, x[BUF ^ 1]);
    fetch(t + 2 * kScanTile);
    __syncthreads();
  };
  if (t0 < t1) {
    fetch(t0);
    ask(std::bool_constant<COLS>{}, t0, 0);
    prepare(std::bool_constant<BACK>{}, 0, t0, x[0]);
    fetch(t0 + kScanTile);
    __syncthreads();
    typedef std::integral_constant<int, 0> even;
    typedef std::integral_constant<int, 1> odd;
    int t = t0;
    if (BACK && t0 == 0) {
      // nothing is in front of the first span (pairs of tiles) that would take its gradient
      for (; t < p.span && t < t1; t += 2 * kScanTile) {
        tile(even{}, std::false_type{}, t);
        tile(odd{}, std::false_type{}, t + kScanTile);
      }
    }
    for (; t < t1; t += 2 * kScanTile) {
      tile(even{}, std::bool_constant<BACK>{}, t);
      if (t + kScanTile >= t1) {
        if (OUT) finish(0, t, t1, x[0]);
        break;
      }
      tile(odd{}, std::bool_constant<BACK>{}, t + kScanTile);
      if (OUT && t + 2 * kScanTile >= t1) finish(1, t + kScanTile, t1, x[1]);
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
    for (int r = 0; r < NPW; ++r) p.ends[i * N + n0 + r] = h[r];
    if (w == 0) p.sums[i] = sum;
  }
}

// Bm and Cm in float32 as the waves read them, zeros behind the sequence.
template <typename T>
__global__ __launch_bounds__(256) void scan_columns_kernel(const ScanParams p) {
  const int tile = kScanTile * 2 * p.N;
  const int64_t n = (int64_t)p.B * p.rows * 2 * p.N;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t q = i / tile;
    const ScanColumn c = scan_column((int)(i - q * tile), p.N);
    const int64_t row = q * kScanTile + c.token;
    const int b = (int)(row / p.rows), t = (int)(row - (int64_t)b * p.rows);
    p.bc[i] = t < p.S ? at<T>(c.which ? p.Cm : p.Bm, b, t, c.state) : 0.0f;
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
  const int64_t n = ((int64_t)p.B * p.rows * 2 * p.N + 255) / 256;
  const dim3 grid((unsigned)(n < (1 << 16) ? n : 1 << 16));
  if (p.bf16)
    hipLaunchKernelGGL(scan_columns_kernel<bf16_t>, grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL(scan_columns_kernel<float>, grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

void scan_cut(ScanParams& p, bool back) {
  const int tiles = p.rows / kScanTile;
  // at most n pieces of whole tiles, two of them at least; every one has tokens
  auto cut = [&](int64_t n, int* pieces, int* length) {
    if (n > tiles / 2) n = tiles / 2;
    if (n > 64) n = 64;
    if (n < 1) n = 1;
    *length = (int)((tiles + n - 1) / n) * kScanTile;
    *pieces = *length ? (p.S + *length - 1) / *length : 1;
  };
  // 512 workgroups are there at a time, two a compute unit; one pass more over the
  // states is paid for more of them (8 chunks of 64 workgroups 2.05 ms, 12 1.97, 16 2.06)
  const int64_t groups = (int64_t)p.B * ((p.D + kScanChannels - 1) / kScanChannels);
  cut(groups <= 256 ? 768 / groups : 1, &p.chunks, &p.chunk);
  p.spans = p.chunks;
  p.span = p.chunk;
  if (back) {
    // 512 workgroups, two a compute unit (states and gradients of 8 sequences of
    // 8192 tokens, 4096 channels of 16 states: 256 workgroups 0.97 + 4.00 ms, 512
    // 1.33 + 2.81, 1024 1.49 + 2.78; of 3 of 1777, 960: 49 + 107, 48 + 81, 52 + 89 us)
    const int ch = scan_back_channels(p.N);
    cut(512 / ((int64_t)p.B * ((p.D + ch - 1) / ch)), &p.spans, &p.span);
    // pairs of tiles in a span, whole spans in a chunk
    p.span = (p.span + 2 * kScanTile - 1) / (2 * kScanTile) * (2 * kScanTile);
    p.spans = p.span ? (p.S + p.span - 1) / p.span : 1;
    if (p.chunks > 1) {
      p.chunk = (p.chunk + p.span - 1) / p.span * p.span;
      p.chunks = (p.S + p.chunk - 1) / p.chunk;
    }
  }
}

hipError_t launch_scan(const ScanParams& p, hipStream_t stream) {
  hipError_t e = p.S > 0 ? launch_columns(p, stream) : hipSuccess;
  if (e == hipSuccess && p.chunks > 1) e = launch<Mode::kEnds>(p, stream);
  if (e == hipSuccess) e = launch<Mode::kOutput>(p, stream);
  return e;
}

hipError_t launch_scan_states(const ScanParams& p, hipStream_t stream) {
  hipError_t e = launch_columns(p, stream);
  if (e == hipSuccess && p.chunks > 1) e = launch<Mode::kEnds>(p, stream);
  if (e == hipSuccess) e = p.spans > 1 ? launch<Mode::kSpans>(p, stream) : launch<Mode::kKept>(p, stream);
  return e;
}

}  // namespace mlstm
