// Short causal convolution of every channel, gfx950, and its gradients.
//   xe = [state, x];  p_t = bias + sum_k w_k xe_{t+k};  y_t = p_t sigmoid(p_t) or p_t
//   g_t = dy_t (d y_t / d p_t);  dxe_j = sum_k w_k g_{j-k}
//   dw_k = sum_t g_t xe_{t+k};   db = sum_t g_t
// Bound by memory: x is read and y written once, in pieces of adjacent channels,
// and the rows of the taps stay in registers.  The backward pass forms p again
// from the x that it reads anyhow.  8 sequences of 8192 x 4096, four taps, bf16:
// forward 205 us for 1.07 GB (5.2 TB/s; threads of eight rows, which read three
// rows and the weights again for each, 303 us), backward 334-356 us for 1.61 GB
// (4.7 TB/s; vector issue, some 33 instructions a value, 89 % of the cycles; with
// addresses advanced row by row 342-348 us) and 7 us for the partial sums.
#include <type_traits>

#include "delta_common.h"
#include "device_common.h"
#include "kernels.h"

namespace mlstm {
namespace {

constexpr int kThreads = 256;

// VEC adjacent channels as they are in memory.
template <typename T, int VEC>
struct Piece {
  T v[VEC];
};
template <>
struct Piece<bf16_t, 4> {
  words2_t v;
};
template <>
struct Piece<bf16_t, 2> {
  uint32_t v[1];
};
template <>
struct Piece<float, 2> {
  words2_t v;
};
template <>
struct Piece<float, 4> {
  words4_t v;
};

template <typename T, int VEC>
__device__ __forceinline__ Piece<T, VEC> read(const void* base, size_t i) {
  return *reinterpret_cast<const Piece<T, VEC>*>(static_cast<const T*>(base) + i);
}
template <typename T, int VEC>
__device__ __forceinline__ void write(void* base, size_t i, const Piece<T, VEC>& x) {
  *reinterpret_cast<Piece<T, VEC>*>(static_cast<T*>(base) + i) = x;
}
template <typename T, int VEC>
__device__ __forceinline__ void floats(const Piece<T, VEC>& x, float (&f)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    if constexpr (sizeof(T) == 2 && VEC > 1)
      f[e] = __uint_as_float(e % 2 ? x.v[e / 2] & 0xffff0000u : x.v[e / 2] << 16);
    else if constexpr (sizeof(T) == 2)
      f[e] = bf16_to_f32(x.v[e].bits);
    else if constexpr (VEC > 1)
      f[e] = __uint_as_float(x.v[e]);
    else
      f[e] = x.v[e];
  }
}
template <typename T, int VEC>
__device__ __forceinline__ Piece<T, VEC> rounded(const float (&f)[VEC]) {
  Piece<T, VEC> x;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    if constexpr (sizeof(T) == 2 && VEC > 1) {
      if (e % 2 == 0) x.v[e / 2] = round_bf16x2(f[e], f[e + 1]);
    } else if constexpr (sizeof(T) == 2) {
      x.v[e].bits = f32_to_bf16(f[e]);
    } else if constexpr (VEC > 1) {
      x.v[e] = __float_as_uint(f[e]);
    } else {
      x.v[e] = f[e];
    }
  }
  return x;
}

__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

template <int K, int VEC>
__device__ __forceinline__ void load_weights(const ConvParams& p, int d, float (&w)[K][VEC], float (&b)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][e] = p.weight[(size_t)(d + e) * K + k];
    b[e] = p.bias ? p.bias[d + e] : 0.0f;
  }
}

// Row i of xe for the channels from d on.
template <typename T, int K, int VEC>
__device__ __forceinline__ Piece<T, VEC> row(const ConvParams& p, int b, int i, int d) {
  if (i >= K - 1) return read<T, VEC>(p.x.p, (size_t)b * p.x.batch + (size_t)(i - (K - 1)) * p.x.token + d);
  if (p.state) return read<T, VEC>(p.state, ((size_t)b * (K - 1) + i) * p.D + d);
  return Piece<T, VEC>{};
}

// Thread: VEC channels of a run of rows of y, walked with the last K rows of xe
// in registers and the next kAhead on their way.  Adjacent threads take adjacent
// channels, then the next run.
constexpr int kAhead = 4;
template <typename T, int K, int VEC>
__global__ __launch_bounds__(kThreads) void conv_kernel(const ConvParams p) {
  const int nv = (p.D + VEC - 1) / VEC, nr = p.runs / p.B;
  const int64_t n = (int64_t)nv * p.runs;
  for (int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x; id < n; id += (int64_t)gridDim.x * kThreads) {
    const int64_t run = id / nv;
    const int d = (int)(id - run * nv) * VEC, b = (int)(run / nr), t0 = (int)(run - (int64_t)b * nr) * p.run;
    const int t1 = min(t0 + p.run, p.S);
    const T* px = static_cast<const T*>(p.x.p) + (size_t)b * p.x.batch + d;
    T* py = static_cast<T*>(p.y) + (size_t)b * p.S * p.D + d;
    Piece<T, VEC> raw[kAhead];
    auto fetch = [&](int t) {  // behind the last row, the last again
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        raw[i] = *reinterpret_cast<const Piece<T, VEC>*>(px + (int64_t)min(t + i, t1 - 1) * p.x.token);
    };
    float w[K][VEC], bias[VEC], x[K][VEC];
    if (t0 < t1) {
      Piece<T, VEC> before[K - 1];
#pragma unroll
      for (int k = 0; k < K - 1; ++k) before[k] = row<T, K, VEC>(p, b, t0 + k, d);
      fetch(t0);
      load_weights<K, VEC>(p, d, w, bias);
#pragma unroll
      for (int k = 0; k < K - 1; ++k) floats<T, VEC>(before[k], x[k + 1]);
    }
    for (int ta = t0; ta < t1; ta += kAhead) {
      float nx[kAhead][VEC];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) floats<T, VEC>(raw[i], nx[i]);
      fetch(ta + kAhead);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        float y[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
#pragma unroll
          for (int k = 0; k < K - 1; ++k) x[k][e] = x[k + 1][e];
          x[K - 1][e] = nx[i][e];
          float s = bias[e];
#pragma unroll
          for (int k = 0; k < K; ++k) s = fmaf(w[k][e], x[k][e], s);
          y[e] = p.silu ? s * sigmoid(s) : s;
        }
        if (ta + i < t1)
          *reinterpret_cast<Piece<T, VEC>*>(py + (size_t)(ta + i) * p.D) = rounded<T, VEC>(y);
      }
    }
    if (t0 + p.run >= p.S && p.state_out)
      for (int i = 0; i < K - 1; ++i)
        write<T, VEC>(p.state_out, ((size_t)b * (K - 1) + i) * p.D + d, row<T, K, VEC>(p, b, p.S + i, d));
  }
}

// One token: the K - 1 rows of the state are read before any is written, so
// that state_out may be the state itself.
template <typename T, int K, int VEC>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(const ConvParams p) {
  const int nv = (p.D + VEC - 1) / VEC;
  const int64_t n = (int64_t)nv * p.B;
  for (int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x; id < n; id += (int64_t)gridDim.x * kThreads) {
    const int b = (int)(id / nv), d = (int)(id - (int64_t)b * nv) * VEC;
    Piece<T, VEC> raw[K];
#pragma unroll
    for (int i = 0; i < K; ++i) raw[i] = row<T, K, VEC>(p, b, i, d);
    float w[K][VEC], s[VEC];
    load_weights<K, VEC>(p, d, w, s);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float x[VEC];
      floats<T, VEC>(raw[k], x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[e] = fmaf(w[k][e], x[e], s[e]);
    }
    if (p.silu) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[e] *= sigmoid(s[e]);
    }
    write<T, VEC>(p.y, (size_t)b * p.D + d, rounded<T, VEC>(s));
#pragma unroll
    for (int i = 0; i < K - 1; ++i) write<T, VEC>(p.state_out, ((size_t)b * (K - 1) + i) * p.D + d, raw[i + 1]);
  }
}

// Thread: VEC channels of a run of tokens.  It walks up the run and K - 1 rows
// past it, whose g reach back into it, with the last K rows of xe and the last K
// values of g in registers and the next kAhead rows on their way.  Row j of xe's
// gradient is complete with g_j: token j - (K - 1), or a row of the state's.
template <typename T, int K, int VEC>
__global__ __launch_bounds__(kThreads) void conv_back_kernel(const ConvParams p) {
  const int nv = (p.D + VEC - 1) / VEC, per = p.runs / p.B;
  const int64_t n = (int64_t)nv * p.runs;
  for (int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x; id < n; id += (int64_t)gridDim.x * kThreads) {
    const int64_t run = id / nv;
    const int d = (int)(id - run * nv) * VEC, b = (int)(run / per), t0 = (int)(run - (int64_t)b * per) * p.run;
    const int t1 = min(t0 + p.run, p.S), last = max(p.S - 1, 0);
    const T* px = static_cast<const T*>(p.x.p) + (size_t)b * p.x.batch + d;
    const T* py = static_cast<const T*>(p.dy) + (size_t)b * p.S * p.D + d;
    T* pdx = static_cast<T*>(p.dx) + (size_t)b * p.S * p.D + d;
    Piece<T, VEC> rx[kAhead], ry[kAhead];
    auto fetch = [&](int j) {  // behind the last row, the last again
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int t = min(j + i, last);
        rx[i] = *reinterpret_cast<const Piece<T, VEC>*>(px + (int64_t)t * p.x.token);
        ry[i] = *reinterpret_cast<const Piece<T, VEC>*>(py + (size_t)t * p.D);
      }
    };
    float w[K][VEC], bias[VEC], dw[K][VEC] = {}, db[VEC] = {}, x[K][VEC] = {}, g[K][VEC] = {};
    if (p.S > 0) {
      Piece<T, VEC> before[K - 1];
#pragma unroll
      for (int k = 0; k < K - 1; ++k) before[k] = row<T, K, VEC>(p, b, t0 + k, d);
      fetch(t0);
#pragma unroll
      for (int k = 0; k < K - 1; ++k) floats<T, VEC>(before[k], x[k + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) rx[i] = ry[i] = Piece<T, VEC>{};
    }
    load_weights<K, VEC>(p, d, w, bias);
    // One row; EDGE: it may lie behind the run, or behind the sequence.
    auto step = [&](auto edge, int j, const Piece<T, VEC>& nx, const Piece<T, VEC>& ny) {
      constexpr bool EDGE = decltype(edge)::value;
      float xn[VEC], yn[VEC], out[VEC];
      floats<T, VEC>(nx, xn);
      floats<T, VEC>(ny, yn);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) x[k][e] = x[k + 1][e];
        x[K - 1][e] = xn[e];
#pragma unroll
        for (int k = K - 1; k > 0; --k) g[k][e] = g[k - 1][e];
        float v = yn[e];
        if (p.silu) {
          float s = bias[e];
#pragma unroll
          for (int k = 0; k < K; ++k) s = fmaf(w[k][e], x[k][e], s);
          const float sg = sigmoid(s);
          v *= sg * fmaf(s, 1.0f - sg, 1.0f);
        }
        if (EDGE && j >= p.S) v = 0.0f;
        g[0][e] = v;
        if (EDGE && j >= t1) v = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][e] = EDGE && j >= t1 ? dw[k][e] : fmaf(v, x[k][e], dw[k][e]);
        db[e] += v;
        out[e] = w[0][e] * g[0][e];
#pragma unroll
        for (int k = 1; k < K; ++k) out[e] = fmaf(w[k][e], g[k][e], out[e]);
      }
      const int t = j - (K - 1);
      if (EDGE && j >= p.S && p.dstate_out) {
        float add[VEC];
        floats<T, VEC>(read<T, VEC>(p.dstate_out, ((size_t)b * (K - 1) + j - p.S) * p.D + d), add);
#pragma unroll
        for (int e = 0; e < VEC; ++e) out[e] += add[e];
      }
      if (t >= t0)
        *reinterpret_cast<Piece<T, VEC>*>(pdx + (size_t)t * p.D) = rounded<T, VEC>(out);
      else if (t < 0 && p.dstate)
        write<T, VEC>(p.dstate, ((size_t)b * (K - 1) + j) * p.D + d, rounded<T, VEC>(out));
    };
    int ja = t0;
    for (; ja + kAhead <= t1; ja += kAhead) {
      Piece<T, VEC> nx[kAhead], ny[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        nx[i] = rx[i];
        ny[i] = ry[i];
      }
      fetch(ja + kAhead);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) step(std::false_type{}, ja + i, nx[i], ny[i]);
    }
    // (at most 2 kAhead - 1 rows)
    for (; ja < t1 + K - 1; ja += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (ja + i < t1 + K - 1) step(std::true_type{}, ja + i, rx[i], ry[i]);
      if (ja + kAhead < t1 + K - 1 && p.S > 0) fetch(ja + kAhead);
    }
    if (p.partial) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int k = 0; k < K; ++k) p.partial[((size_t)run * (K + 1) + k) * p.D + d + e] = dw[k][e];
        p.partial[((size_t)run * (K + 1) + K) * p.D + d + e] = db[e];
      }
    }
  }
}

// Partial sums of 64 (tap or bias, channel), added in the order of their runs:
// sixteen strands, one a wave, then the strands.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void conv_sum_kernel(const ConvParams p) {
  constexpr int STRANDS = kSumThreads / 64;
  __shared__ float s_part[STRANDS][64];
  const int lane = threadIdx.x & 63, strand = threadIdx.x >> 6;
  const size_t n = (size_t)(p.K + 1) * p.D;
  // the same trip count for every thread of a workgroup
  for (size_t i0 = (size_t)blockIdx.x * 64; i0 < n; i0 += (size_t)gridDim.x * 64) {
    const size_t i = i0 + lane;
    float s = 0.0f;
    for (int k = strand; k < p.runs; k += 4 * STRANDS) {
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = i < n && k + j * STRANDS < p.runs ? p.partial[(size_t)(k + j * STRANDS) * n + i] : 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) s += x[j];
    }
    s_part[strand][lane] = s;
    __syncthreads();
    if (strand == 0 && i < n) {
#pragma unroll
      for (int k = 1; k < STRANDS; ++k) s += s_part[k][lane];
      const size_t k = i / p.D, d = i - k * p.D;
      if ((int)k < p.K) {
        if (p.dweight) p.dweight[d * p.K + k] = s;
      } else if (p.dbias) {
        p.dbias[d] = s;
      }
    }
    __syncthreads();  // the strands are read out
  }
}

enum class Pass { kForward, kBack, kStep };

unsigned groups_for(int64_t threads) {
  const int64_t g = (threads + kThreads - 1) / kThreads;
  return (unsigned)(g < (1 << 20) ? g : 1 << 20);
}

template <typename T, int K, int VEC>
hipError_t launch(const ConvParams& p, Pass pass, hipStream_t stream) {
  const int64_t nv = (p.D + VEC - 1) / VEC;
  if (pass == Pass::kForward)
    hipLaunchKernelGGL((conv_kernel<T, K, VEC>), dim3(groups_for(nv * p.runs)), dim3(kThreads), 0, stream, p);
  else if (pass == Pass::kBack)
    hipLaunchKernelGGL((conv_back_kernel<T, K, VEC>), dim3(groups_for(nv * p.runs)), dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((conv_step_kernel<T, K, VEC>), dim3(groups_for(nv * p.B)), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t launch_taps(const ConvParams& p, Pass pass, hipStream_t stream) {
  switch (p.K) {
    case 2: return launch<T, 2, VEC>(p, pass, stream);
    case 3: return launch<T, 3, VEC>(p, pass, stream);
    case 4: return launch<T, 4, VEC>(p, pass, stream);
    default: return hipErrorInvalidValue;
  }
}

// Whether every row of every tensor begins at a multiple of 16 bytes.
bool wide(const ConvParams& p) {
  const int size = p.bf16 ? 2 : 4;
  uintptr_t at = 0;
  for (const void* q : {p.x.p, p.state, (const void*)p.y, (const void*)p.state_out, p.dy, p.dstate_out,
                        (const void*)p.dx, (const void*)p.dstate})
    at |= reinterpret_cast<uintptr_t>(q);
  at |= (uintptr_t)(p.x.batch * size) | (uintptr_t)(p.x.token * size) | (uintptr_t)((int64_t)p.D * size);
  return at % 16 == 0;
}

// Eight bytes a lane forward (8 sequences of 8192 x 4096 in bf16: 205 us, with
// sixteen 206, with single channels, as rows at odd places need them, 272), four
// backward (334 us; eight, in twice the registers, 354, and 13.9 against 17.4 at 3
// of 1777 x 960; single channels 354 against 343 with the sums); in float32 sixteen
// and eight bytes (8 of 4096 x 4096 backward: 323 us, with sixteen 370; 4 of 8192 x
// 4096 forward 204 us, by single channels 214, backward 328 and 362).
hipError_t launch_types(const ConvParams& p, Pass pass, hipStream_t stream) {
  if (!wide(p)) return p.bf16 ? launch_taps<bf16_t, 1>(p, pass, stream) : launch_taps<float, 1>(p, pass, stream);
  if (pass == Pass::kBack) return p.bf16 ? launch_taps<bf16_t, 2>(p, pass, stream) : launch_taps<float, 2>(p, pass, stream);
  return p.bf16 ? launch_taps<bf16_t, 4>(p, pass, stream) : launch_taps<float, 4>(p, pass, stream);
}

}  // namespace

// Runs that leave about 8192 waves of four channels a lane, of 8 rows at least and
// 64 at most; backward 4096, 16 and 512, for every run leaves partial sums.  8
// sequences of 8192 x 4096: forward 205 us in runs of 64 and of 32, 197 to 202 of
// 128; backward with its sums 340 us with half the waves, 348 as here, 367 with
// twice (the median of ten calls varies by 10 us from run to run).
// 3 of 1777 x 960: forward 8.3 us in runs of 8, 9.2 of 4, 9.4 of 16; backward with
// its sums 18.9 us in runs of 16, 21.2 of 8, 19.5 of 32; 1 of 256 x 64 forward 4.2
// in runs of 8, 5.2 of 16.
void conv_runs(int B, int S, int D, bool back, int* run, int* runs) {
  const int64_t lanes = (int64_t)B * ((D + 3) / 4), rows = S;
  const int64_t waves = back ? 4096 : 8192, least = back ? 16 : 8, most = back ? 512 : 64;
  int64_t per = (waves * 64 + lanes - 1) / lanes, len = (rows + per - 1) / per;
  if (len < least) len = least;
  if (len > most) len = most;
  len = (len + kAhead - 1) / kAhead * kAhead;
  *run = (int)len;
  *runs = (int)(rows > 0 ? (rows + len - 1) / len : 1) * B;
}

hipError_t launch_conv(const ConvParams& p, hipStream_t stream) { return launch_types(p, Pass::kForward, stream); }
hipError_t launch_conv_step(const ConvParams& p, hipStream_t stream) { return launch_types(p, Pass::kStep, stream); }

hipError_t launch_conv_back(const ConvParams& p, hipStream_t stream) {
  hipError_t e = launch_types(p, Pass::kBack, stream);
  if (e != hipSuccess || !p.partial) return e;
  const size_t groups = ((size_t)(p.K + 1) * p.D + 63) / 64;
  hipLaunchKernelGGL(conv_sum_kernel, dim3((unsigned)(groups < (1 << 20) ? groups : 1 << 20)), dim3(kSumThreads), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace mlstm
