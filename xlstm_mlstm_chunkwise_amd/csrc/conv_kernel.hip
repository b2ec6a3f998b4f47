// Short causal convolution of every channel, gfx950, and its gradients.
//   xe = [state, x];  p_t = bias + sum_k w_k xe_{t+k};  y_t = p_t sigmoid(p_t) or p_t
//   g_t = dy_t (d y_t / d p_t);  dxe_j = sum_k w_k g_{j-k}
//   dw_k = sum_t g_t xe_{t+k};   db = sum_t g_t
// Everything is bound by memory: x is read and y written once, in 16-byte
// pieces of adjacent channels, and the rows of the taps stay in registers.
// The backward pass forms p again from the x that it reads anyhow.
#include "delta_common.h"
#include "device_common.h"
#include "kernels.h"

namespace mlstm {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;  // rows of y a thread of the forward pass has

// VEC adjacent channels as they are in memory.
template <typename T, int VEC>
struct Piece {
  T v[VEC];
};
template <>
struct Piece<bf16_t, 8> {
  words4_t v;
};
template <>
struct Piece<bf16_t, 4> {
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

// Thread: VEC channels of kRows rows of y.  Adjacent threads take adjacent
// channels, then the next rows.
template <typename T, int K, int VEC>
__global__ __launch_bounds__(kThreads) void conv_kernel(const ConvParams p) {
  const int nv = (p.D + VEC - 1) / VEC, nr = p.S > 0 ? (p.S + kRows - 1) / kRows : 1;
  const int64_t n = (int64_t)nv * nr * p.B;
  for (int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x; id < n; id += (int64_t)gridDim.x * kThreads) {
    const int64_t run = id / nv;
    const int d = (int)(id - run * nv) * VEC, b = (int)(run / nr), r = (int)(run - (int64_t)b * nr), t0 = r * kRows;
    Piece<T, VEC> raw[kRows + K - 1] = {};
#pragma unroll
    for (int i = 0; i < kRows + K - 1; ++i)
      if (t0 + i < p.S + K - 1) raw[i] = row<T, K, VEC>(p, b, t0 + i, d);
    float w[K][VEC], bias[VEC];
    load_weights<K, VEC>(p, d, w, bias);
    float x[kRows + K - 1][VEC];
#pragma unroll
    for (int i = 0; i < kRows + K - 1; ++i) floats<T, VEC>(raw[i], x[i]);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (t0 + i >= p.S) break;
      float y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float s = bias[e];
#pragma unroll
        for (int k = 0; k < K; ++k) s = fmaf(w[k][e], x[i + k][e], s);
        y[e] = p.silu ? s * sigmoid(s) : s;
      }
      write<T, VEC>(p.y, ((size_t)b * p.S + t0 + i) * p.D + d, rounded<T, VEC>(y));
    }
    if (r == nr - 1 && p.state_out)
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

// Thread: VEC channels of a run of rows j of xe.  It walks up the run with the
// last K rows of xe and the last K values of g in registers, beginning K - 1
// rows below it for the g that reach into it; the next kAhead rows are on their
// way meanwhile.
constexpr int kAhead = 4;
template <typename T, int K, int VEC>
__global__ __launch_bounds__(kThreads) void conv_back_kernel(const ConvParams p) {
  const int nv = (p.D + VEC - 1) / VEC, per = p.runs / p.B, last = p.S + K - 1;
  const int64_t n = (int64_t)nv * p.runs;
  for (int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x; id < n; id += (int64_t)gridDim.x * kThreads) {
    const int64_t run = id / nv;
    const int d = (int)(id - run * nv) * VEC, b = (int)(run / per), j0 = (int)(run - (int64_t)b * per) * p.run;
    const int j1 = min(j0 + p.run, last), first = max(j0 - (K - 1), 0);
    float w[K][VEC], bias[VEC], dw[K][VEC] = {}, db[VEC] = {};
    load_weights<K, VEC>(p, d, w, bias);
    float x[K][VEC], g[K][VEC] = {};
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[k + 1][e] = 0.0f;
      if (first + k < last) floats<T, VEC>(row<T, K, VEC>(p, b, first + k, d), x[k + 1]);
    }
    Piece<T, VEC> rx[kAhead], ry[kAhead];
    auto fetch = [&](int j) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        rx[i] = ry[i] = Piece<T, VEC>{};
        if (j + i < p.S && j + i < j1) {
          rx[i] = row<T, K, VEC>(p, b, j + i + K - 1, d);
          ry[i] = read<T, VEC>(p.dy, ((size_t)b * p.S + j + i) * p.D + d);
        }
      }
    };
    fetch(first);
    for (int ja = first; ja < j1; ja += kAhead) {
      float nx[kAhead][VEC], ny[kAhead][VEC];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        floats<T, VEC>(rx[i], nx[i]);
        floats<T, VEC>(ry[i], ny[i]);
      }
      if (ja + kAhead < j1) fetch(ja + kAhead);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = ja + i;
        if (j >= j1) break;
        float out[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
#pragma unroll
          for (int k = 0; k < K - 1; ++k) x[k][e] = x[k + 1][e];
          x[K - 1][e] = nx[i][e];
#pragma unroll
          for (int k = K - 1; k > 0; --k) g[k][e] = g[k - 1][e];
          float dy = 0.0f;
          if (j < p.S) {
            dy = ny[i][e];
            if (p.silu) {
              float s = bias[e];
#pragma unroll
              for (int k = 0; k < K; ++k) s = fmaf(w[k][e], x[k][e], s);
              const float sg = sigmoid(s);
              dy *= sg * (1.0f + s * (1.0f - sg));
            }
          }
          g[0][e] = dy;
          out[e] = 0.0f;
#pragma unroll
          for (int k = 0; k < K; ++k) out[e] = fmaf(w[k][e], g[k][e], out[e]);
        }
        if (j < j0) continue;
        if (j < p.S) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k][e] = fmaf(g[0][e], x[k][e], dw[k][e]);
            db[e] += g[0][e];
          }
        } else if (p.dstate_out) {
          float add[VEC];
          floats<T, VEC>(read<T, VEC>(p.dstate_out, ((size_t)b * (K - 1) + j - p.S) * p.D + d), add);
#pragma unroll
          for (int e = 0; e < VEC; ++e) out[e] += add[e];
        }
        if (j >= K - 1)
          write<T, VEC>(p.dx, ((size_t)b * p.S + j - (K - 1)) * p.D + d, rounded<T, VEC>(out));
        else if (p.dstate)
          write<T, VEC>(p.dstate, ((size_t)b * (K - 1) + j) * p.D + d, rounded<T, VEC>(out));
      }
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
  const int64_t nv = (p.D + VEC - 1) / VEC, nr = p.S > 0 ? (p.S + kRows - 1) / kRows : 1;
  if (pass == Pass::kForward)
    hipLaunchKernelGGL((conv_kernel<T, K, VEC>), dim3(groups_for(nv * nr * p.B)), dim3(kThreads), 0, stream, p);
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

hipError_t launch_types(const ConvParams& p, Pass pass, hipStream_t stream) {
  if (!wide(p)) return p.bf16 ? launch_taps<bf16_t, 1>(p, pass, stream) : launch_taps<float, 1>(p, pass, stream);
  if (!p.bf16) return launch_taps<float, 4>(p, pass, stream);
  return pass == Pass::kBack ? launch_taps<bf16_t, 4>(p, pass, stream) : launch_taps<bf16_t, 8>(p, pass, stream);
}

}  // namespace

void conv_runs(int B, int S, int D, int K, int* run, int* runs) {
  const int64_t lanes = (int64_t)B * ((D + 3) / 4), rows = (int64_t)S + K - 1;
  int64_t per = (2048 * 64 + lanes - 1) / lanes, len = (rows + per - 1) / per;
  if (len < 16) len = 16;
  if (len > 512) len = 512;
  *run = (int)len;
  *runs = (int)((rows + len - 1) / len) * B;
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
