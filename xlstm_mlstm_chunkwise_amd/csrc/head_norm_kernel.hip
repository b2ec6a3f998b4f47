// Head norm: the layer norm of every row of H over its D values, with a
// weight and a bias per head and channel, gfx950.
//   n = (x - mean) rstd,  rstd = 1 / sqrt(var + eps),  y = w n + c
//   g = w dy,  dx = rstd (g - mean(g) - n mean(g n))
//   dw = sum over the head's rows of dy n,  dc = the same sum of dy
// x and dx are (B, NH, S, D), y and dy (B, S, NH, D): the norm also turns the
// cell's layout into the one of the projection behind it, so no transposed
// copy is made.
//
// Both passes are bound by memory.  A row is held in registers by 8, 16, 32
// or 64 lanes, eight values each, and read once; mean and variance take two
// passes over the registers.  The backward pass forms them again from x,
// which it reads anyhow, instead of reading saved ones.  Its workgroups take
// the rows of one head, keep their sums of dy n and dy in registers, and
// leave one partial sum each; a second kernel adds the partial sums in a
// fixed order, so that equal inputs give equal bits.
//
// 64 heads of 512 values, 8192 rows each, bf16: forward 190-197 us for 1.07 GB
// (5.5 TB/s; a large copy reaches 5.1), backward 350 us for 1.61 GB (4.6 TB/s;
// contiguous rows a workgroup, twice the workgroups or non-temporal accesses:
// 341-353 us) and 5.6 us for the partial sums.
#include "delta_common.h"
#include "kernels.h"

namespace mlstm {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void store8f(T* p, const float (&x)[8]) {
  store4(p, x[0], x[1], x[2], x[3]);
  store4(p + 4, x[4], x[5], x[6], x[7]);
}
template <>
__device__ __forceinline__ void store8f<bf16_t>(bf16_t* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(round_bf16x2(x[0], x[1]), round_bf16x2(x[2], x[3]),
                                            round_bf16x2(x[4], x[5]), round_bf16x2(x[6], x[7]));
}

// Sum over the LPR lanes of a row, in every lane, without LDS: within sixteen
// lanes by quad permutes and mirrors, across them by row swaps (of a value
// with itself: each half of the result holds one operand of the sum).
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
  auto plus = [&](auto moved) { x += __int_as_float(moved(__float_as_int(x))); };
  plus([](int v) { return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true); });   // lane ^ 1
  plus([](int v) { return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true); });   // lane ^ 2
  plus([](int v) { return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true); });  // the other quad of eight
  if constexpr (LPR >= 16) plus([](int v) { return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true); });
  if constexpr (LPR >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if constexpr (LPR == 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return x;
}

// n and rstd of a row held eight values a lane; `in`: the lane has values.
template <int LPR>
__device__ __forceinline__ float normalise(float (&x)[8], bool in, float inv_d, float eps) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s += x[e];
  const float mean = row_sum<LPR>(in ? s : 0.0f) * inv_d;
  float q = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] -= mean;
    q += x[e] * x[e];
  }
  const float rstd = 1.0f / sqrtf(row_sum<LPR>(in ? q : 0.0f) * inv_d + eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= rstd;
  return rstd;
}

// Eight values a lane as they are in memory: they become floats where they are
// used, so that nothing waits for the loads before.
template <typename T>
struct Raw8 {
  words4_t w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, bool in) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      w[i] = (words4_t){0u, 0u, 0u, 0u};
      if (in) w[i] = reinterpret_cast<const words4_t*>(p)[i];
    }
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (sizeof(T) == 2)
        x[e] = __uint_as_float(e % 2 ? w[0][e / 2] & 0xffff0000u : w[0][e / 2] << 16);
      else
        x[e] = __uint_as_float(w[e / 4][e % 4]);
    }
  }
};

// R rows one after another: their loads go out together, and a head's weight
// and bias (64 bytes a lane against a bf16 row's 16) are read once for them.
template <typename TX, typename TY, int LPR, int R>
__global__ __launch_bounds__(kThreads) void head_norm_kernel(const HeadNormParams p) {
  constexpr int RPB = kThreads / LPR;  // row groups a workgroup
  const uint32_t rows = (uint32_t)p.B * p.NH * p.S;
  const uint32_t r0 = (blockIdx.x * RPB + threadIdx.x / LPR) * R;
  const int d = 8 * (threadIdx.x % LPR);
  const bool in = d < p.D;
  Raw8<TX> raw[R];
#pragma unroll
  for (int j = 0; j < R; ++j) raw[j].load(static_cast<const TX*>(p.x) + (size_t)(r0 + j) * p.D + d, in && r0 + j < rows);
  uint32_t bh = r0 / p.S, t = r0 - bh * p.S, h = bh % p.NH;
  float w[8], c[8];
  auto affine = [&] {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] = 1.0f;
      c[e] = 0.0f;
    }
    if (in && p.weight) Ops<float>::load8(p.weight + (size_t)h * p.D + d, w);
    if (in && p.bias) Ops<float>::load8(p.bias + (size_t)h * p.D + d, c);
  };
  affine();
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float x[8];
    raw[j].floats(x);
    normalise<LPR>(x, in, 1.0f / (float)p.D, p.eps);
    if (in && r0 + j < rows) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * w[e] + c[e];
      store8f(static_cast<TY*>(p.y) + ((size_t)(bh / p.NH * p.S + t) * p.NH + h) * p.D + d, x);
    }
    if (j + 1 < R && ++t == (uint32_t)p.S) {
      t = 0;
      h = ++bh % p.NH;
      affine();
    }
  }
}

template <typename TX, typename TY, int LPR>
__global__ __launch_bounds__(kThreads) void head_norm_back_kernel(const HeadNormParams p) {
  constexpr int RPB = kThreads / LPR;
  __shared__ float s_sum[2][RPB][8 * LPR];
  const int h = blockIdx.x % p.NH, blk = blockIdx.x / p.NH;
  const int g = threadIdx.x / LPR, d = 8 * (threadIdx.x % LPR);
  const bool in = d < p.D;
  const float inv_d = 1.0f / (float)p.D;
  float w[8], dw[8], dc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    w[e] = 1.0f;
    dw[e] = dc[e] = 0.0f;
  }
  if (in && p.weight) Ops<float>::load8(p.weight + (size_t)h * p.D + d, w);
  const uint32_t rows = (uint32_t)p.B * p.S, step = (uint32_t)p.blocks * RPB;
  auto offset = [&](uint32_t i) {
    const uint32_t b = i / p.S, t = i - b * p.S;
    return ((size_t)(b * p.NH + h) * p.S + t) * p.D + d;
  };
  Raw8<TX> rx;
  Raw8<TY> ry;
  auto fetch = [&](uint32_t i) {
    const bool ok = in && i < rows;
    rx.load(static_cast<const TX*>(p.x) + (ok ? offset(i) : 0), ok);
    ry.load(static_cast<const TY*>(p.dy) + ((size_t)i * p.NH + h) * p.D + d, ok);
  };
  if (rows) fetch(blk * RPB + g);
  // the same trip count for every lane: the sums of a row run over lanes; the
  // next row's loads are on their way while this one is worked on
  for (uint32_t i0 = blk * RPB; i0 < rows; i0 += step) {
    const uint32_t i = i0 + g;
    const bool ok = in && i < rows;
    float n[8], dy[8];
    rx.floats(n);
    ry.floats(dy);
    if (i0 + step < rows) fetch(i + step);
    const float rstd = normalise<LPR>(n, in, inv_d, p.eps);
    float sg = 0.0f, sgn = 0.0f, gw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      gw[e] = w[e] * dy[e];
      sg += gw[e];
      sgn += gw[e] * n[e];
    }
    sg = row_sum<LPR>(ok ? sg : 0.0f) * inv_d;
    sgn = row_sum<LPR>(ok ? sgn : 0.0f) * inv_d;
    if (ok) {
      float dx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dx[e] = rstd * (gw[e] - sg - n[e] * sgn);
        dw[e] += dy[e] * n[e];
        dc[e] += dy[e];
      }
      store8f(static_cast<TX*>(p.dx) + offset(i), dx);
    }
  }
  if (!p.partial) return;
  Ops<float>::store8(&s_sum[0][g][d], dw);
  Ops<float>::store8(&s_sum[1][g][d], dc);
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
    const int which = i / p.D, dd = i % p.D;
    float s = 0.0f;
    for (int k = 0; k < RPB; ++k) s += s_sum[which][k][dd];
    p.partial[(((size_t)blk * p.NH + h) * 2 + which) * p.D + dd] = s;
  }
}

// The partial sums of 64 (head, which, channel), added in the order of their
// workgroups: sixteen runs, one a wave, then the runs.  A run's loads go out
// four at a time: 5.6 us for 256 of them, 3.7 us for 167 (a lane that adds all
// of them one after another waits out a memory latency each: 25 and 13 us).
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void head_norm_sum_kernel(const HeadNormParams p) {
  constexpr int RUNS = kSumThreads / 64;
  __shared__ float s_run[RUNS][64];
  const int lane = threadIdx.x & 63, run = threadIdx.x >> 6;
  const size_t n = (size_t)p.NH * 2 * p.D;
  // the same trip count for every thread of a workgroup
  for (size_t i0 = (size_t)blockIdx.x * 64; i0 < n; i0 += (size_t)gridDim.x * 64) {
    const size_t i = i0 + lane;  // n is a multiple of 64
    float s = 0.0f;
    for (int k = run; k < p.blocks; k += 4 * RUNS) {
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = k + j * RUNS < p.blocks ? p.partial[(size_t)(k + j * RUNS) * n + i] : 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) s += x[j];
    }
    s_run[run][lane] = s;
    __syncthreads();
    if (run == 0) {
#pragma unroll
      for (int k = 1; k < RUNS; ++k) s += s_run[k][lane];
      const size_t h = i / (2 * p.D), which = i / p.D % 2, d = i % p.D;
      float* out = which ? p.dbias : p.dweight;
      if (out) out[h * p.D + d] = s;
    }
    __syncthreads();  // the runs are read out
  }
}

// Four rows a group where that leaves 2048 workgroups, eight a CU: 524288 rows
// of 512 values 197 us against 213 with one; 26655 rows of 192 (833 workgroups
// of four) 9.7 against 8.2, 64 rows of 512 5.2 against 3.2.
constexpr long long kManyGroups = 2048;
template <typename TX, typename TY, int LPR>
hipError_t launch_rows(const HeadNormParams& p, bool back, hipStream_t stream) {
  const long long rpb = kThreads / LPR;
  if (back) {
    hipLaunchKernelGGL((head_norm_back_kernel<TX, TY, LPR>), dim3((unsigned)((long long)p.blocks * p.NH)), dim3(kThreads),
                       0, stream, p);
  } else {
    const long long rows = (long long)p.B * p.NH * p.S;
    if (rows >= 4 * rpb * kManyGroups)
      hipLaunchKernelGGL((head_norm_kernel<TX, TY, LPR, 4>), dim3((unsigned)((rows + 4 * rpb - 1) / (4 * rpb))),
                         dim3(kThreads), 0, stream, p);
    else
      hipLaunchKernelGGL((head_norm_kernel<TX, TY, LPR, 1>), dim3((unsigned)((rows + rpb - 1) / rpb)), dim3(kThreads),
                         0, stream, p);
  }
  return hipGetLastError();
}

template <typename TX, typename TY>
hipError_t launch_types(const HeadNormParams& p, bool back, hipStream_t stream) {
  switch (head_norm_lanes(p.D)) {
    case 8: return launch_rows<TX, TY, 8>(p, back, stream);
    case 16: return launch_rows<TX, TY, 16>(p, back, stream);
    case 32: return launch_rows<TX, TY, 32>(p, back, stream);
    case 64: return launch_rows<TX, TY, 64>(p, back, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch(const HeadNormParams& p, bool back, hipStream_t stream) {
  if (p.x_bf16)
    return p.y_bf16 ? launch_types<bf16_t, bf16_t>(p, back, stream) : launch_types<bf16_t, float>(p, back, stream);
  return p.y_bf16 ? launch_types<float, bf16_t>(p, back, stream) : launch_types<float, float>(p, back, stream);
}

}  // namespace

int head_norm_lanes(int D) {
  int n = 8;
  while (n < D / 8) n *= 2;
  return n;
}

// Workgroups to fill the chip eight times over (twice as many: 351 us and 9.1
// for the partial sums against 356 and 5.7, at 64 heads of 8192 rows of 512),
// but four rows a group before that (15 heads of 1777 rows of 192: 13.4 us and
// 3.7 for the sums; sixteen rows a group 25.1 and 3.9, one row 13.4 and 4.8).
int head_norm_blocks(int B, int NH, int S, int D) {
  const long long rpb = kThreads / head_norm_lanes(D), rows = (long long)B * S;
  long long n = (rows + 4 * rpb - 1) / (4 * rpb);
  const long long most = NH < 2048 ? 2048 / NH : 1;
  if (n > most) n = most;
  return (int)(n < 1 ? 1 : n);
}

hipError_t launch_head_norm(const HeadNormParams& p, hipStream_t stream) { return launch(p, false, stream); }

hipError_t launch_head_norm_back(const HeadNormParams& p, hipStream_t stream) {
  hipError_t e = launch(p, true, stream);
  if (e != hipSuccess || !p.partial) return e;
  // 2^20 workgroups at most: a launch has to stay below 2^32 threads, which one
  // a 64 sums would reach at NH D = 2^27
  const size_t groups = (size_t)p.NH * 2 * p.D / 64, most = 1 << 20;
  hipLaunchKernelGGL(head_norm_sum_kernel, dim3((unsigned)(groups < most ? groups : most)), dim3(kSumThreads), 0, stream,
                     p);
  return hipGetLastError();
}

}  // namespace mlstm
