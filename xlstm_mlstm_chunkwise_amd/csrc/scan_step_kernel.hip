// Selective scan, one token, gfx950: the state is read and written once, in
// pieces of four states a lane, and C . h is added over the lanes of a channel.
// 8 sequences of 4096 channels of 16 states: 3.8 us, a launch's latency (4.7 MB:
// 1 us).
#include "scan_common.h"

namespace mlstm {
namespace {

constexpr int kThreads = 256;

template <typename T, int N>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(const ScanParams p) {
  constexpr int L = N / 4;  // lanes a channel
  const int64_t n = (int64_t)p.B * p.D * L;
  // whole waves: the lanes of a channel stay together
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    const int64_t bd = i / L;
    const int n0 = 4 * (int)(i - bd * L), b = (int)(bd / p.D), d = (int)(bd - (int64_t)b * p.D);
    auto at = [&](const View& v, int col) { return scan_load(static_cast<const T*>(v.p) + (size_t)b * v.batch + col); };
    float4 h = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (p.h0) h = *reinterpret_cast<const float4*>(p.h0 + bd * N + n0);
    const float4 A = *reinterpret_cast<const float4*>(p.A + (size_t)d * N + n0);
    const float x = at(p.x, d), dl = softplus(at(p.dt, d) + (p.bias ? p.bias[d] : 0.0f)), u = dl * x;
    h.x = fmaf(decay(dl, kLog2e * A.x), h.x, u * at(p.Bm, n0));
    h.y = fmaf(decay(dl, kLog2e * A.y), h.y, u * at(p.Bm, n0 + 1));
    h.z = fmaf(decay(dl, kLog2e * A.z), h.z, u * at(p.Bm, n0 + 2));
    h.w = fmaf(decay(dl, kLog2e * A.w), h.w, u * at(p.Bm, n0 + 3));
    *reinterpret_cast<float4*>(p.h_out + bd * N + n0) = h;
    float y = at(p.Cm, n0) * h.x + at(p.Cm, n0 + 1) * h.y + at(p.Cm, n0 + 2) * h.z + at(p.Cm, n0 + 3) * h.w;
#pragma unroll
    for (int o = 1; o < L; o *= 2) y += __shfl_xor(y, o, 64);
    if (n0 == 0) {
      if (p.Dskip) y = fmaf(p.Dskip[d], x, y);
      if (p.z.p) {
        const float z = at(p.z, d);
        y *= z * scan_sigmoid(z);
      }
      scan_store(static_cast<T*>(p.y) + bd, y);
    }
  }
}

template <typename T, int N>
hipError_t launch(const ScanParams& p, hipStream_t stream) {
  const int64_t n = ((int64_t)p.B * p.D * (N / 4) + kThreads - 1) / kThreads;
  hipLaunchKernelGGL((scan_step_kernel<T, N>), dim3((unsigned)(n < (1 << 20) ? n : 1 << 20)), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_states(const ScanParams& p, hipStream_t stream) {
  switch (p.N) {
    case 16: return launch<T, 16>(p, stream);
    case 32: return launch<T, 32>(p, stream);
    case 64: return launch<T, 64>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_scan_step(const ScanParams& p, hipStream_t stream) {
  return p.bf16 ? launch_states<bf16_t>(p, stream) : launch_states<float>(p, stream);
}

}  // namespace mlstm
