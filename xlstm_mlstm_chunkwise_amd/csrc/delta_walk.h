// Pieces shared by the two forms of the gated delta rule's walks
// (delta_walk_kernel.hip, delta_split_kernel.hip).
#pragma once

#include "delta_common.h"
#include "kernels.h"
#include "pair_store.h"

namespace mlstm {

// Four values s_x[16 rt + 4 grp ..] of a row vector in LDS.
__device__ __forceinline__ float4_t row4(const float* x, int rt, int grp) {
  return *reinterpret_cast<const float4_t*>(x + 16 * rt + 4 * grp);
}

// A slice of rows of a row-major matrix of `ld` columns, one lane a column:
// a buffer resource over `rows` rows from `base` (reads behind them give
// zero, stores are dropped) and this lane's offset, element (row 4 grp, its
// column).
template <typename T>
struct Slice {
  __amdgpu_buffer_rsrc_t rsrc;
  int lane_off, row_bytes;
  __device__ __forceinline__ Slice(const T* base, int ld, int rows, int off)
      : rsrc(make_rsrc(base, (uint32_t)rows * ld * (uint32_t)sizeof(T))), lane_off(off * (int)sizeof(T)),
        row_bytes(ld * (int)sizeof(T)) {}
};

// The values as they are in memory; they become floats where they are used,
// so that nothing waits for the loads before.
template <typename T, int N>
struct RawTiles {
  uint32_t x[N][4];
  __device__ __forceinline__ void load(const Slice<T>& s) {
#pragma unroll
    for (int rt = 0; rt < N; ++rt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int off = s.lane_off + (16 * rt + r) * s.row_bytes;
        if constexpr (sizeof(T) == 2) x[rt][r] = __builtin_amdgcn_raw_buffer_load_b16(s.rsrc, off, 0, 0);
        else x[rt][r] = __builtin_amdgcn_raw_buffer_load_b32(s.rsrc, off, 0, 0);
      }
  }
  __device__ __forceinline__ float4_t tile(int rt) const {
    float4_t v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = __uint_as_float(sizeof(T) == 2 ? x[rt][r] << 16 : x[rt][r]);
    return v;
  }
};

// Every row is in range: the row offset may be a scalar, which the range
// check leaves out.
__device__ __forceinline__ void store_rows(const Slice<float>& s, int rt, const float4_t& x) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[r]), s.rsrc, s.lane_off, (16 * rt + r) * s.row_bytes, 0);
}
template <int N>
__device__ __forceinline__ void store_whole(const Slice<float>& s, const float4_t (&x)[N]) {
#pragma unroll
  for (int rt = 0; rt < N; ++rt) store_rows(s, rt, x[rt]);
}
template <int N>
__device__ __forceinline__ void load_whole(const Slice<float>& s, float4_t (&x)[N]) {
#pragma unroll
  for (int rt = 0; rt < N; ++rt)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      x[rt][r] = __int_as_float(
          (int)__builtin_amdgcn_raw_buffer_load_b32(s.rsrc, s.lane_off, (16 * rt + r) * s.row_bytes, 0));
}

// One accumulator tile in the type of H or V, adjacent lanes paired so that
// each stores two neighbouring values of a row at once.
template <typename T>
__device__ __forceinline__ void store_tile(const Slice<T>& s, int rt, const float4_t& x, float scale, int lane) {
  const bool odd = lane & 1;
  const int base = s.lane_off + (odd ? s.row_bytes - (int)sizeof(T) : 0);  // the pair's even column
#pragma unroll
  for (int r = 0; r < 4; r += 2) {
    const float2 v = pair_rows_to_cols(scale * x[r], scale * x[r + 1], odd);
    const int off = base + (16 * rt + r) * s.row_bytes;
    if constexpr (sizeof(T) == 2) {
      __builtin_amdgcn_raw_buffer_store_b32(round_bf16x2(v.x, v.y), s.rsrc, off, 0, 0);
    } else {
      const v2i32_t w = {__float_as_int(v.x), __float_as_int(v.y)};
      __builtin_amdgcn_raw_buffer_store_b64(w, s.rsrc, off, 0, 0);
    }
  }
}

// acc[rt] += a[rt] . b
template <int N, int NA, int NB>
__device__ __forceinline__ void rows_times(const Parts<NA> (&a)[N], const Parts<NB>& b, float4_t (&acc)[N]) {
  constexpr int M = NA > NB ? NA : NB;
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < M)
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] = mma16b(a[n].p[i], b.p[j], acc[n]);
}

// w x of one 32-row block as operand parts.
__device__ __forceinline__ Parts<3> scaled_parts(const float* w, const float4_t* x, int ts, int grp) {
  float y[8];
  tiles8(row4(w, 2 * ts, grp) * x[2 * ts], row4(w, 2 * ts + 1, grp) * x[2 * ts + 1], y);
  return split_parts<3>(y);
}

}  // namespace mlstm
