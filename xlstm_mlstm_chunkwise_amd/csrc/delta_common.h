// Device helpers of the gated delta rule's kernels: operands carried in
// several bf16 parts, and the 16 x 16 x 32 products over them.
//
// A float32 value is cut into three bf16 parts of eight significant bits
// each (hi + mid + lo, exact unless a part falls below the smallest normal).
// A product of an n-part and an m-part operand runs the part pairs (i, j)
// with i + j < max(n, m): a bf16 input (one part) times a three-part operand
// takes three matrix instructions and loses nothing but the float32
// accumulation; three parts times three take six and drop mid x lo twice.  The
// parts are truncated, so mid is below 2^-7 and lo below 2^-15 of the leading
// power of two: the two dropped terms are below 2^-21 of the product, always of
// its sign, and about 2^-23 on average.
// The state is carried from chunk to chunk in float32 and every chunk
// multiplies it, so two-part operands (2^-17 a rounding) would show in the
// float32 outputs (final state, gate gradients: 4e-6 to 9e-6 of their norm
// instead of below 1e-6); only results that are stored as bf16 (H, dK) use two.
#pragma once

#include "device_common.h"
#include "kernels.h"

namespace mlstm {

typedef uint32_t words2_t __attribute__((ext_vector_type(2)));
typedef uint32_t words4_t __attribute__((ext_vector_type(4)));

template <int N>
struct Parts {
  bf16x8_t p[N];
};

// Eight floats as N parts.  N = 3: each part is the leading sixteen bits of
// what the parts before it left (truncation; the remainders are exact).
// N = 2: nearest-even roundings.
template <int N>
__device__ __forceinline__ Parts<N> split_parts(const float (&x)[8]) {
  Parts<N> f;
  if constexpr (N == 1) {
    f.p[0] = Ops<bf16_t>::round(x);
  } else if constexpr (N == 2) {
    Ops<bf16_t>::split(x, f.p[0], f.p[1]);
  } else {
    uint32_t w[3][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a = x[2 * e], b = x[2 * e + 1];
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
        w[n][e] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
        if (n < 2) {
          a -= __uint_as_float(ua & 0xffff0000u);
          b -= __uint_as_float(ub & 0xffff0000u);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < 3; ++n) f.p[n] = as_bf16x8(make_uint4(w[n][0], w[n][1], w[n][2], w[n][3]));
  }
  return f;
}

// Four floats as N parts, two words each.  (Words as native vectors: arrays of
// HIP's uint2 end up in memory.)
template <int N>
__device__ __forceinline__ void split4(const float4_t& x, words2_t (&w)[N]) {
  if constexpr (N == 3) {
    float a[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = __float_as_uint(a[e]);
      w[n] = (words2_t){__builtin_amdgcn_perm(u[1], u[0], 0x07060302u), __builtin_amdgcn_perm(u[3], u[2], 0x07060302u)};
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] -= __uint_as_float(u[e] & 0xffff0000u);
    }
  } else {
    static_assert(N == 2, "two or three parts");
    uint32_t h0, l0, h1, l1;
    split_bf16x2(x[0], x[1], h0, l0);
    split_bf16x2(x[2], x[3], h1, l1);
    w[0] = (words2_t){h0, h1};
    w[1] = (words2_t){l0, l1};
  }
}

// The same eight values' parts from two split halves.
__device__ __forceinline__ Parts<3> join_halves(const words2_t (&a)[3], const words2_t (&b)[3]) {
  Parts<3> f;
#pragma unroll
  for (int n = 0; n < 3; ++n)
    f.p[n] = __builtin_bit_cast(bf16x8_t, (words4_t){a[n][0], a[n][1], b[n][0], b[n][1]});
  return f;
}

template <int N, int M>
__device__ __forceinline__ Parts<N> first_parts(const Parts<M>& x) {
  Parts<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) f.p[n] = x.p[n];
  return f;
}

__device__ __forceinline__ Parts<3> widen_parts(const Parts<2>& x) {
  Parts<3> f;
  f.p[0] = x.p[0];
  f.p[1] = f.p[2] = x.p[1];  // the third is not read
  return f;
}

// Two accumulator tiles (rows 0..15 and 16..31 of a 32-row block, one
// column per lane) as the eight values of one operand.
__device__ __forceinline__ void tiles8(const float4_t& a, const float4_t& b, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = a[e];
    x[e + 4] = b[e];
  }
}

template <int NA, int NB>
__device__ __forceinline__ float4_t mma_parts(const Parts<NA>& a, const Parts<NB>& b, float4_t c) {
  constexpr int M = NA > NB ? NA : NB;
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < M) c = mma16b(a.p[i], b.p[j], c);
  return c;
}

// The same for N accumulators, part pair by part pair, so that a product does
// not wait for the one before it on its own accumulator.
template <int N, int NA, int NB, typename B>
__device__ __forceinline__ void mma_parts_n(const Parts<NA> (&a)[N], B b, float4_t* const (&c)[N]) {
  constexpr int M = NA > NB ? NA : NB;
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < M)
#pragma unroll
        for (int n = 0; n < N; ++n) *c[n] = mma16b(a[n].p[i], b(n).p[j], *c[n]);
}

template <int NA, int NB>
constexpr int mma_count() {
  int n = 0;
  for (int i = 0; i < NA; ++i)
    for (int j = 0; j < NB; ++j) n += i + j < (NA > NB ? NA : NB);
  return n;
}

// Operand parts out of LDS planes (plane stride in elements).
// Row operand whose slots are 8 * (l / 16) + e: one 16-byte read a plane.
template <int N>
__device__ __forceinline__ Parts<N> lds_row8(const uint16_t* p, int plane) {
  Parts<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) f.p[n] = as_bf16x8(*reinterpret_cast<const uint4*>(p + n * plane));
  return f;
}
__device__ __forceinline__ uint2 lds_tr4(const uint16_t* p) {
  return __builtin_bit_cast(
      uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4_t*)(p)));
}
// Column operand: lane l gets column c0 + l % 16 of a row-major tile X, rows
// r0 + {0..3} (slots 0..3) and r0 + d + {0..3} (slots 4..7), r0 counted from
// the lane group's own base.
template <int N>
__device__ __forceinline__ Parts<N> lds_col(const uint16_t* X, int ld, int plane, int r0, int d, int c0, int lane) {
  const int j = lane & 15;
  const uint16_t* p = X + (r0 + (j >> 2)) * ld + c0 + 4 * (j & 3);
  Parts<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint2 a = lds_tr4(p + n * plane), b = lds_tr4(p + n * plane + d * ld);
    f.p[n] = as_bf16x8(make_uint4(a.x, a.y, b.x, b.y));
  }
  return f;
}

// Storage of Q, K, V by input type: parts and tokens per chunk.  A float32
// input is itself carried in three parts, so its chunk has half the rows for
// the same LDS.
template <typename TIn>
struct DeltaIn;
template <>
struct DeltaIn<bf16_t> {
  static constexpr int kParts = 1, kChunk = kDeltaChunkBf16;
};
template <>
struct DeltaIn<float> {
  static constexpr int kParts = 3, kChunk = kDeltaChunkF32;
};

__device__ __forceinline__ void store4(bf16_t* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = make_uint2(round_bf16x2(a, b), round_bf16x2(c, d));
}
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}

// Eight consecutive inputs as operand parts (global memory, 16-byte aligned).
__device__ __forceinline__ Parts<1> load_parts(const bf16_t* p) {
  Parts<1> f;
  f.p[0] = as_bf16x8(*reinterpret_cast<const uint4*>(p));
  return f;
}
__device__ __forceinline__ Parts<3> load_parts(const float* p) {
  float x[8];
  Ops<float>::load8(p, x);
  return split_parts<3>(x);
}
template <int N>
__device__ __forceinline__ Parts<N> zero_parts() {
  Parts<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) f.p[n] = as_bf16x8(make_uint4(0u, 0u, 0u, 0u));
  return f;
}
template <int N>
__device__ __forceinline__ void store_parts(uint16_t* p, int plane, const Parts<N>& f) {
#pragma unroll
  for (int n = 0; n < N; ++n) *reinterpret_cast<uint4*>(p + n * plane) = __builtin_bit_cast(uint4, f.p[n]);
}

// Rows [t0, t0 + ROWS) of a row-major input of S rows and W columns into LDS
// planes, zeros behind the last row.
template <typename TIn, int ROWS, int W>
__device__ __forceinline__ void stage_rows(uint16_t* dst, int ld, int plane, const TIn* src, int t0, int S, int tid,
                                           int threads) {
  constexpr int NP = DeltaIn<TIn>::kParts;
  for (int i = tid; i < ROWS * (W / 8); i += threads) {
    const int r = i / (W / 8), c = 8 * (i % (W / 8));
    const Parts<NP> f = t0 + r < S ? load_parts(src + (size_t)(t0 + r) * W + c) : zero_parts<NP>();
    store_parts<NP>(dst + r * ld + c, plane, f);
  }
}

// ---------------------------------------------------------------------------
// K and Q tiles of the walks: rows of DK values without padding, the 16-byte
// pieces of a row permuted by its number (piece p of row r sits at p ^
// swizzle(r)).  Two reads have to be free of bank conflicts: a piece's half
// from sixteen rows at once (the row operand), and 32 consecutive bytes from
// eight rows at once (the transposing read).  Rotating the row number's bits
// by one gives sixteen different slots to the first and different pairs of
// slots to the second.  (A row of 64 values spans half the banks and a row of
// 32 a quarter, so there two or four rows share a swizzle.)
template <int DK>
__device__ __forceinline__ int tile_swizzle(int r) {
  if constexpr (DK == 32) {
    const int x = (r >> 2) & 3;
    return ((x << 1) | (x >> 1)) & 3;
  } else if constexpr (DK == 64) {
    const int x = (r >> 1) & 7;
    return ((x << 1) | (x >> 2)) & 7;
  } else {
    const int x = r & 15;
    return ((x << 1) | (x >> 3)) & 15;
  }
}
template <int DK>
__device__ __forceinline__ int tile_at(int r, int piece) {
  return r * DK + 8 * (piece ^ tile_swizzle<DK>(r));
}

// Byte offsets of the two reads.  Everything that varies within a chunk is an
// exclusive or with a constant or a constant distance, so one seed a lane
// serves all of them.
//
// Keeps what follows from x inside the loop where it is used: the compiler
// would compute all offsets ahead of the chunk loop and hold them in registers.
__device__ __forceinline__ void keep_in_loop(int& x) { asm volatile("" : "+v"(x)); }

// Row operand: rows 16 rt + l % 16, contraction block 32 ks, in the slot order
// of two accumulator tiles.
template <int DK>
__device__ __forceinline__ int tile_row_seed(int row, int grp) {
  return 2 * tile_at<DK>(row, grp >> 1) + 8 * (grp & 1);
}
template <int N, int DK>
__device__ __forceinline__ Parts<N> tile_row(const uint16_t* X, int plane, int seed, int rt, int ks) {
  const char* a = reinterpret_cast<const char*>(X) + (seed ^ (64 * ks)) + 32 * rt * DK;
  const char* b = reinterpret_cast<const char*>(X) + (seed ^ (64 * ks + 32)) + 32 * rt * DK;
  Parts<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    // volatile: merged with another row tile's read, the halves would land
    // apart and cost a move each
    const words2_t x = *(const volatile __attribute__((address_space(3))) words2_t*)(a + 2 * n * plane);
    const words2_t y = *(const volatile __attribute__((address_space(3))) words2_t*)(b + 2 * n * plane);
    f.p[n] = as_bf16x8(make_uint4(x.x, x.y, y.x, y.y));
  }
  return f;
}
// Column operand: column 16 kt + l % 16, rows 32 ts + 4 grp + {0..3} and the
// same sixteen rows on.
template <int DK>
__device__ __forceinline__ int tile_col_seed(int grp, int lane) {
  const int j = lane & 15;
  return 2 * tile_at<DK>(4 * grp + (j >> 2), (j & 3) >> 1) + 8 * (j & 1);
}
template <int N, int DK>
__device__ __forceinline__ Parts<N> tile_col(const uint16_t* X, int plane, int seed, int ts, int kt) {
  const uint16_t* a = X + ((seed ^ (32 * kt)) >> 1) + 32 * ts * DK;
  Parts<N> f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint2 x = lds_tr4(a + n * plane), y = lds_tr4(a + n * plane + 16 * DK);
    f.p[n] = as_bf16x8(make_uint4(x.x, x.y, y.x, y.y));
  }
  return f;
}

// Order of one step of a pipelined phase: RD LDS reads for the next step, then
// MM matrix instructions of this one with up to VV vector instructions
// (conversions for the next) in the shadow of each.  (Left alone, the compiler
// puts every read right before its products and waits for it, and does the
// conversions in one run while the matrix cores idle.)
template <int RD, int MM, int VV>
__device__ __forceinline__ void end_step() {
  if constexpr (RD > 0) __builtin_amdgcn_sched_group_barrier(0x100, RD, 0);
#pragma unroll
  for (int i = 0; i < MM; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, VV, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

// A tile on its way from memory to LDS: the loads go out a chunk ahead and
// wait in registers for the barrier that frees the tile.
template <typename TIn, int DK, int THREADS>
struct TileStage {
  static constexpr int L = DeltaIn<TIn>::kChunk, NP = DeltaIn<TIn>::kParts;
  static constexpr int kPieces = L * (DK / 8), kN = (kPieces + THREADS - 1) / THREADS;
  static constexpr int kWords = sizeof(TIn) == 2 ? 1 : 2;  // 16-byte words a piece
  words4_t x[kN][kWords];

  // The tile's rows lie one behind the other: rows [0, rows) from src, zeros
  // behind them (range check of the buffer resource).
  __device__ __forceinline__ void load(const TIn* src, int rows, int tid) {
    const int bytes = __builtin_amdgcn_readfirstlane(rows * DK * (int)sizeof(TIn));
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int off = n * THREADS * 16 * kWords;
      const __amdgpu_buffer_rsrc_t r = make_rsrc(
          reinterpret_cast<const char*>(src) + off, (uint32_t)__builtin_amdgcn_readfirstlane(bytes > off ? bytes - off : 0));
#pragma unroll
      for (int w = 0; w < kWords; ++w)
        x[n][w] = __builtin_bit_cast(words4_t, __builtin_amdgcn_raw_buffer_load_b128(r, 16 * kWords * tid + 16 * w, 0, 0));
    }
  }
  __device__ __forceinline__ void store(uint16_t* dst, int plane, int tid) const {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int i = tid + n * THREADS, r = i / (DK / 8), p = i % (DK / 8);
      if (kPieces % THREADS != 0 && i >= kPieces) continue;
      uint16_t* o = dst + tile_at<DK>(r, p);
      if constexpr (sizeof(TIn) == 2) {
        *reinterpret_cast<words4_t*>(o) = x[n][0];
      } else {
        const float4 a = __builtin_bit_cast(float4, x[n][0]), b = __builtin_bit_cast(float4, x[n][kWords - 1]);
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        store_parts<NP>(o, plane, split_parts<NP>(v));
      }
    }
  }
};

// The same for W of the DK columns, in a tile of that width.
template <typename TIn, int DK, int W, int THREADS>
struct PartStage {
  static constexpr int L = DeltaIn<TIn>::kChunk, NP = DeltaIn<TIn>::kParts;
  static constexpr int kRow = W / 8, kN = L * kRow / THREADS, kWords = sizeof(TIn) == 2 ? 1 : 2;
  words4_t x[kN * kWords];

  static_assert(kN * THREADS == L * kRow, "whole rounds");
  // src: the chunk's first row at the first column, which is column `col`
  __device__ __forceinline__ void load(const TIn* src, int col, int rows, int tid) {
    const __amdgpu_buffer_rsrc_t r = make_rsrc(src, (uint32_t)__builtin_amdgcn_readfirstlane((rows * DK - col) * (int)sizeof(TIn)));
    int off = (tid / kRow * DK + 8 * (tid % kRow)) * (int)sizeof(TIn);
#pragma unroll
    for (int n = 0; n < kN; ++n) {
#pragma unroll
      for (int w = 0; w < kWords; ++w)
        x[n * kWords + w] = __builtin_bit_cast(words4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off + 16 * w, 0, 0));
      off += THREADS / kRow * DK * (int)sizeof(TIn);
    }
  }
  __device__ __forceinline__ void store(uint16_t* dst, int plane, int tid) const {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      uint16_t* o = dst + tile_at<W>(tid / kRow + n * (THREADS / kRow), tid % kRow);
      if constexpr (sizeof(TIn) == 2) {
        *reinterpret_cast<words4_t*>(o) = x[n];
      } else {
        const float4 a = __builtin_bit_cast(float4, x[n * kWords]), b = __builtin_bit_cast(float4, x[n * kWords + kWords - 1]);
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        store_parts<NP>(o, plane, split_parts<NP>(v));
      }
    }
  }
};

// ---------------------------------------------------------------------------
// T and P of a chunk in operand order.  A lower triangular L x L matrix M is
// the left operand of a product over its columns as fragments (row tile rt,
// 32-column block ts <= rt / 2); M^T as fragments (rt, ts >= rt / 2).  A
// fragment is three planes of 64 lanes x 8 bf16: lane l has row 16 rt + l % 16
// of the operand and the slots 32 ts + 4 (l / 16) + {0..3} and sixteen on.
template <int L>
constexpr int square_frags() {
  return L == 64 ? 6 : 2;
}
constexpr int kFragElems = 512;  // one plane of one fragment

template <int L>
__device__ __forceinline__ constexpr int frag_rt(bool up, int f) {
  return L != 64 ? f : up ? (f < 4 ? f / 2 : f - 2) : (f < 2 ? f : 1 + f / 2);
}
template <int L>
__device__ __forceinline__ constexpr int frag_ts(bool up, int f) {
  return L != 64 ? 0 : up ? (f < 4 ? f % 2 : 1) : (f < 2 ? 0 : f % 2);
}

// Fragments in pairs of different row tiles.
template <int L>
__device__ __forceinline__ constexpr int frag_order(bool up, int i) {
  // M: (0,0) (1,0) | (2,0) (3,0) | (2,1) (3,1);  M^T: (0,0) (1,0) | (0,1) (1,1) | (2,1) (3,1)
  return L != 64 ? i : i == 0 || i == 5 ? i : up ? (i == 1 ? 2 : i == 2 ? 1 : i) : (i == 3 ? 4 : i == 4 ? 3 : i);
}

struct NoSideWork {
  __device__ __forceinline__ void operator()(int) const {}
};

// acc[rt] += M . X (UP: M^T . X), with the NM-plane fragments of M (M^T) in
// LDS and X in 32-row blocks.  side(i) is the caller's work for step i of
// square_frags<L>(): VV of its vector instructions go into each matrix
// instruction's shadow.
template <int L, bool UP, int NM, int NX, int VV, typename Side = NoSideWork>
__device__ __forceinline__ void square_times(const uint16_t* M, const Parts<NX> (&x)[L / 32], float4_t (&acc)[L / 16],
                                             int lane, Side side = Side()) {
  constexpr int NF = square_frags<L>();
  Parts<NM> f[2], next[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    f[h] = lds_row8<NM>(M + frag_order<L>(UP, h) * NM * kFragElems + 8 * lane, kFragElems);
#pragma unroll
  for (int i = 0; i < NF; i += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      next[h] = f[h];
      if (i + 2 < NF) next[h] = lds_row8<NM>(M + frag_order<L>(UP, i + 2 + h) * NM * kFragElems + 8 * lane, kFragElems);
    }
    side(i);
    side(i + 1);
    const int f0 = frag_order<L>(UP, i), f1 = frag_order<L>(UP, i + 1);
    float4_t* const c[2] = {&acc[frag_rt<L>(UP, f0)], &acc[frag_rt<L>(UP, f1)]};
    mma_parts_n<2, NM, NX>(f, [&](int n) -> const Parts<NX>& { return x[frag_ts<L>(UP, n ? f1 : f0)]; }, c);
    if (i + 2 < NF) end_step<2 * NM, 2 * mma_count<NM, NX>(), VV>();
    else end_step<0, 2 * mma_count<NM, NX>(), VV>();
#pragma unroll
    for (int h = 0; h < 2; ++h) f[h] = next[h];
  }
}

// acc[kt] += X^T[rows 16 kt ..] . y over the 32 rows of block ts, X a K or Q
// tile in LDS; side(i) for step i of DK / 32.
template <int NP, int DK, int VV, typename Side = NoSideWork>
__device__ __forceinline__ void tile_cols_times(const uint16_t* X, int plane, int seed, int ts, const Parts<3>& y,
                                                float4_t (&acc)[DK / 16], Side side = Side()) {
  constexpr int KT = DK / 16;
  Parts<NP> f[2], next[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) f[h] = tile_col<NP, DK>(X, plane, seed, ts, h);
#pragma unroll
  for (int k = 0; k < KT; k += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      next[h] = f[h];
      if (k + 2 < KT) next[h] = tile_col<NP, DK>(X, plane, seed, ts, k + 2 + h);
    }
    side(k / 2);
    float4_t* const c[2] = {&acc[k], &acc[k + 1]};
    mma_parts_n<2, NP, 3>(f, [&](int) -> const Parts<3>& { return y; }, c);
    if (k + 2 < KT) end_step<4 * NP, 2 * mma_count<NP, 3>(), VV>();
    else end_step<0, 2 * mma_count<NP, 3>(), VV>();
#pragma unroll
    for (int h = 0; h < 2; ++h) f[h] = next[h];
  }
}

// Fragments on their way from memory to LDS (NM planes of each).
template <int L, int NM, int THREADS>
struct SquareStage {
  static constexpr int kPieces = square_frags<L>() * NM * 64, kN = (kPieces + THREADS - 1) / THREADS;
  words4_t x[kN];
  __device__ __forceinline__ void load(const uint16_t* src, int tid) {
    // a last round with fewer pieces than threads reads zeros behind them
#pragma unroll
    for (int n = 0; n < kN; ++n)
      x[n] = __builtin_bit_cast(words4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                              make_rsrc_at(src, 16 * kPieces, n * THREADS * 16), 16 * tid, 0, 0));
  }
  __device__ __forceinline__ void store(uint16_t* dst, int tid) const {
#pragma unroll
    for (int n = 0; n < kN; ++n)
      if ((n + 1) * THREADS <= kPieces || tid + n * THREADS < kPieces)
        *reinterpret_cast<words4_t*>(dst + 8 * (tid + n * THREADS)) = x[n];
  }
};

}  // namespace mlstm
