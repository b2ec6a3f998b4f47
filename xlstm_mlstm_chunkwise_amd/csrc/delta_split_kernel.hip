// Gated delta rule: the chunks of a head in order where there are few heads,
// gfx950.
//
// The walk of delta_walk_kernel.hip gives a wave sixteen value columns of one
// head; with few heads that leaves most of the chip idle and a chunk takes as
// long as one wave's products.  Here the waves of a workgroup share sixteen
// columns: wave i holds rows i DHQK / RW .. of the state (two waves at DHQK 64,
// four above) and owns row tile i of the chunk's sixteen-token tiles.  Per chunk
//   - each wave forms its rows' share of K C and Q C (L x 16); the shares meet
//     in LDS;
//   - the owner forms its tile of V - e K C, which all owners read as operand,
//     its tile of U = T (..), which all waves read, and its tile of H;
//   - each wave updates its own rows, C <- g C + K^T (w U).
// Three barriers a chunk.  A wave reads only its own columns of K and Q (staged
// in LDS that no other wave touches, for the transposing reads) and only its
// own row tiles of T and P (operand order, straight from memory), all a chunk
// ahead in registers.  The loads go out in three lots between the phases: a
// chunk is 94 KB, which a CU takes in no faster than 64 bytes a cycle, and a
// wave that issues all its loads at once computes nothing meanwhile.
//
// A chunk's chain of dependent steps bounds it, not memory (with all loads
// answered by the caches it is no faster): 8 heads of 256 x 512 at 65536
// tokens, 1024 chunks one after another, take 3.1 ms, 3.0 us a chunk, of which
// the matrix cores are busy a fifth; the column walk takes 6.8 ms there.  64
// heads of 128 x 128 at 2048 tokens: 121 us forward, 122 with the states, 195
// backward.  Two row tiles a wave instead of one cost 80 us against 68 for 15
// heads of 64 x 192 at 1777 tokens.
#include "delta_walk.h"

namespace mlstm {
namespace {

template <typename TIn, int DK>
struct SplitShape {
  static constexpr int L = DeltaIn<TIn>::kChunk, NP = DeltaIn<TIn>::kParts;
  static constexpr int RT = L / 16, TS = L / 32;
  static constexpr int RW = DK == 64 ? 2 : 4;           // waves that hold rows of the state
  static constexpr int W = DK / RW;                     // rows each
  static constexpr int NW = RT > RW ? RT : RW;          // waves: wave i owns row tile i
  static constexpr int kSlots = RT > RW ? RW : RW - 1;  // shares an owner receives, at most
  static constexpr int kPlane = L * W, kTile = NP * kPlane;
  static constexpr int kFragWords = kFragElems / 2;     // one operand fragment plane, in 32-bit words
};

// One owner's tile of an operand (four values a lane) into the fragment of
// its 32-row block, N parts.
template <int N>
__device__ __forceinline__ void put_operand(uint16_t* frags, int rt, const float4_t& x, int lane) {
  words2_t w[N];
  split4<N>(x, w);
#pragma unroll
  for (int n = 0; n < N; ++n)
    *reinterpret_cast<words2_t*>(frags + ((rt >> 1) * N + n) * kFragElems + 8 * lane + 4 * (rt & 1)) = w[n];
}

// acc += row tile rt of M (UP: of M^T) . X, fragments of M in registers and of
// X in LDS.  One tile is one accumulator, so its products go in chains of
// their own by part class and 32-row block; a single chain would wait out the
// latency of every product.
template <int L, bool UP, int NM, int NX>
__device__ __forceinline__ void tile_times(const Parts<NM> (&m)[L / 32], const uint16_t* x, int rt, float4_t& acc,
                                           int lane) {
  constexpr int TS = L / 32, CLASSES = NM > NX ? NM : NX;
  float4_t sum[TS][CLASSES];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts)
#pragma unroll
    for (int k = 0; k < CLASSES; ++k) sum[ts][k] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  Parts<NX> f[TS];
#pragma unroll
  for (int ts = 0; ts < TS; ++ts) f[ts] = lds_row8<NX>(x + ts * NX * kFragElems + 8 * lane, kFragElems);
  // a block on the other side of the diagonal has zero fragments
#pragma unroll
  for (int i = 0; i < NM; ++i)
#pragma unroll
    for (int j = 0; j < NX; ++j)
      if (i + j < CLASSES)
#pragma unroll
        for (int ts = 0; ts < TS; ++ts) sum[ts][i + j] = mma16b(m[ts].p[i], f[ts].p[j], sum[ts][i + j]);
#pragma unroll
  for (int k = CLASSES - 1; k >= 0; --k)
#pragma unroll
    for (int ts = 0; ts < TS; ++ts) acc += sum[ts][k];
}

// The fragments of row tile rt, from memory (zeros where the triangle has none:
// the resource is empty).
template <int L, bool UP, int NM>
__device__ __forceinline__ void load_square_rows(const uint16_t* M, int rt, Parts<NM> (&m)[L / 32], int lane) {
#pragma unroll
  for (int ts = 0; ts < L / 32; ++ts) {
    const bool in = rt < L / 16 && (UP ? ts >= (rt >> 1) : ts <= (rt >> 1));
    const int f = L != 64 ? rt : UP ? (rt < 2 ? 2 * rt + ts : rt + 2) : (rt < 2 ? rt : 2 * rt - 2 + ts);
    const __amdgpu_buffer_rsrc_t r =
        make_rsrc(M + (in ? f * NM * kFragElems : 0), (uint32_t)__builtin_amdgcn_readfirstlane(in ? NM * kFragElems * 2 : 0));
#pragma unroll
    for (int n = 0; n < NM; ++n)
      m[ts].p[n] = __builtin_bit_cast(bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(r, 16 * lane + 2 * n * kFragElems, 0, 0));
  }
}

// acc[rt] += rows of X against this wave's part of a state (KT tiles).
template <int NP, int W, int PP, int RT>
__device__ __forceinline__ void part_rows_times(const uint16_t* X, int plane, int seed, const Parts<3> (&c)[W / 32],
                                                float4_t (&acc)[RT]) {
  Parts<NP> f[RT];
#pragma unroll
  for (int ks = 0; ks < W / 32; ++ks) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) f[rt] = tile_row<NP, W>(X, plane, seed, rt, ks);
    rows_times(f, first_parts<PP>(c[ks]), acc);
  }
}

template <int W>
__device__ __forceinline__ void state_parts(const float4_t (&C)[W / 16], Parts<3> (&c)[W / 32]) {
#pragma unroll
  for (int ks = 0; ks < W / 32; ++ks) {
    float x[8];
    tiles8(C[2 * ks], C[2 * ks + 1], x);
    c[ks] = split_parts<3>(x);
  }
}

// The shares of the waves, one 1 KiB slot per row tile and sending wave; an
// owner with rows of its own adds that share from registers.
template <typename S>
__device__ __forceinline__ void send_shares(float4_t* slots, const float4_t (&x)[S::RT], int wave, int lane) {
#pragma unroll
  for (int rt = 0; rt < S::RT; ++rt)
    if (rt != wave) slots[(rt * S::kSlots + (rt >= S::RW || wave < rt ? wave : wave - 1)) * 64 + lane] = x[rt];
}
template <typename S>
__device__ __forceinline__ float4_t take_shares(const float4_t* slots, const float4_t (&x)[S::RT], int rt, int lane) {
  float4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < S::RT; ++i) {
    float4_t own = x[i];
    asm("" : "+v"(own));  // a value each: as an indexed array the tiles would leave the registers
    if (rt == i && rt < S::RW) v = own;
  }
#pragma unroll
  for (int i = 0; i < S::kSlots; ++i)
    if (i < S::RW - 1 || rt >= S::RW) v += slots[(rt * S::kSlots + i) * 64 + lane];
  return v;
}

// One row tile of V, dH or U: four values a lane.  `rows` rows from `base`;
// each row has a resource of its own, so that a lane keeps one offset.
template <typename T>
struct OneTile {
  uint32_t x[4];
  __device__ __forceinline__ void load(const T* base, int ld, int rows, int rt, int io_off) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int skip = 16 * rt + r, left = rows > skip ? rows - skip : 0;
      const __amdgpu_buffer_rsrc_t b =
          make_rsrc(base + (size_t)skip * ld, (uint32_t)__builtin_amdgcn_readfirstlane(left * ld * (int)sizeof(T)));
      if constexpr (sizeof(T) == 2) x[r] = __builtin_amdgcn_raw_buffer_load_b16(b, 2 * io_off, 0, 0);
      else x[r] = __builtin_amdgcn_raw_buffer_load_b32(b, 4 * io_off, 0, 0);
    }
  }
  __device__ __forceinline__ float4_t tile() const {
    float4_t v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = __uint_as_float(sizeof(T) == 2 ? x[r] << 16 : x[r]);
    return v;
  }
};

__device__ __forceinline__ void store_one(const Slice<float>& s, int rt, const float4_t& x) {
  int off = s.lane_off + 16 * rt * s.row_bytes;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[r]), s.rsrc, off, 0, 0);
    off += s.row_bytes;
  }
}

// FWD and TH as in delta_walk_kernel.
template <typename TIn, typename TH, int DK, bool FWD>
__global__ __launch_bounds__((64 * SplitShape<TIn, DK>::NW)) void delta_split_kernel(const DeltaParams p) {
  typedef SplitShape<TIn, DK> S;
  constexpr int L = S::L, NP = S::NP, W = S::W, RT = S::RT, TS = S::TS, KT = W / 16;
  constexpr int PP = sizeof(TH) == 2 ? 2 : 3;
  __shared__ uint4 s_tiles[S::RW * (FWD ? 2 : 1) * S::kTile * 2 / 16];
  __shared__ float4_t s_kc[RT * S::kSlots * 64], s_qc[FWD ? RT * S::kSlots * 64 : 1];
  __shared__ uint4 s_x[TS * 3 * 64], s_wu[TS * 3 * 64], s_u[FWD ? TS * PP * 64 : 1];
  uint16_t* x_frags = reinterpret_cast<uint16_t*>(s_x);
  uint16_t* wu_frags = reinterpret_cast<uint16_t*>(s_wu);
  uint16_t* u_frags = reinterpret_cast<uint16_t*>(s_u);

  const int bh = blockIdx.x % p.BH, slice = blockIdx.x / p.BH;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, grp = lane >> 4;
  const int col = 16 * slice + row;
  // row tile `wave` is this wave's; the first RW waves hold rows of the state
  const int rt = wave;
  const bool owner = S::RT == S::NW || wave < S::RT, holds = S::RW == S::NW || wave < S::RW;
  uint16_t* s_K = reinterpret_cast<uint16_t*>(s_tiles) + (holds ? wave : 0) * (FWD ? 2 : 1) * S::kTile;
  uint16_t* s_Q = s_K + S::kTile;
  const TIn* K = static_cast<const TIn*>(p.K) + (size_t)bh * p.S * DK + wave * W;
  const TIn* Q = static_cast<const TIn*>(p.Q) + (size_t)bh * p.S * DK + wave * W;
  const TIn* V = static_cast<const TIn*>(p.V) + (size_t)bh * p.S * p.DV;
  constexpr int kSquare = square_frags<L>() * 3 * kFragElems;
  const int io_off = 4 * grp * p.DV + col;
  const int row_seed = tile_row_seed<W>(row, grp), col_seed = tile_col_seed<W>(grp, lane);

  float4_t C[KT];
#pragma unroll
  for (int k = 0; k < KT; ++k) C[k] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  if (p.C0 && holds) load_whole(Slice<float>(p.C0 + ((size_t)bh * DK + wave * W) * p.DV, p.DV, W, io_off), C);

  PartStage<TIn, DK, W, 64> gk, gq;
  Parts<3> gt[TS];
  Parts<PP> gp[TS];
  OneTile<TIn> gv;
  float4_t ge, gw;
  float gg = 0.0f;
  // The loads by where their registers are free again: K and Q once they are
  // in LDS, the rest behind V - e K C, U and H.
  auto rows_of = [&](int c) { return p.S - c * L < L ? p.S - c * L : L; };
  auto row4_of = [&](const float* x, int c) {
    return *reinterpret_cast<const float4_t*>(x + ((size_t)bh * p.Nc + c) * L + (owner ? 16 * rt + 4 * grp : 0));
  };
  auto fetch_k = [&](int c) {
    if (holds) gk.load(K + (size_t)c * L * DK, wave * W, rows_of(c), lane);
  };
  auto fetch_q = [&](int c) {
    if constexpr (FWD)
      if (holds) gq.load(Q + (size_t)c * L * DK, wave * W, rows_of(c), lane);
  };
  auto fetch_v = [&](int c) {
    gv.load(V + (size_t)c * L * p.DV, p.DV, rows_of(c), rt, io_off);
    ge = row4_of(p.e, c);
  };
  auto fetch_t = [&](int c) {
    load_square_rows<L, false, 3>(p.T + ((size_t)bh * p.Nc + c) * kSquare, rt, gt, lane);
    gw = row4_of(p.w, c);
    gg = p.e[((size_t)bh * p.Nc + c) * L + L - 1];
  };
  auto fetch_p = [&](int c) {
    if constexpr (FWD) load_square_rows<L, false, PP>(p.P + ((size_t)bh * p.Nc + c) * kSquare, rt, gp, lane);
  };
  if (p.Nc) {
    fetch_k(0);
    fetch_v(0);
    fetch_q(0);
    fetch_t(0);
    fetch_p(0);
  }

  for (int c = 0; c < p.Nc; ++c) {
    const int t0 = c * L;
    const size_t at = (size_t)bh * p.Nc + c;
    const int next = c + 1 < p.Nc ? c + 1 : c;
    float4_t kc[RT], qc[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) kc[j] = qc[j] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
    if (holds) {
      gk.store(s_K, S::kPlane, lane);
      if constexpr (FWD) gq.store(s_Q, S::kPlane, lane);
      __builtin_amdgcn_wave_barrier();
      if constexpr (!FWD) store_whole(Slice<float>(p.C_states + (at * DK + wave * W) * p.DV, p.DV, W, io_off), C);

      // this wave's share of K C and Q C
      Parts<3> cp[W / 32];
      state_parts<W>(C, cp);
      part_rows_times<NP, W, 3>(s_K, S::kPlane, row_seed, cp, kc);
      send_shares<S>(s_kc, kc, wave, lane);
      if constexpr (FWD) {
        part_rows_times<NP, W, PP>(s_Q, S::kPlane, row_seed, cp, qc);
        send_shares<S>(s_qc, qc, wave, lane);
      }
#pragma unroll
      for (int k = 0; k < KT; ++k) C[k] *= gg;
    }
    fetch_k(next);
    __syncthreads();

    // the owners' tiles of V - e K C
    float4_t h = {0.0f, 0.0f, 0.0f, 0.0f};
    if (owner) {
      put_operand<3>(x_frags, rt, gv.tile() - ge * take_shares<S>(s_kc, kc, rt, lane), lane);
      if constexpr (FWD) h = ge * take_shares<S>(s_qc, qc, rt, lane);
    }
    fetch_v(next);
    fetch_q(next);
    __syncthreads();

    // ... and of U
    if (owner) {
      float4_t u = {0.0f, 0.0f, 0.0f, 0.0f};
      tile_times<L, false, 3, 3>(gt, x_frags, rt, u, lane);
      put_operand<3>(wu_frags, rt, gw * u, lane);
      if constexpr (FWD) put_operand<PP>(u_frags, rt, u, lane);
      else store_one(Slice<float>(p.U + at * L * p.DV, p.DV, L, io_off), rt, u);
    }
    fetch_t(next);
    __syncthreads();

    // C <- g C + K^T (w U), H = s (e Q C + P U)
    if (holds) {
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        const Parts<3> wu = lds_row8<3>(wu_frags + ts * 3 * kFragElems + 8 * lane, kFragElems);
#pragma unroll
        for (int k = 0; k < KT; ++k)
          C[k] = mma_parts<NP, 3>(tile_col<NP, W>(s_K, S::kPlane, col_seed, ts, k), wu, C[k]);
      }
    }
    if constexpr (FWD) {
      if (owner) {
        tile_times<L, false, PP, PP>(gp, u_frags, rt, h, lane);
        store_tile(Slice<TH>(static_cast<TH*>(p.H) + ((size_t)bh * p.S + t0) * p.DV, p.DV, rows_of(c), io_off), rt, h,
                   p.scale, lane);
      }
    }
    fetch_p(next);
  }

  if (p.C_out && holds) store_whole(Slice<float>(p.C_out + ((size_t)bh * DK + wave * W) * p.DV, p.DV, W, io_off), C);
}

// The backward walk in the same form; formulas and outputs as in
// delta_walk_back_kernel, whose anchor slots hold one sum per sixteen columns.
template <typename TIn, typename TH, int DK>
__global__ __launch_bounds__((64 * SplitShape<TIn, DK>::NW)) void delta_split_back_kernel(const DeltaParams p) {
  typedef SplitShape<TIn, DK> S;
  constexpr int L = S::L, NP = S::NP, W = S::W, RT = S::RT, TS = S::TS, KT = W / 16;
  __shared__ uint4 s_tiles[S::RW * 2 * S::kTile * 2 / 16];
  __shared__ float4_t s_kg[RT * S::kSlots * 64];
  __shared__ uint4 s_h[TS * 3 * 64], s_eh[TS * 3 * 64], s_du[TS * 3 * 64], s_dv[TS * 3 * 64];
  __shared__ float s_anchor[2][RT];
  uint16_t* h_frags = reinterpret_cast<uint16_t*>(s_h);
  uint16_t* eh_frags = reinterpret_cast<uint16_t*>(s_eh);
  uint16_t* du_frags = reinterpret_cast<uint16_t*>(s_du);
  uint16_t* dv_frags = reinterpret_cast<uint16_t*>(s_dv);

  const int bh = blockIdx.x % p.BH, slice = blockIdx.x / p.BH;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, grp = lane >> 4;
  const int col = 16 * slice + row;
  // row tile `wave` is this wave's; the first RW waves hold rows of the state
  const int rt = wave;
  const bool owner = S::RT == S::NW || wave < S::RT, holds = S::RW == S::NW || wave < S::RW;
  uint16_t* s_K = reinterpret_cast<uint16_t*>(s_tiles) + (holds ? wave : 0) * 2 * S::kTile;
  uint16_t* s_Q = s_K + S::kTile;
  const TIn* K = static_cast<const TIn*>(p.K) + (size_t)bh * p.S * DK + wave * W;
  const TIn* Q = static_cast<const TIn*>(p.Q) + (size_t)bh * p.S * DK + wave * W;
  const TH* dH = static_cast<const TH*>(p.dH) + (size_t)bh * p.S * p.DV;
  constexpr int kSquare = square_frags<L>() * 3 * kFragElems;
  const int io_off = 4 * grp * p.DV + col;
  const int row_seed = tile_row_seed<W>(row, grp), col_seed = tile_col_seed<W>(grp, lane);

  float4_t G[KT];
#pragma unroll
  for (int k = 0; k < KT; ++k) G[k] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  if (p.dC_out && holds) load_whole(Slice<float>(p.dC_out + ((size_t)bh * DK + wave * W) * p.DV, p.DV, W, io_off), G);

  PartStage<TIn, DK, W, 64> gk, gq;
  Parts<3> gt[TS], gp[TS];
  OneTile<TH> gh;
  OneTile<float> gu;
  float4_t ge, gw;
  float gg = 0.0f;
  auto rows_of = [&](int c) { return p.S - c * L < L ? p.S - c * L : L; };
  auto row4_of = [&](const float* x, int c) {
    return *reinterpret_cast<const float4_t*>(x + ((size_t)bh * p.Nc + c) * L + (owner ? 16 * rt + 4 * grp : 0));
  };
  auto fetch_k = [&](int c) {
    if (holds) gk.load(K + (size_t)c * L * DK, wave * W, rows_of(c), lane);
  };
  auto fetch_q = [&](int c) {
    if (holds) gq.load(Q + (size_t)c * L * DK, wave * W, rows_of(c), lane);
  };
  auto fetch_h = [&](int c) {
    gh.load(dH + (size_t)c * L * p.DV, p.DV, rows_of(c), rt, io_off);
    ge = row4_of(p.e, c);
    gg = p.e[((size_t)bh * p.Nc + c) * L + L - 1];
  };
  auto fetch_p = [&](int c) {
    const size_t at = (size_t)bh * p.Nc + c;
    load_square_rows<L, true, 3>(p.P + at * kSquare, rt, gp, lane);
    gu.load(p.U + at * L * p.DV, p.DV, L, rt, io_off);
    gw = row4_of(p.w, c);
  };
  auto fetch_t = [&](int c) {
    load_square_rows<L, true, 3>(p.Tt + ((size_t)bh * p.Nc + c) * kSquare, rt, gt, lane);
  };
  if (p.Nc) {
    fetch_h(p.Nc - 1);
    fetch_k(p.Nc - 1);
    fetch_q(p.Nc - 1);
    fetch_p(p.Nc - 1);
    fetch_t(p.Nc - 1);
  }

  for (int c = p.Nc - 1; c >= 0; --c) {
    const int t0 = c * L;
    const size_t at = (size_t)bh * p.Nc + c;
    const int next = c > 0 ? c - 1 : c;
    const float4_t e = ge;
    if (owner) {
      const float4_t h = p.scale * gh.tile();
      put_operand<3>(h_frags, rt, h, lane);
      put_operand<3>(eh_frags, rt, e * h, lane);
    }
    float4_t kg[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) kg[j] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
    if (holds) {
      gk.store(s_K, S::kPlane, lane);
      gq.store(s_Q, S::kPlane, lane);
      __builtin_amdgcn_wave_barrier();
      store_whole(Slice<float>(p.G_states + (at * DK + wave * W) * p.DV, p.DV, W, io_off), G);

      // this wave's share of K G
      Parts<3> gs[W / 32];
      state_parts<W>(G, gs);
      part_rows_times<NP, W, 3>(s_K, S::kPlane, row_seed, gs, kg);
      send_shares<S>(s_kg, kg, wave, lane);
#pragma unroll
      for (int k = 0; k < KT; ++k) G[k] *= gg;
    }
    fetch_h(next);
    fetch_k(next);
    __syncthreads();

    // the owners' tiles of dU = s P^T dH + w K G
    float anchor = 0.0f;
    if (owner) {
      const float4_t u = gu.tile();
      float4_t du = gw * take_shares<S>(s_kg, kg, rt, lane);
#pragma unroll
      for (int r = 0; r < 4; ++r) anchor += du[r] * u[r];
      tile_times<L, true, 3, 3>(gp, h_frags, rt, du, lane);
      put_operand<3>(du_frags, rt, du, lane);
    }
    fetch_q(next);
    fetch_p(next);
    __syncthreads();

    // ... and of dV = T^T dU
    if (owner) {
      float4_t dv = {0.0f, 0.0f, 0.0f, 0.0f};
      tile_times<L, true, 3, 3>(gt, du_frags, rt, dv, lane);
      put_operand<3>(dv_frags, rt, -e * dv, lane);
      store_one(Slice<float>(p.R + at * L * p.DV, p.DV, L, io_off), rt, dv);
      store_tile(Slice<TIn>(static_cast<TIn*>(p.dV) + ((size_t)bh * p.S + t0) * p.DV, p.DV, rows_of(c), io_off), rt, dv,
                 1.0f, lane);
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) anchor += __shfl_xor(anchor, o, 64);
      if (lane == 0) s_anchor[c & 1][wave] = anchor;
    }

    // G <- g G + Q^T (s e dH), before the barrier that dV needs, and - K^T (e dV)
    if (holds) {
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        const Parts<3> h = lds_row8<3>(eh_frags + ts * 3 * kFragElems + 8 * lane, kFragElems);
#pragma unroll
        for (int k = 0; k < KT; ++k)
          G[k] = mma_parts<NP, 3>(tile_col<NP, W>(s_Q, S::kPlane, col_seed, ts, k), h, G[k]);
      }
    }
    fetch_t(next);
    __syncthreads();
    if (holds) {
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        const Parts<3> d = lds_row8<3>(dv_frags + ts * 3 * kFragElems + 8 * lane, kFragElems);
#pragma unroll
        for (int k = 0; k < KT; ++k)
          G[k] = mma_parts<NP, 3>(tile_col<NP, W>(s_K, S::kPlane, col_seed, ts, k), d, G[k]);
      }
    }
    if (threadIdx.x == 0) {
      float a = 0.0f;
#pragma unroll
      for (int i = 0; i < RT; ++i) a += s_anchor[c & 1][i];
      p.anchor[at * (p.DV / 16) + slice] = a;
    }
  }

  if (p.dC0 && holds) store_whole(Slice<float>(p.dC0 + ((size_t)bh * DK + wave * W) * p.DV, p.DV, W, io_off), G);
}

template <typename TIn, typename TH, int DK>
hipError_t launch_dk(const DeltaParams& p, DeltaWalk what, hipStream_t stream) {
  const dim3 grid((unsigned)((long long)p.BH * (p.DV / 16))), block(64 * SplitShape<TIn, DK>::NW);
  switch (what) {
    case DeltaWalk::kForward:
      hipLaunchKernelGGL((delta_split_kernel<TIn, TH, DK, true>), grid, block, 0, stream, p);
      break;
    case DeltaWalk::kStates:
      hipLaunchKernelGGL((delta_split_kernel<TIn, float, DK, false>), grid, block, 0, stream, p);
      break;
    case DeltaWalk::kBack:
      hipLaunchKernelGGL((delta_split_back_kernel<TIn, TH, DK>), grid, block, 0, stream, p);
      break;
  }
  return hipGetLastError();
}

template <typename TIn, typename TH>
hipError_t launch_types(const DeltaParams& p, DeltaWalk what, hipStream_t stream) {
  switch (p.DK) {
    case 64: return launch_dk<TIn, TH, 64>(p, what, stream);
    case 128: return launch_dk<TIn, TH, 128>(p, what, stream);
    case 256: return launch_dk<TIn, TH, 256>(p, what, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_delta_split(const DeltaParams& p, DeltaWalk what, hipStream_t stream) {
  if (p.DV <= 0 || p.DV % 16 != 0) return hipErrorInvalidValue;
  if (p.qkv_bf16)
    return p.h_bf16 ? launch_types<bf16_t, bf16_t>(p, what, stream) : launch_types<bf16_t, float>(p, what, stream);
  return p.h_bf16 ? launch_types<float, bf16_t>(p, what, stream) : launch_types<float, float>(p, what, stream);
}

}  // namespace mlstm
