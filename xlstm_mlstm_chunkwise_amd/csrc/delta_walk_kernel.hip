// Gated delta rule: the chunks of a head in order, gfx950.
//
// One workgroup walks the chunks of one head for a slice of the value
// columns.  The columns of the state are independent of each other, so each
// wave carries all DHQK rows of sixteen columns in accumulator registers and
// no wave waits for another's result; the waves of a workgroup share the
// chunk's K, Q, T and P in LDS.  Per chunk (delta_prep_kernel.hip has T, P
// and the decays e, w; g = e of the chunk's last row):
//   U = T (V - e K C),   H = s (e Q C + P U),   C <- g C + K^T (w U).
// The accumulator tiles of C, of V - e K C and of U feed straight back as
// the right operand of the next product: the slot order of two accumulator
// tiles is matched by how the left operands are read from LDS.  The next
// chunk's K, Q, T and P are loaded into registers while this one computes and,
// where two buffers fit, stored to LDS under its last products; the backward
// walk, whose registers are full, stores them between two barriers.
//
// Bounds, at 64 heads of 256 x 512, 8192 tokens (128 chunks one after another
// on every CU):
// - the forward walk, 1.28-1.41 ms, by the matrix and vector instructions of
//   its waves together: the matrix cores are busy 50 % of the time at the 2.0
//   GHz that the load leaves, and of two conversions a matrix instruction the
//   third no longer hides.  Without the products with the state it would be
//   1.01 ms, without those of K^T 1.04, without the staging 1.29 (of 1.50).
//   Its 1.65 GB would take 0.32 ms.
// - the walk that keeps the states, 1.31 ms, and the backward walk, 2.45 ms,
//   also by the 4.3 GB of states each: written all at once at the start of a
//   chunk they took 1.65 and 2.55 ms, the waves waiting for the store queue.
#include "delta_walk.h"

namespace mlstm {
namespace {

// LDS of a workgroup: two input tiles (K, Q), two squares (T, P) and e, w.
template <typename TIn, int DK, int PP>
struct WalkLds {
  static constexpr int L = DeltaIn<TIn>::kChunk, NP = DeltaIn<TIn>::kParts, NF = square_frags<L>();
  static constexpr int kPlane = L * DK;
  static constexpr int kBytes = 2 * (2 * NP * kPlane + NF * (3 + PP) * kFragElems) + 4 * 2 * L;
  // two buffers of everything but Q (PP = 0: no Q and no P)
  static constexpr int kTwice = 2 * ((PP ? 3 : 2) * NP * kPlane + 2 * NF * (3 + PP) * kFragElems) + 4 * 4 * L;
  static constexpr bool kDouble = kTwice <= 160 * 1024;
};

// FWD: H (type TH) and the final state.  !FWD: the state entering every chunk
// and U, for the backward pass.  A bf16 H keeps eight bits: its own products
// take the state and P in two parts.
template <typename TIn, typename TH, int DK, int NW, bool FWD>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NW / 4, NW / 4))) void delta_walk_kernel(const DeltaParams p) {
  constexpr int PP = sizeof(TH) == 2 ? 2 : 3;
  typedef WalkLds<TIn, DK, FWD ? PP : 0> W;
  constexpr int L = W::L, NP = W::NP, RT = L / 16, TS = L / 32, KT = DK / 16, THREADS = 64 * NW;
  // With two buffers the next chunk's tiles are stored while this one is still
  // read, under the last products; Q, which only the first phase reads, needs
  // one, freed by a barrier behind that phase.
  constexpr bool DB = W::kDouble;
  constexpr int BUFS = DB ? 2 : 1, kTileK = NP * W::kPlane, kFragT = W::NF * 3 * kFragElems;
  constexpr int kFragP = FWD ? W::NF * PP * kFragElems : 0;
  __shared__ uint4 smem[(DB ? W::kTwice : W::kBytes) / 16];
  uint16_t* const m_K = reinterpret_cast<uint16_t*>(smem);
  uint16_t* const s_Q = m_K + BUFS * kTileK;
  uint16_t* const m_T = s_Q + (FWD || !DB ? kTileK : 0);
  uint16_t* const m_P = m_T + BUFS * kFragT;
  float* const m_e = reinterpret_cast<float*>(m_P + BUFS * kFragP);

  // slices of one head share an XCD's L2 where the head count is a multiple of 8
  const int bh = blockIdx.x % p.BH, slice = blockIdx.x / p.BH;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const int col = (slice * NW + wave) * 16 + row;
  const TIn* K = static_cast<const TIn*>(p.K) + (size_t)bh * p.S * DK;
  const TIn* Q = static_cast<const TIn*>(p.Q) + (size_t)bh * p.S * DK;
  const TIn* V = static_cast<const TIn*>(p.V) + (size_t)bh * p.S * p.DV;
  constexpr int kSquare = W::NF * 3 * kFragElems;
  int io_off = 4 * grp * p.DV + col;  // rows 16 rt + 4 grp + r of its column
  int row_seed = tile_row_seed<DK>(row, grp), col_seed = tile_col_seed<DK>(grp, lane);

  float4_t C[KT];
#pragma unroll
  for (int k = 0; k < KT; ++k) C[k] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  if (p.C0) load_whole(Slice<float>(p.C0 + (size_t)bh * DK * p.DV, p.DV, DK, io_off), C);

  TileStage<TIn, DK, THREADS> gk, gq;
  SquareStage<L, 3, THREADS> gt;
  SquareStage<L, PP, THREADS> gp;
  float ge = 0.0f;
  auto fetch = [&](int c) {
    const size_t at = (size_t)bh * p.Nc + c;
    const int rows = p.S - c * L < L ? p.S - c * L : L;
    gk.load(K + (size_t)c * L * DK, rows, tid);
    if constexpr (FWD) gq.load(Q + (size_t)c * L * DK, rows, tid);
    gt.load(p.T + at * kSquare, tid);
    if constexpr (FWD) gp.load(p.P + at * kSquare, tid);
    if (tid < 2 * L) ge = tid < L ? p.e[at * L + tid] : p.w[at * L + tid - L];
  };
  auto store = [&](int buf, int part) {
    if (part == 0) gk.store(m_K + buf * kTileK, W::kPlane, tid);
    if (FWD && part == 1) gq.store(s_Q, W::kPlane, tid);
    if (part == 2) gt.store(m_T + buf * kFragT, tid);
    if (FWD && part == 3) gp.store(m_P + buf * kFragP, tid);
    if (part == 3 && tid < 2 * L) m_e[buf * 2 * L + tid] = ge;
  };
  if (p.Nc) {
    fetch(0);
    if (DB)
      for (int i = 0; i < 4; ++i) store(0, i);
  }

  for (int c = 0; c < p.Nc; ++c) {
    const int t0 = c * L, buf = DB ? c & 1 : 0, next = c + 1 < p.Nc ? c + 1 : c;
    const size_t at = (size_t)bh * p.Nc + c;
    const uint16_t* s_K = m_K + buf * kTileK;
    const uint16_t* s_T = m_T + buf * kFragT;
    const uint16_t* s_P = m_P + buf * kFragP;
    const float* s_e = m_e + buf * 2 * L;
    const float* s_w = s_e + L;
    keep_in_loop(row_seed);
    keep_in_loop(col_seed);
    keep_in_loop(io_off);
    __syncthreads();  // the chunk before is read out (two buffers: and this one stored)
    if constexpr (!DB) {
#pragma unroll
      for (int i = 0; i < 4; ++i) store(0, i);
      __syncthreads();
      fetch(next);
    }
    RawTiles<TIn, RT> v;
    const int rows = p.S - t0 < L ? p.S - t0 : L;
    v.load(Slice<TIn>(V + (size_t)t0 * p.DV, p.DV, rows, io_off));
    __builtin_amdgcn_sched_barrier(0);  // all loads are on their way

    // The state entering a chunk leaves in two halves: the even tiles as soon
    // as the chunk before has finished them, the odd ones before they are
    // scaled.  All at once they fill the store queue, and the waves wait.
    const Slice<float> keep(FWD ? nullptr : p.C_states + at * DK * p.DV, p.DV, FWD ? 0 : DK, io_off);
    const Slice<float> keep_next(FWD ? nullptr : p.C_states + (at + 1) * DK * p.DV, p.DV, FWD || c + 1 == p.Nc ? 0 : DK,
                                 io_off);
    if constexpr (!FWD)
      if (c == 0)
#pragma unroll
        for (int k = 0; k < KT; k += 2) store_rows(keep, k, C[k]);

    // K C and Q C: a step is one 32-row block of the state against K's rows,
    // the next one against Q's.  A block that has become operand parts is
    // scaled by g on the way.
    const float g = s_e[L - 1];
    float4_t kc[RT], qc[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) kc[rt] = qc[rt] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
    {
      Parts<NP> f[RT], next[RT];
      float x[8];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) f[rt] = tile_row<NP, DK>(s_K, W::kPlane, row_seed, rt, 0);
      tiles8(C[0], C[1], x);
      Parts<3> cp = split_parts<3>(x), cn = cp;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) {
        const bool more = ks + 1 < DK / 32;
        words2_t lo[3] = {}, hi[3] = {};
        if constexpr (FWD) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) next[rt] = tile_row<NP, DK>(s_Q, W::kPlane, row_seed, rt, ks);
          if (more) split4<3>(C[2 * ks + 2], lo);
          rows_times(f, cp, kc);
          end_step<2 * NP * RT, RT * mma_count<NP, 3>(), 2>();
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) f[rt] = next[rt];
        }
        if constexpr (!FWD) store_rows(keep, 2 * ks + 1, C[2 * ks + 1]);
        C[2 * ks] *= g;
        C[2 * ks + 1] *= g;
        if (more) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) next[rt] = tile_row<NP, DK>(s_K, W::kPlane, row_seed, rt, ks + 1);
          if constexpr (!FWD) split4<3>(C[2 * ks + 2], lo);
          split4<3>(C[2 * ks + 3], hi);
          cn = join_halves(lo, hi);
        }
        if constexpr (FWD) rows_times(f, first_parts<PP>(cp), qc);
        else rows_times(f, cp, kc);
        if (more) end_step<2 * NP * RT, RT * (FWD ? mma_count<NP, PP>() : mma_count<NP, 3>()), 4>();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) f[rt] = next[rt];
        cp = cn;
      }
    }

    if constexpr (DB) {
      if constexpr (FWD) __syncthreads();  // Q is read out
      fetch(next);
      __builtin_amdgcn_sched_barrier(0);
    }

    // U = T (V - e K C)
    float4_t u[RT];
    {
      Parts<3> xp[TS];
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        float x[8];
        tiles8(v.tile(2 * ts) - row4(s_e, 2 * ts, grp) * kc[2 * ts],
               v.tile(2 * ts + 1) - row4(s_e, 2 * ts + 1, grp) * kc[2 * ts + 1], x);
        xp[ts] = split_parts<3>(x);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) u[rt] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
      __builtin_amdgcn_sched_barrier(0);
      square_times<L, false, 3, 3, 1>(s_T, xp, u, lane, [&](int i) {
        if (FWD && i < RT) qc[i] *= row4(s_e, i, grp);
      });
    }
    if constexpr (!FWD) store_whole(Slice<float>(p.U + at * L * p.DV, p.DV, L, io_off), u);

    // H = s (e Q C + P U), the parts of w U on the way
    Parts<3> wp[TS];
    if constexpr (FWD) {
      Parts<PP> up[TS];
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) {
        float x[8];
        tiles8(u[2 * ts], u[2 * ts + 1], x);
        up[ts] = split_parts<PP>(x);
      }
      __builtin_amdgcn_sched_barrier(0);
      square_times<L, false, PP, PP, 6>(s_P, up, qc, lane, [&](int i) {
        if (i < TS) wp[i] = scaled_parts(s_w, u, i, grp);
      });
    } else {
#pragma unroll
      for (int ts = 0; ts < TS; ++ts) wp[ts] = scaled_parts(s_w, u, ts, grp);
      __builtin_amdgcn_sched_barrier(0);
    }

    // C <- g C + K^T (w U), the stores of H on the way
    const Slice<TH> out(FWD ? static_cast<TH*>(p.H) + ((size_t)bh * p.S + t0) * p.DV : nullptr, p.DV, rows, io_off);
#pragma unroll
    for (int ts = 0; ts < TS; ++ts)
      tile_cols_times<NP, DK, 3>(s_K, W::kPlane, col_seed, ts, wp[ts], C, [&](int i) {
        const int rt = ts * (DK / 32) + i;
        if (FWD && rt < RT) store_tile(out, rt, qc[rt], p.scale, lane);
        if (!FWD && ts == TS - 1 && i > 0) store_rows(keep_next, 2 * i - 2, C[2 * i - 2]);
        if (DB && ts == TS - 1)
#pragma unroll
          for (int part = 0; part < 4; ++part)
            if (i == (part < DK / 32 ? part : DK / 32 - 1)) store(buf ^ 1, part);
      });
    if constexpr (!FWD) store_rows(keep_next, KT - 2, C[KT - 2]);
  }

  if (p.C_out) store_whole(Slice<float>(p.C_out + (size_t)bh * DK * p.DV, p.DV, DK, io_off), C);
}

// The backward walk, last chunk first.  G is the gradient of the state
// behind the chunk:
//   dU = s P^T dH + w K G,   dV = T^T dU,
//   G <- g G + Q^T (s e dH) - K^T (e dV).
// It writes G of every chunk and dV for the gradient kernel, and per column
// slice the chunk's sum of w_t u_t . (K G)_t, one half of <C, G> behind the
// chunk that the gate gradient needs.
template <typename TIn, typename TH, int DK, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NW / 4, NW / 4))) void delta_walk_back_kernel(const DeltaParams p) {
  typedef WalkLds<TIn, DK, 3> W;
  constexpr int L = W::L, NP = W::NP, RT = L / 16, TS = L / 32, KT = DK / 16, THREADS = 64 * NW;
  __shared__ uint4 smem[W::kBytes / 16];
  uint16_t* s_K = reinterpret_cast<uint16_t*>(smem);
  uint16_t* s_Q = s_K + NP * W::kPlane;
  uint16_t* s_T = s_Q + NP * W::kPlane;
  uint16_t* s_P = s_T + W::NF * 3 * kFragElems;
  float* s_e = reinterpret_cast<float*>(s_P + W::NF * 3 * kFragElems);
  float* s_w = s_e + L;

  const int bh = blockIdx.x % p.BH, slice = blockIdx.x / p.BH;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const int col = (slice * NW + wave) * 16 + row;
  const TIn* K = static_cast<const TIn*>(p.K) + (size_t)bh * p.S * DK;
  const TIn* Q = static_cast<const TIn*>(p.Q) + (size_t)bh * p.S * DK;
  const TH* dH = static_cast<const TH*>(p.dH) + (size_t)bh * p.S * p.DV;
  constexpr int kSquare = W::NF * 3 * kFragElems;
  int io_off = 4 * grp * p.DV + col;  // rows 16 rt + 4 grp + r of its column
  int row_seed = tile_row_seed<DK>(row, grp), col_seed = tile_col_seed<DK>(grp, lane);

  float4_t G[KT];
#pragma unroll
  for (int k = 0; k < KT; ++k) G[k] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  if (p.dC_out) load_whole(Slice<float>(p.dC_out + (size_t)bh * DK * p.DV, p.DV, DK, io_off), G);

  TileStage<TIn, DK, THREADS> gk, gq;
  SquareStage<L, 3, THREADS> gt, gp;
  float ge = 0.0f;
  auto fetch = [&](int c) {
    const size_t at = (size_t)bh * p.Nc + c;
    const int rows = p.S - c * L < L ? p.S - c * L : L;
    gk.load(K + (size_t)c * L * DK, rows, tid);
    gq.load(Q + (size_t)c * L * DK, rows, tid);
    gt.load(p.Tt + at * kSquare, tid);
    gp.load(p.P + at * kSquare, tid);
    if (tid < 2 * L) ge = tid < L ? p.e[at * L + tid] : p.w[at * L + tid - L];
  };
  if (p.Nc) fetch(p.Nc - 1);

  for (int c = p.Nc - 1; c >= 0; --c) {
    const int t0 = c * L;
    const size_t at = (size_t)bh * p.Nc + c;
    keep_in_loop(row_seed);
    keep_in_loop(col_seed);
    keep_in_loop(io_off);
    __syncthreads();  // the chunk before is read out
    gk.store(s_K, W::kPlane, tid);
    gq.store(s_Q, W::kPlane, tid);
    gt.store(s_T, tid);
    gp.store(s_P, tid);
    if (tid < 2 * L) s_e[tid] = ge;
    __syncthreads();
    if (c > 0) fetch(c - 1);
    float4_t u[RT], dh[RT];
    RawTiles<TH, RT> raw;
    const int rows = p.S - t0 < L ? p.S - t0 : L;
    load_whole(Slice<float>(p.U + at * L * p.DV, p.DV, L, io_off), u);
    raw.load(Slice<TH>(dH + (size_t)t0 * p.DV, p.DV, rows, io_off));
    __builtin_amdgcn_sched_barrier(0);  // all loads are on their way
    // in two halves, as the forward states
    const Slice<float> keep_g(p.G_states + at * DK * p.DV, p.DV, DK, io_off);
    const Slice<float> keep_next(p.G_states + (at - (c > 0)) * DK * p.DV, p.DV, c > 0 ? DK : 0, io_off);
    if (c == p.Nc - 1)
#pragma unroll
      for (int k = 0; k < KT; k += 2) store_rows(keep_g, k, G[k]);

    // w K G, and its product with u; blocks of G are scaled by g on the way
    const float g = s_e[L - 1];
    float4_t kg[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) kg[rt] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
    {
      Parts<NP> f[RT], next[RT];
      float x[8];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) f[rt] = tile_row<NP, DK>(s_K, W::kPlane, row_seed, rt, 0);
      tiles8(G[0], G[1], x);
      Parts<3> gs = split_parts<3>(x), gn = gs;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) {
        store_rows(keep_g, 2 * ks + 1, G[2 * ks + 1]);
        G[2 * ks] *= g;
        G[2 * ks + 1] *= g;
        if (ks + 1 < DK / 32) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) next[rt] = tile_row<NP, DK>(s_K, W::kPlane, row_seed, rt, ks + 1);
          tiles8(G[2 * ks + 2], G[2 * ks + 3], x);
          gn = split_parts<3>(x);
        }
        rows_times(f, gs, kg);
        if (ks + 1 < DK / 32) end_step<2 * NP * RT, RT * mma_count<NP, 3>(), 5>();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) f[rt] = next[rt];
        gs = gn;
      }
    }
    float anchor = 0.0f;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      kg[rt] *= row4(s_w, rt, grp);
#pragma unroll
      for (int r = 0; r < 4; ++r) anchor += kg[rt][r] * u[rt][r];
      dh[rt] = p.scale * raw.tile(rt);
    }

    // dU
    Parts<3> xp[TS], hp[TS];
#pragma unroll
    for (int ts = 0; ts < TS; ++ts) {
      float x[8];
      tiles8(dh[2 * ts], dh[2 * ts + 1], x);
      xp[ts] = split_parts<3>(x);
    }
    __builtin_amdgcn_sched_barrier(0);
    square_times<L, true, 3, 3, 3>(s_P, xp, kg, lane, [&](int i) {
      if (i < TS) hp[i] = scaled_parts(s_e, dh, i, grp);
    });

    // dV = T^T dU
    float4_t dv[RT];
#pragma unroll
    for (int ts = 0; ts < TS; ++ts) {
      float x[8];
      tiles8(kg[2 * ts], kg[2 * ts + 1], x);
      xp[ts] = split_parts<3>(x);
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) dv[rt] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
    __builtin_amdgcn_sched_barrier(0);
    square_times<L, true, 3, 3, 1>(s_T, xp, dv, lane);

    // G <- g G + Q^T (s e dH) - K^T (e dV), the stores of dV and the parts of
    // -e dV on the way
    const Slice<TIn> out(static_cast<TIn*>(p.dV) + ((size_t)bh * p.S + t0) * p.DV, p.DV, rows, io_off);
    const Slice<float> keep(p.R + at * L * p.DV, p.DV, L, io_off);
#pragma unroll
    for (int ts = 0; ts < TS; ++ts)
      tile_cols_times<NP, DK, 3>(s_Q, W::kPlane, col_seed, ts, hp[ts], G, [&](int i) {
        const int rt = ts * (DK / 32) + i;
        if (rt < RT) {
          store_tile(out, rt, dv[rt], 1.0f, lane);
          store_rows(keep, rt, dv[rt]);
        }
        if (i == DK / 32 - 1) {
#pragma unroll
          for (int h = 0; h < 2; ++h) dv[2 * ts + h] = -dv[2 * ts + h];
          xp[ts] = scaled_parts(s_e, dv, ts, grp);
        }
      });
#pragma unroll
    for (int ts = 0; ts < TS; ++ts)
      tile_cols_times<NP, DK, 2>(s_K, W::kPlane, col_seed, ts, xp[ts], G, [&](int i) {
        if (ts == TS - 1 && i > 0) store_rows(keep_next, 2 * i - 2, G[2 * i - 2]);
      });
    store_rows(keep_next, KT - 2, G[KT - 2]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) anchor += __shfl_xor(anchor, o, 64);
    if (lane == 0) p.anchor[at * (p.DV / 16) + slice * NW + wave] = anchor;
  }

  if (p.dC0) store_whole(Slice<float>(p.dC0 + (size_t)bh * DK * p.DV, p.DV, DK, io_off), G);
}

template <typename TIn, typename TH, int DK, int NW>
hipError_t launch_nw(const DeltaParams& p, DeltaWalk what, hipStream_t stream) {
  const dim3 grid((unsigned)((long long)p.BH * (p.DV / (16 * NW)))), block(64 * NW);
  switch (what) {
    case DeltaWalk::kForward:
      hipLaunchKernelGGL((delta_walk_kernel<TIn, TH, DK, NW, true>), grid, block, 0, stream, p);
      break;
    case DeltaWalk::kStates:
      hipLaunchKernelGGL((delta_walk_kernel<TIn, float, DK, NW, false>), grid, block, 0, stream, p);
      break;
    case DeltaWalk::kBack:
      hipLaunchKernelGGL((delta_walk_back_kernel<TIn, TH, DK, NW>), grid, block, 0, stream, p);
      break;
  }
  return hipGetLastError();
}

// Waves a workgroup, sixteen columns each: eight where that still leaves a
// workgroup for every CU (256), since they share the staging of K, Q, T and P.
// Forward and backward pass in us at 2048 tokens, 64 heads of 128 x 512 (256
// workgroups of eight): 228 and 1240, with four waves 316 and 1418; 256 heads
// of 128 x 128: 333 and 1549, with four 434 and 1735.  Below that eight waves
// would leave CUs idle.
template <typename TIn, typename TH, int DK>
hipError_t launch_dk(const DeltaParams& p, DeltaWalk what, hipStream_t stream) {
  if (p.DV % 128 == 0 && (long long)p.BH * (p.DV / 128) >= 256) return launch_nw<TIn, TH, DK, 8>(p, what, stream);
  return launch_nw<TIn, TH, DK, 4>(p, what, stream);
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

hipError_t launch_delta_walk(const DeltaParams& p, DeltaWalk what, hipStream_t stream) {
  if (p.DV <= 0 || p.DV % 64 != 0) return hipErrorInvalidValue;
  // Four-wave workgroups for every CU, or the form with the state's rows split
  // over the waves.  Forward and backward pass in us at 2048 tokens: 64 heads
  // of 128 x 128 (128 such workgroups) 177 and 601, split 148 and 569; 16 of
  // 256 x 512 (128) 219 and 735, split 209 and 667; 64 of 128 x 256 (256) 179
  // and 775, split 254 and 976; 32 of 256 x 512 (256) 240 and 1037, split 404
  // and 1345; float32, 1024 tokens, 64 of 128 x 256 (256) 160 and 588, split
  // 204 and 702.
  if ((long long)p.BH * (p.DV / 64) < 256) return launch_delta_split(p, what, stream);
  if (p.qkv_bf16)
    return p.h_bf16 ? launch_types<bf16_t, bf16_t>(p, what, stream) : launch_types<bf16_t, float>(p, what, stream);
  return p.h_bf16 ? launch_types<float, bf16_t>(p, what, stream) : launch_types<float, float>(p, what, stream);
}

}  // namespace mlstm
