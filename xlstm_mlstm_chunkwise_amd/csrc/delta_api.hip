// C ABI of the gated delta rule and of the head norm: argument validation,
// workspace layout and launches.  See include/mlstm_tfla.h for the contract
// of every entry point.
#include <math.h>
#include <initializer_list>
#include <stdint.h>

#include "kernels.h"
#include "mlstm_tfla.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_aligned(std::initializer_list<const void*> ptrs, uintptr_t a) {
  for (const void* p : ptrs)
    if (p && !aligned(p, a)) return MLSTM_E_ALIGN;
  return MLSTM_OK;
}

bool known_dtype(int32_t t) { return t == MLSTM_F32 || t == MLSTM_BF16; }

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

int chunk_rows(const mlstm_delta_desc_t* d) {
  return d->qkv_dtype == MLSTM_BF16 ? mlstm::kDeltaChunkBf16 : mlstm::kDeltaChunkF32;
}

int64_t num_chunks(const mlstm_delta_desc_t* d) {
  const int L = chunk_rows(d);
  return ((int64_t)d->S + L - 1) / L;
}

int validate(const mlstm_delta_desc_t* d) {
  if (!d) return MLSTM_E_NULLPTR;
  if (d->B < 1 || d->NH < 1 || d->S < 0 || d->S > (1 << 30)) return MLSTM_E_SHAPE;
  if (d->DHQK != 64 && d->DHQK != 128 && d->DHQK != 256) return MLSTM_E_SHAPE;
  if (d->DHV < 64 || d->DHV > 512 || d->DHV % 64 != 0) return MLSTM_E_SHAPE;
  if (!known_dtype(d->qkv_dtype) || !known_dtype(d->h_dtype)) return MLSTM_E_DTYPE;
  if (!isfinite(d->qk_scale)) return MLSTM_E_ARG;
  for (int32_t r : d->reserved)
    if (r) return MLSTM_E_ARG;
  // grids of 512-thread workgroups stay below 2^32 threads
  const int64_t BH = (int64_t)d->B * d->NH, lim = 1 << 23;
  if (BH >= lim || BH * (((int64_t)d->S + 31) / 32) >= lim || BH * (d->DHV / 64) >= lim) return MLSTM_E_SHAPE;
  return MLSTM_OK;
}

struct Layout {
  size_t T, P, bsum, e, w, fw_total, Tt, C, G, U, R, anchor, bw_total;
};

Layout layout(const mlstm_delta_desc_t* d) {
  const size_t n = (size_t)d->B * d->NH * (size_t)num_chunks(d), L = (size_t)chunk_rows(d);
  const size_t state = (size_t)d->DHQK * d->DHV;
  Layout l;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += round_up(bytes);
    return at;
  };
  const size_t square = mlstm::delta_square_bytes((int)L);
  l.T = take(n * square);
  l.P = take(n * square);
  l.bsum = take(n * L * sizeof(double));
  l.e = take(n * L * sizeof(float));
  l.w = take(n * L * sizeof(float));
  l.fw_total = off;
  l.Tt = take(n * square);
  l.C = take(n * state * sizeof(float));
  l.G = take(n * state * sizeof(float));
  l.U = take(n * L * d->DHV * sizeof(float));
  l.R = take(n * L * d->DHV * sizeof(float));
  l.anchor = take(n * (d->DHV / 16) * sizeof(float));
  l.bw_total = off;
  return l;
}

mlstm::DeltaParams params(const mlstm_delta_desc_t* d, const Layout& l, const void* Q, const void* K, const void* V,
                          const float* i_pre, const float* f_pre, const float* C0, void* workspace) {
  mlstm::DeltaParams p = {};
  char* ws = static_cast<char*>(workspace);
  auto at = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  p.Q = Q;
  p.K = K;
  p.V = V;
  p.i_pre = i_pre;
  p.f_pre = f_pre;
  p.C0 = C0;
  if (ws) {
    p.T = reinterpret_cast<uint16_t*>(ws + l.T);
    p.P = reinterpret_cast<uint16_t*>(ws + l.P);
    p.bsum = reinterpret_cast<double*>(ws + l.bsum);
    p.e = at(l.e);
    p.w = at(l.w);
  }
  p.scale = d->qk_scale > 0.0f ? d->qk_scale : 1.0f / sqrtf((float)d->DHQK);
  p.BH = d->B * d->NH;
  p.S = d->S;
  p.DK = d->DHQK;
  p.DV = d->DHV;
  p.Nc = (int)num_chunks(d);
  p.qkv_bf16 = d->qkv_dtype == MLSTM_BF16;
  p.h_bf16 = d->h_dtype == MLSTM_BF16;
  return p;
}

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws && bytes >= need && aligned(ws, 256));
}

int status(hipError_t e) { return e == hipSuccess ? MLSTM_OK : MLSTM_E_HIP; }

int lanes_limit_ok(const mlstm_head_norm_desc_t* d) {
  const int64_t rows = (int64_t)d->B * d->S;
  return rows < (1LL << 30) && rows * d->NH < (1LL << 26) && d->NH < (1 << 22);
}

int validate(const mlstm_head_norm_desc_t* d) {
  if (!d) return MLSTM_E_NULLPTR;
  if (d->B < 1 || d->NH < 1 || d->S < 0) return MLSTM_E_SHAPE;
  if (d->D < 64 || d->D > 512 || d->D % 64 != 0) return MLSTM_E_SHAPE;
  if (!lanes_limit_ok(d)) return MLSTM_E_SHAPE;
  if (!known_dtype(d->x_dtype) || !known_dtype(d->y_dtype)) return MLSTM_E_DTYPE;
  if (!(d->eps >= 0.0f) || !isfinite(d->eps)) return MLSTM_E_ARG;
  for (int32_t r : d->reserved)
    if (r) return MLSTM_E_ARG;
  return MLSTM_OK;
}

mlstm::HeadNormParams params(const mlstm_head_norm_desc_t* d) {
  mlstm::HeadNormParams p = {};
  p.eps = d->eps;
  p.B = d->B;
  p.NH = d->NH;
  p.S = d->S;
  p.D = d->D;
  p.blocks = mlstm::head_norm_blocks(d->B, d->NH, d->S, d->D);
  p.x_bf16 = d->x_dtype == MLSTM_BF16;
  p.y_bf16 = d->y_dtype == MLSTM_BF16;
  return p;
}

}  // namespace

extern "C" {

int mlstm_delta_validate(const mlstm_delta_desc_t* desc) { return validate(desc); }

size_t mlstm_delta_fw_workspace_bytes(const mlstm_delta_desc_t* desc) {
  return validate(desc) == MLSTM_OK ? layout(desc).fw_total : 0;
}

size_t mlstm_delta_bw_workspace_bytes(const mlstm_delta_desc_t* desc) {
  return validate(desc) == MLSTM_OK ? layout(desc).bw_total : 0;
}

int mlstm_delta_fw(const mlstm_delta_desc_t* desc, const void* Q, const void* K, const void* V, const float* i_pre,
                   const float* f_pre, const float* C0, void* H, float* C_out, void* workspace,
                   size_t workspace_bytes, void* stream) {
  int st = validate(desc);
  if (st != MLSTM_OK) return st;
  if (desc->S > 0 && (!Q || !K || !V || !i_pre || !f_pre || !H)) return MLSTM_E_NULLPTR;
  if ((st = check_aligned({Q, K, V, H}, 16)) != MLSTM_OK) return st;
  if ((st = check_aligned({i_pre, f_pre, C0, C_out}, 4)) != MLSTM_OK) return st;
  const Layout l = layout(desc);
  if (!workspace_ok(workspace, workspace_bytes, l.fw_total)) return MLSTM_E_WORKSPACE;
  mlstm::DeltaParams p = params(desc, l, Q, K, V, i_pre, f_pre, C0, workspace);
  p.H = H;
  p.C_out = C_out;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = p.Nc ? mlstm::launch_delta_prep(p, false, s) : hipSuccess;
  if (e == hipSuccess && (p.Nc || C_out)) e = mlstm::launch_delta_walk(p, mlstm::DeltaWalk::kForward, s);
  return status(e);
}

int mlstm_delta_bw(const mlstm_delta_desc_t* desc, const void* Q, const void* K, const void* V, const float* i_pre,
                   const float* f_pre, const float* C0, const void* dH, const float* dC_out, void* dQ, void* dK,
                   void* dV, float* d_i, float* d_f, float* dC0, void* workspace, size_t workspace_bytes,
                   void* stream) {
  int st = validate(desc);
  if (st != MLSTM_OK) return st;
  if (desc->S > 0 && (!Q || !K || !V || !i_pre || !f_pre || !dH || !dQ || !dK || !dV || !d_i || !d_f))
    return MLSTM_E_NULLPTR;
  if ((st = check_aligned({Q, K, V, dH, dQ, dK, dV}, 16)) != MLSTM_OK) return st;
  if ((st = check_aligned({i_pre, f_pre, C0, dC_out, d_i, d_f, dC0}, 4)) != MLSTM_OK) return st;
  const Layout l = layout(desc);
  if (!workspace_ok(workspace, workspace_bytes, l.bw_total)) return MLSTM_E_WORKSPACE;
  mlstm::DeltaParams p = params(desc, l, Q, K, V, i_pre, f_pre, C0, workspace);
  char* ws = static_cast<char*>(workspace);
  if (ws) {
    p.Tt = reinterpret_cast<uint16_t*>(ws + l.Tt);
    p.C_states = reinterpret_cast<float*>(ws + l.C);
    p.G_states = reinterpret_cast<float*>(ws + l.G);
    p.U = reinterpret_cast<float*>(ws + l.U);
    p.R = reinterpret_cast<float*>(ws + l.R);
    p.anchor = reinterpret_cast<float*>(ws + l.anchor);
  }
  p.dH = dH;
  p.dC_out = dC_out;
  p.dQ = dQ;
  p.dK = dK;
  p.dV = dV;
  p.d_i = d_i;
  p.d_f = d_f;
  p.dC0 = dC0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (p.Nc) {
    e = mlstm::launch_delta_prep(p, true, s);
    if (e == hipSuccess) e = mlstm::launch_delta_walk(p, mlstm::DeltaWalk::kStates, s);
  }
  if (e == hipSuccess && (p.Nc || dC0)) e = mlstm::launch_delta_walk(p, mlstm::DeltaWalk::kBack, s);
  if (e == hipSuccess && p.Nc) e = mlstm::launch_delta_grads(p, s);
  return status(e);
}

int mlstm_delta_step(const mlstm_delta_desc_t* desc, const void* q, const void* k, const void* v, const float* i_pre,
                     const float* f_pre, const float* C_in, void* h, float* C_out, void* stream) {
  int st = validate(desc);
  if (st != MLSTM_OK) return st;
  if (desc->S != 1) return MLSTM_E_SHAPE;
  if (!q || !k || !v || !i_pre || !f_pre || !h || !C_out) return MLSTM_E_NULLPTR;
  if ((st = check_aligned({q, k, v, h, C_in, C_out}, 16)) != MLSTM_OK) return st;
  if ((st = check_aligned({i_pre, f_pre}, 4)) != MLSTM_OK) return st;
  mlstm::DeltaStepParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.i_pre = i_pre;
  p.f_pre = f_pre;
  p.C_in = C_in;
  p.h = h;
  p.C_out = C_out;
  p.scale = desc->qk_scale > 0.0f ? desc->qk_scale : 1.0f / sqrtf((float)desc->DHQK);
  p.BH = desc->B * desc->NH;
  p.DK = desc->DHQK;
  p.DV = desc->DHV;
  p.qkv_bf16 = desc->qkv_dtype == MLSTM_BF16;
  p.h_bf16 = desc->h_dtype == MLSTM_BF16;
  return status(mlstm::launch_delta_step(p, static_cast<hipStream_t>(stream)));
}

int mlstm_head_norm_validate(const mlstm_head_norm_desc_t* desc) { return validate(desc); }

size_t mlstm_head_norm_bw_workspace_bytes(const mlstm_head_norm_desc_t* desc) {
  if (validate(desc) != MLSTM_OK) return 0;
  return round_up((size_t)params(desc).blocks * desc->NH * 2 * desc->D * sizeof(float));
}

int mlstm_head_norm_fw(const mlstm_head_norm_desc_t* desc, const void* x, const float* weight, const float* bias,
                       void* y, void* stream) {
  int st = validate(desc);
  if (st != MLSTM_OK) return st;
  if (desc->S == 0) return MLSTM_OK;
  if (!x || !y) return MLSTM_E_NULLPTR;
  if ((st = check_aligned({x, weight, bias, y}, 16)) != MLSTM_OK) return st;
  mlstm::HeadNormParams p = params(desc);
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.y = y;
  return status(mlstm::launch_head_norm(p, static_cast<hipStream_t>(stream)));
}

int mlstm_head_norm_bw(const mlstm_head_norm_desc_t* desc, const void* x, const float* weight, const void* dy,
                       void* dx, float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                       void* stream) {
  int st = validate(desc);
  if (st != MLSTM_OK) return st;
  if (desc->S > 0 && (!x || !dy || !dx)) return MLSTM_E_NULLPTR;
  if ((st = check_aligned({x, weight, dy, dx}, 16)) != MLSTM_OK) return st;
  if ((st = check_aligned({dweight, dbias}, 4)) != MLSTM_OK) return st;
  const bool sums = dweight || dbias;
  if (sums && !workspace_ok(workspace, workspace_bytes, mlstm_head_norm_bw_workspace_bytes(desc)))
    return MLSTM_E_WORKSPACE;
  if (desc->S == 0 && !sums) return MLSTM_OK;
  mlstm::HeadNormParams p = params(desc);
  p.x = x;
  p.weight = weight;
  p.dy = dy;
  p.dx = dx;
  p.dweight = dweight;
  p.dbias = dbias;
  p.partial = sums ? static_cast<float*>(workspace) : nullptr;
  return status(mlstm::launch_head_norm_back(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
