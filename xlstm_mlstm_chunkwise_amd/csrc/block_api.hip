// C ABI of the short causal convolution, the selective scan and dropout:
// argument validation, workspace layout and launches.  See
// include/mlstm_tfla.h for the contract of every entry point.
#include <math.h>
#include <array>
#include <initializer_list>
#include <stdint.h>

#include "kernels.h"
#include "mlstm_tfla.h"

namespace {

int check_aligned(std::initializer_list<const void*> ptrs, uintptr_t a) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & (a - 1)) return MLSTM_E_ALIGN;
  return MLSTM_OK;
}

bool any_null(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!p) return true;
  return false;
}

bool known_dtype(int32_t t) { return t == MLSTM_F32 || t == MLSTM_BF16; }
uintptr_t size_of(int32_t t) { return t == MLSTM_BF16 ? 2 : 4; }
size_t round_up(size_t x) { return (x + 255) / 256 * 256; }
int status(hipError_t e) { return e == hipSuccess ? MLSTM_OK : MLSTM_E_HIP; }

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws && bytes >= need && (reinterpret_cast<uintptr_t>(ws) & 255) == 0);
}

// A tensor's memory, from its first byte to behind its last; empty if it is not given.
struct Span {
  uintptr_t first, end;
};

Span span(const void* p, int64_t bytes) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return {at, p ? at + (uintptr_t)bytes : at};
}

Span span(const mlstm::View& v, int64_t B, int64_t S, int64_t columns, int64_t size) {
  return span(v.p, S ? ((B - 1) * v.batch + (S - 1) * v.token + columns) * size : 0);
}

// Whether an output shares memory with an input: other threads read that after
// it is written.
template <typename Ins>
int check_apart(std::initializer_list<Span> outs, const Ins& ins) {
  for (const Span& o : outs)
    for (const Span& i : ins)
      if (o.first < o.end && i.first < i.end && o.first < i.end && i.first < o.end) return MLSTM_E_OVERLAP;
  return MLSTM_OK;
}
typedef std::initializer_list<Span> Spans;

// 0 stands for a contiguous tensor's strides.
mlstm::View view(const void* p, const int64_t (&strides)[2], int64_t S, int64_t columns) {
  return {p, strides[0] ? strides[0] : S * columns, strides[1] ? strides[1] : columns};
}

// A token's columns lie side by side and tokens do not overlap; a token's
// stride keeps offsets over a few tokens in 32 bits, a batch's the others in 62.
bool bad_strides(const int64_t (&s)[2], int64_t B, int64_t columns) {
  return s[0] < 0 || s[0] > ((int64_t)1 << 59) / B || (s[1] && (s[1] < columns || s[1] >= (1 << 25)));
}

// B, S and D as the descriptors' comments have them.
bool bad_shape(int64_t B, int64_t S, int64_t D, int64_t more) {
  return B < 1 || D < 1 || S < 0 || S >= (1 << 30) || B * (S + more) >= ((int64_t)1 << 40) ||
         (B * (S + more)) * (D < (1 << 23) ? D : (int64_t)1 << 23) >= ((int64_t)1 << 40) || D >= (1 << 22);
}

int validate(const mlstm_conv_desc_t* d) {
  if (!d) return MLSTM_E_NULLPTR;
  if (bad_shape(d->B, d->S, d->D, 3)) return MLSTM_E_SHAPE;
  if (d->B >= (1 << 16) || (int64_t)d->B * (d->S + 3) >= ((int64_t)1 << 32)) return MLSTM_E_SHAPE;
  if (d->K < 2 || d->K > 4) return MLSTM_E_SHAPE;
  if (!known_dtype(d->dtype)) return MLSTM_E_DTYPE;
  if (d->silu != 0 && d->silu != 1) return MLSTM_E_ARG;
  if (bad_strides(d->x_strides, d->B, d->D)) return MLSTM_E_ARG;
  for (int32_t r : d->reserved)
    if (r) return MLSTM_E_ARG;
  return MLSTM_OK;
}

mlstm::ConvParams params(const mlstm_conv_desc_t* d, const void* x, const float* weight, const float* bias,
                         const void* state, bool back) {
  mlstm::ConvParams p = {};
  p.x = view(x, d->x_strides, d->S, d->D);
  p.weight = weight;
  p.bias = bias;
  p.state = state;
  p.B = d->B;
  p.S = d->S;
  p.D = d->D;
  p.K = d->K;
  p.bf16 = d->dtype == MLSTM_BF16;
  p.silu = d->silu;
  mlstm::conv_runs(p.B, p.S, p.D, back, &p.run, &p.runs);
  return p;
}

// The inputs' memory but the state's, and the bytes of x's rows, the state and the weights.
struct ConvSpans {
  int64_t rows, state, weight, bias;
  std::array<Span, 3> in;
  ConvSpans(const mlstm_conv_desc_t* d, const mlstm::ConvParams& p) {
    const int64_t size = (int64_t)size_of(d->dtype), B = d->B, S = d->S, D = d->D, K = d->K;
    rows = B * S * D * size;
    state = B * (K - 1) * D * size;
    weight = 4 * D * K;
    bias = 4 * D;
    in = {span(p.x, B, S, D, size), span(p.weight, weight), span(p.bias, bias)};
  }
};

int validate(const mlstm_scan_desc_t* d) {
  if (!d) return MLSTM_E_NULLPTR;
  if (bad_shape(d->B, d->S, d->D, 0)) return MLSTM_E_SHAPE;
  if ((int64_t)d->B * (((int64_t)d->D + 63) / 64) >= (1 << 20)) return MLSTM_E_SHAPE;
  if (d->N != 16 && d->N != 32 && d->N != 64) return MLSTM_E_SHAPE;
  if (!known_dtype(d->dtype)) return MLSTM_E_DTYPE;
  for (const int64_t(*s)[2] : {&d->x_strides, &d->dt_strides, &d->z_strides})
    if (bad_strides(*s, d->B, d->D)) return MLSTM_E_ARG;
  if (bad_strides(d->B_strides, d->B, d->N) || bad_strides(d->C_strides, d->B, d->N)) return MLSTM_E_ARG;
  if (d->reserved0) return MLSTM_E_ARG;
  for (int32_t r : d->reserved)
    if (r) return MLSTM_E_ARG;
  return MLSTM_OK;
}

mlstm::ScanParams params(const mlstm_scan_desc_t* d, const void* x, const void* dt, const float* A, const void* Bm,
                         const void* Cm, const float* Dskip, const void* z, const float* bias, const float* h0) {
  mlstm::ScanParams p = {};
  p.x = view(x, d->x_strides, d->S, d->D);
  p.dt = view(dt, d->dt_strides, d->S, d->D);
  p.z = view(z, d->z_strides, d->S, d->D);
  p.Bm = view(Bm, d->B_strides, d->S, d->N);
  p.Cm = view(Cm, d->C_strides, d->S, d->N);
  p.A = A;
  p.Dskip = Dskip;
  p.bias = bias;
  p.h0 = h0;
  p.B = d->B;
  p.S = d->S;
  p.D = d->D;
  p.N = d->N;
  p.bf16 = d->dtype == MLSTM_BF16;
  return p;
}

// The inputs' memory but the state's, and the bytes of x's rows, Bm's, the state,
// A and a value a channel.
struct ScanSpans {
  int64_t rows, columns, state, A, channels;
  std::array<Span, 8> in;
  ScanSpans(const mlstm_scan_desc_t* d, const mlstm::ScanParams& p) {
    const int64_t size = (int64_t)size_of(d->dtype), B = d->B, S = d->S, D = d->D, N = d->N;
    rows = B * S * D * size;
    columns = B * S * N * size;
    state = 4 * B * D * N;
    A = 4 * D * N;
    channels = 4 * D;
    in = {span(p.x, B, S, D, size),  span(p.dt, B, S, D, size), span(p.z, B, S, D, size),  span(p.Bm, B, S, N, size),
          span(p.Cm, B, S, N, size), span(p.A, A),              span(p.Dskip, channels), span(p.bias, channels)};
  }
};

// Cuts the sequence, places the workspace (none: sizes only) and returns its bytes.
size_t place(mlstm::ScanParams& p, bool back, void* workspace) {
  p.rows = (p.S + mlstm::kScanTile - 1) / mlstm::kScanTile * mlstm::kScanTile;
  mlstm::scan_cut(p, back);
  size_t off = 0;
  char* ws = static_cast<char*>(workspace);
  auto take = [&](size_t floats) {
    float* at = ws ? reinterpret_cast<float*>(ws + off) : nullptr;
    off += round_up(floats * sizeof(float));
    return at;
  };
  const size_t B = p.B, S = p.S, D = p.D, N = p.N, states = B * p.chunks * D, spans = B * p.spans * D;
  if (!S) return 0;
  p.bc = take(B * p.rows * 2 * N);
  if (p.chunks > 1) {
    p.ends = take(states * N);
    p.sums = take(states);
  }
  if (back) {
    const size_t ch = mlstm::scan_back_channels(p.N);
    if (p.spans > 1) {
      p.grads = take(spans * N);
      p.span_sums = take(spans);
    }
    p.kept = take(B * (p.rows / mlstm::kScanBlock) * D * N);
    p.part_bc = take((D + ch - 1) / ch * B * S * 2 * N);
    p.part_a = take(spans * N);
    p.part_d = take(spans * 2);
  }
  return off;
}

size_t workspace_bytes(const mlstm_scan_desc_t* d, bool back) {
  if (validate(d) != MLSTM_OK) return 0;
  mlstm::ScanParams p = params(d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  return place(p, back, nullptr);
}

int validate(const mlstm_dropout_desc_t* d) {
  if (!d) return MLSTM_E_NULLPTR;
  if (d->n < 0 || d->n > ((int64_t)1 << 40)) return MLSTM_E_SHAPE;
  if (!known_dtype(d->dtype)) return MLSTM_E_DTYPE;
  if (!(d->p >= 0.0 && d->p < 1.0)) return MLSTM_E_ARG;
  for (int32_t r : d->reserved)
    if (r) return MLSTM_E_ARG;
  return MLSTM_OK;
}

}  // namespace

extern "C" {

int mlstm_conv_validate(const mlstm_conv_desc_t* desc) { return validate(desc); }

size_t mlstm_conv_bw_workspace_bytes(const mlstm_conv_desc_t* desc) {
  if (validate(desc) != MLSTM_OK) return 0;
  const mlstm::ConvParams p = params(desc, nullptr, nullptr, nullptr, nullptr, true);
  return round_up((size_t)p.runs * (p.K + 1) * p.D * sizeof(float));
}

int mlstm_conv_fw(const mlstm_conv_desc_t* desc, const void* x, const float* weight, const float* bias,
                  const void* state, void* y, void* state_out, void* stream) {
  int st = validate(desc);
  if (st != MLSTM_OK) return st;
  if (!weight || (desc->S > 0 && any_null({x, y}))) return MLSTM_E_NULLPTR;
  if ((st = check_aligned({x, state, y, state_out}, size_of(desc->dtype))) != MLSTM_OK) return st;
  if ((st = check_aligned({weight, bias}, 4)) != MLSTM_OK) return st;
  mlstm::ConvParams p = params(desc, x, weight, bias, state, false);
  p.y = y;
  p.state_out = state_out;
  const ConvSpans n(desc, p);
  const Spans outs = {span(y, n.rows), span(state_out, n.state)};
  if ((st = check_apart(outs, n.in)) != MLSTM_OK) return st;
  if ((st = check_apart(outs, Spans{span(state, n.state)})) != MLSTM_OK) return st;
  if (p.S == 0 && !state_out) return MLSTM_OK;
  return status(mlstm::launch_conv(p, static_cast<hipStream_t>(stream)));
}

int mlstm_conv_bw(const mlstm_conv_desc_t* desc, const void* x, const float* weight, const float* bias,
                  const void* state, const void* dy, const void* dstate_out, void* dx, void* dstate, float* dweight,
                  float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  int st = validate(desc);
  if (st != MLSTM_OK) return st;
  if (!weight || (desc->S > 0 && any_null({x, dy, dx}))) return MLSTM_E_NULLPTR;
  if ((st = check_aligned({x, state, dy, dstate_out, dx, dstate}, size_of(desc->dtype))) != MLSTM_OK) return st;
  if ((st = check_aligned({weight, bias, dweight, dbias}, 4)) != MLSTM_OK) return st;
  const bool sums = dweight || dbias;
  if (sums && !workspace_ok(workspace, workspace_bytes, mlstm_conv_bw_workspace_bytes(desc))) return MLSTM_E_WORKSPACE;
  mlstm::ConvParams p = params(desc, x, weight, bias, state, true);
  p.dy = dy;
  p.dstate_out = dstate_out;
  p.dx = dx;
  p.dstate = dstate;
  p.dweight = dweight;
  p.dbias = dbias;
  p.partial = sums ? static_cast<float*>(workspace) : nullptr;
  const ConvSpans n(desc, p);
  const Spans outs = {span(dx, n.rows), span(dstate, n.state), span(dweight, n.weight), span(dbias, n.bias)};
  if ((st = check_apart(outs, n.in)) != MLSTM_OK) return st;
  if ((st = check_apart(outs, Spans{span(state, n.state), span(dy, n.rows), span(dstate_out, n.state)})) != MLSTM_OK) return st;
  return status(mlstm::launch_conv_back(p, static_cast<hipStream_t>(stream)));
}

int mlstm_conv_step(const mlstm_conv_desc_t* desc, const void* x, const float* weight, const float* bias,
                    const void* state, void* y, void* state_out, void* stream) {
  int st = validate(desc);
  if (st != MLSTM_OK) return st;
  if (desc->S != 1) return MLSTM_E_SHAPE;
  if (any_null({x, weight, y, state_out})) return MLSTM_E_NULLPTR;
  if ((st = check_aligned({x, state, y, state_out}, size_of(desc->dtype))) != MLSTM_OK) return st;
  if ((st = check_aligned({weight, bias}, 4)) != MLSTM_OK) return st;
  mlstm::ConvParams p = params(desc, x, weight, bias, state, false);
  p.y = y;
  p.state_out = state_out;
  const ConvSpans n(desc, p);
  if ((st = check_apart({span(y, n.rows), span(state_out, n.state)}, n.in)) != MLSTM_OK) return st;
  if ((st = check_apart({span(y, n.rows), span(state != state_out ? state_out : nullptr, n.state)},
                        Spans{span(state, n.state)})) != MLSTM_OK)
    return st;
  return status(mlstm::launch_conv_step(p, static_cast<hipStream_t>(stream)));
}

int mlstm_scan_validate(const mlstm_scan_desc_t* desc) { return validate(desc); }

size_t mlstm_scan_fw_workspace_bytes(const mlstm_scan_desc_t* desc) { return workspace_bytes(desc, false); }
size_t mlstm_scan_bw_workspace_bytes(const mlstm_scan_desc_t* desc) { return workspace_bytes(desc, true); }

int mlstm_scan_fw(const mlstm_scan_desc_t* desc, const void* x, const void* dt, const float* A, const void* Bm,
                  const void* Cm, const float* Dskip, const void* z, const float* dt_bias, const float* h0, void* y,
                  float* h_out, void* workspace, size_t workspace_bytes, void* stream) {
  int st = validate(desc);
  if (st != MLSTM_OK) return st;
  if (!A || (desc->S > 0 && any_null({x, dt, Bm, Cm, y}))) return MLSTM_E_NULLPTR;
  if ((st = check_aligned({x, dt, Bm, Cm, z, y}, size_of(desc->dtype))) != MLSTM_OK) return st;
  if ((st = check_aligned({Dskip, dt_bias}, 4)) != MLSTM_OK) return st;
  if ((st = check_aligned({A, h0, h_out}, 16)) != MLSTM_OK) return st;
  mlstm::ScanParams p = params(desc, x, dt, A, Bm, Cm, Dskip, z, dt_bias, h0);
  if (!workspace_ok(workspace, workspace_bytes, place(p, false, workspace))) return MLSTM_E_WORKSPACE;
  p.y = y;
  p.h_out = h_out;
  const ScanSpans n(desc, p);
  const Spans outs = {span(y, n.rows), span(h_out, n.state)};
  if ((st = check_apart(outs, n.in)) != MLSTM_OK) return st;
  if ((st = check_apart(outs, Spans{span(h0, n.state)})) != MLSTM_OK) return st;
  if (p.S == 0 && !h_out) return MLSTM_OK;
  return status(mlstm::launch_scan(p, static_cast<hipStream_t>(stream)));
}

int mlstm_scan_bw(const mlstm_scan_desc_t* desc, const void* x, const void* dt, const float* A, const void* Bm,
                  const void* Cm, const float* Dskip, const void* z, const float* dt_bias, const float* h0,
                  const void* dy, const float* dh_out, void* dx, void* ddt, float* dA, void* dBm, void* dCm,
                  float* dDskip, void* dz, float* dbias, float* dh0, void* workspace, size_t workspace_bytes,
                  void* stream) {
  int st = validate(desc);
  if (st != MLSTM_OK) return st;
  if (!A || !dA || (desc->S > 0 && any_null({x, dt, Bm, Cm, dy, dx, ddt, dBm, dCm}))) return MLSTM_E_NULLPTR;
  if (desc->S > 0 && z && !dz) return MLSTM_E_NULLPTR;
  if (!z && dz) return MLSTM_E_UNSUPPORTED;
  if ((st = check_aligned({x, dt, Bm, Cm, z, dy, dx, ddt, dBm, dCm, dz}, size_of(desc->dtype))) != MLSTM_OK) return st;
  if ((st = check_aligned({Dskip, dt_bias, dDskip, dbias}, 4)) != MLSTM_OK) return st;
  if ((st = check_aligned({A, h0, dh_out, dA, dh0}, 16)) != MLSTM_OK) return st;
  mlstm::ScanParams p = params(desc, x, dt, A, Bm, Cm, Dskip, z, dt_bias, h0);
  if (!workspace_ok(workspace, workspace_bytes, place(p, true, workspace))) return MLSTM_E_WORKSPACE;
  p.dy = dy;
  p.dh_out = dh_out;
  p.dx = dx;
  p.ddt = ddt;
  p.dA = dA;
  p.dBm = dBm;
  p.dCm = dCm;
  p.dDskip = dDskip;
  p.dz = dz;
  p.dbias = dbias;
  p.dh0 = dh0;
  const ScanSpans n(desc, p);
  const Spans outs = {span(dx, n.rows),        span(ddt, n.rows),       span(dA, n.A),
                      span(dBm, n.columns),    span(dCm, n.columns),    span(dDskip, n.channels),
                      span(dz, n.rows),        span(dbias, n.channels), span(dh0, n.state)};
  if ((st = check_apart(outs, n.in)) != MLSTM_OK) return st;
  if ((st = check_apart(outs, Spans{span(h0, n.state), span(dy, n.rows), span(dh_out, n.state)})) != MLSTM_OK) return st;
  return status(mlstm::launch_scan_back(p, static_cast<hipStream_t>(stream)));
}

int mlstm_scan_step(const mlstm_scan_desc_t* desc, const void* x, const void* dt, const float* A, const void* Bm,
                    const void* Cm, const float* Dskip, const void* z, const float* dt_bias, const float* h_in,
                    void* y, float* h_out, void* stream) {
  int st = validate(desc);
  if (st != MLSTM_OK) return st;
  if (desc->S != 1) return MLSTM_E_SHAPE;
  if (any_null({x, dt, A, Bm, Cm, y, h_out})) return MLSTM_E_NULLPTR;
  if ((st = check_aligned({x, dt, Bm, Cm, z, y}, size_of(desc->dtype))) != MLSTM_OK) return st;
  if ((st = check_aligned({Dskip, dt_bias}, 4)) != MLSTM_OK) return st;
  if ((st = check_aligned({A, h_in, h_out}, 16)) != MLSTM_OK) return st;
  mlstm::ScanParams p = params(desc, x, dt, A, Bm, Cm, Dskip, z, dt_bias, h_in);
  p.y = y;
  p.h_out = h_out;
  const ScanSpans n(desc, p);
  if ((st = check_apart({span(y, n.rows), span(h_out, n.state)}, n.in)) != MLSTM_OK) return st;
  if ((st = check_apart({span(y, n.rows), span(h_in != h_out ? h_out : nullptr, n.state)},
                        Spans{span(h_in, n.state)})) != MLSTM_OK)
    return st;
  return status(mlstm::launch_scan_step(p, static_cast<hipStream_t>(stream)));
}

int mlstm_dropout_validate(const mlstm_dropout_desc_t* desc) { return validate(desc); }

int mlstm_dropout(const mlstm_dropout_desc_t* desc, const void* x, const void* residual, const int64_t* seed_dev,
                  void* y, void* stream) {
  int st = validate(desc);
  if (st != MLSTM_OK) return st;
  if (desc->n == 0) return MLSTM_OK;
  if (any_null({x, y})) return MLSTM_E_NULLPTR;
  if ((st = check_aligned({x, residual, y}, size_of(desc->dtype))) != MLSTM_OK) return st;
  if ((st = check_aligned({seed_dev}, 8)) != MLSTM_OK) return st;
  const int64_t bytes = desc->n * (int64_t)size_of(desc->dtype);
  if ((st = check_apart({span(y, bytes)}, Spans{span(x != y ? x : nullptr, bytes), span(residual != y ? residual : nullptr, bytes),
                                                span(seed_dev, 16)})) != MLSTM_OK)
    return st;
  mlstm::DropoutParams p = {};
  p.x = x;
  p.residual = residual;
  p.seed_dev = seed_dev;
  p.y = y;
  p.n = desc->n;
  p.seed = (uint64_t)desc->seed;
  p.offset = (uint64_t)desc->offset;
  p.limit = (uint32_t)floor(desc->p * 4294967296.0);
  p.scale = (float)(1.0 / (1.0 - desc->p));
  p.bf16 = desc->dtype == MLSTM_BF16;
  return status(mlstm::launch_dropout(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
