// C ABI of the decoder-layer operators beside the linears: rotary positions, the norms around
// the residual add, attention. Argument checks and launch sequences; see include/qlora.h.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "../../include/qlora.h"
#include "attention.h"
#include "qlora_kernels.h"

using namespace qlora;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool bad_ptr(const void* p) { return p == nullptr || !aligned16(p); }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA; }

constexpr double kTwoPi = 6.28318530717958647693;

}  // namespace

extern "C" {

int qlora_rotary_init(const qlora_rotary_config* c, qlora_rotary* out) {
  if (c == nullptr || out == nullptr) return QLORA_ERR_INVALID;
  if (c->layout != QLORA_ROTARY_HALF && c->layout != QLORA_ROTARY_INTERLEAVED) return QLORA_ERR_INVALID;
  if (c->head_dim < 1 || c->rot_dim < 1 || c->rot_dim > c->head_dim) return QLORA_ERR_INVALID;
  if (!(c->base > 1.0) || !std::isfinite(c->base) || !std::isfinite(c->magnitude)) return QLORA_ERR_INVALID;
  const bool scaled = c->scaling != QLORA_ROTARY_SCALE_NONE;
  if (scaled && (!(c->factor > 0.0) || !std::isfinite(c->factor))) return QLORA_ERR_INVALID;
  const bool banded = c->scaling == QLORA_ROTARY_SCALE_BANDS || c->scaling == QLORA_ROTARY_SCALE_YARN;
  if (banded && (!(c->original_length > 0.0) || !std::isfinite(c->original_length) || !(c->low > 0.0) ||
                 !(c->high > c->low) || !std::isfinite(c->high)))
    return QLORA_ERR_INVALID;
  if (scaled && !banded && c->scaling != QLORA_ROTARY_SCALE_LINEAR) return QLORA_ERR_INVALID;
  if (c->head_dim % 8 != 0 || c->rot_dim % 8 != 0 || c->head_dim > 256) return QLORA_ERR_UNSUPPORTED;

  std::memset(out, 0, sizeof(*out));
  out->head_dim = c->head_dim;
  out->rot_dim = c->rot_dim;
  out->layout = c->layout;
  out->magnitude = static_cast<float>(c->magnitude);
  const int d = c->rot_dim;
  double lo = 0.0, hi = 0.0;
  if (c->scaling == QLORA_ROTARY_SCALE_YARN) {
    // the pairs that make `high` (fast) and `low` (slow) turns over the original length
    auto pair = [&](double turns) {
      return d * std::log(c->original_length / (turns * kTwoPi)) / (2.0 * std::log(c->base));
    };
    lo = std::max(std::floor(pair(c->high)), 0.0);
    hi = std::min(std::ceil(pair(c->low)), static_cast<double>(d - 1));
  }
  for (int i = 0; i < d / 2; ++i) {
    double f = std::pow(c->base, -2.0 * i / d);
    if (c->scaling == QLORA_ROTARY_SCALE_LINEAR) {
      f /= c->factor;
    } else if (c->scaling == QLORA_ROTARY_SCALE_BANDS) {
      const double turns = c->original_length * f / kTwoPi;
      const double keep = std::min(1.0, std::max(0.0, (turns - c->low) / (c->high - c->low)));
      f *= keep + (1.0 - keep) / c->factor;
    } else if (c->scaling == QLORA_ROTARY_SCALE_YARN) {
      const double ramp = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 1e-3)));
      f *= ramp / c->factor + (1.0 - ramp);
    }
    out->turns[i] = f / kTwoPi;
  }
  return QLORA_OK;
}

int qlora_rotary_apply(const qlora_rotary* rot, const int32_t* positions, int64_t m, const uint16_t* q, int64_t ld_q,
                       int32_t heads_q, uint16_t* q_out, int64_t ld_q_out, const uint16_t* k, int64_t ld_k,
                       int32_t heads_k, uint16_t* k_out, int64_t ld_k_out, int32_t transpose, qlora_stream_t stream) {
  if (rot == nullptr || m < 0 || heads_q < 1 || heads_k < 0) return QLORA_ERR_INVALID;
  if (m > 0 && (k == nullptr) != (heads_k == 0)) return QLORA_ERR_INVALID;
  if (rot->head_dim < 8 || rot->head_dim > 256 || rot->head_dim % 8 != 0 || rot->rot_dim < 8 ||
      rot->rot_dim > rot->head_dim || rot->rot_dim % 8 != 0)
    return QLORA_ERR_INVALID;
  if (rot->layout != QLORA_ROTARY_HALF && rot->layout != QLORA_ROTARY_INTERLEAVED) return QLORA_ERR_INVALID;
  const int64_t d = rot->head_dim;
  if (ld_q < heads_q * d || ld_q_out < heads_q * d) return QLORA_ERR_INVALID;
  if (heads_k > 0 && (ld_k < heads_k * d || ld_k_out < heads_k * d)) return QLORA_ERR_INVALID;
  if (m == 0) return QLORA_OK;
  if (bad_ptr(q) || bad_ptr(q_out) || positions == nullptr || (reinterpret_cast<uintptr_t>(positions) & 3u) != 0)
    return QLORA_ERR_INVALID;
  if (k != nullptr && (!aligned16(k) || bad_ptr(k_out))) return QLORA_ERR_INVALID;
  if (ld_q % 8 != 0 || ld_q_out % 8 != 0 || (k != nullptr && (ld_k % 8 != 0 || ld_k_out % 8 != 0)))
    return QLORA_ERR_UNSUPPORTED;
  if (m > INT32_MAX || heads_q > 32767 || heads_k > 32767) return QLORA_ERR_UNSUPPORTED;
  // in place means the same rows: the same address with another stride would be read after it is written
  if ((q == q_out && ld_q != ld_q_out) || (k != nullptr && k == k_out && ld_k != ld_k_out)) return QLORA_ERR_INVALID;
  RotaryParams p;
  std::memset(&p, 0, sizeof(p));
  p.positions = positions;
  p.m = m;
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.ld_q = ld_q;
  p.ld_k = ld_k;
  p.ld_q_out = ld_q_out;
  p.ld_k_out = ld_k_out;
  p.heads_q = heads_q;
  p.heads_k = heads_k;
  p.head_dim = rot->head_dim;
  p.rot_dim = rot->rot_dim;
  p.transpose = transpose != 0;
  p.magnitude = rot->magnitude;
  std::memcpy(p.turns, rot->turns, sizeof(p.turns));
  return cuda_status(launch_rotary(p, rot->layout == QLORA_ROTARY_INTERLEAVED, host_num_sms(),
                                   reinterpret_cast<cudaStream_t>(stream)));
}

// Shared checks of the two directions; *f32 receives the stream's type.
static int norm_shape_status(const qlora_norm* n, bool* f32) {
  if (n == nullptr || n->rows < 0 || n->cols < 1) return QLORA_ERR_INVALID;
  if (n->res_dtype != QLORA_DTYPE_BF16 && n->res_dtype != QLORA_DTYPE_FP32) return QLORA_ERR_INVALID;
  if (!(n->eps >= 0.f) || !std::isfinite(n->eps) || !std::isfinite(n->scale)) return QLORA_ERR_INVALID;
  if (n->cols % 8 != 0 || n->cols > kNormMaxCols || n->rows > INT32_MAX) return QLORA_ERR_UNSUPPORTED;
  *f32 = n->res_dtype == QLORA_DTYPE_FP32;
  return QLORA_OK;
}

int qlora_norm_residual_fwd(const qlora_norm* n, const void* x, const uint16_t* y, const float* w_post,
                            const float* gate, const float* w_pre, void* r, uint16_t* h, qlora_stream_t stream) {
  bool f32 = false;
  const int st = norm_shape_status(n, &f32);
  if (st != QLORA_OK) return st;
  if (n->rows == 0) return QLORA_OK;
  if ((w_pre == nullptr) != (h == nullptr) || (r == nullptr && h == nullptr)) return QLORA_ERR_INVALID;
  if (y == nullptr && (w_post != nullptr || gate != nullptr || r != nullptr)) return QLORA_ERR_INVALID;
  if (bad_ptr(x) || !aligned16(y) || !aligned16(w_post) || !aligned16(gate) || !aligned16(w_pre) || !aligned16(r) ||
      !aligned16(h))
    return QLORA_ERR_INVALID;
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.rows = n->rows;
  p.cols = n->cols;
  p.eps = n->eps;
  p.scale = n->scale;
  p.x = x;
  p.y = y;
  p.w_post = w_post;
  p.gate = gate;
  p.w_pre = w_pre;
  p.r = r;
  p.h = h;
  return cuda_status(launch_norm_fwd(p, f32, host_num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

size_t qlora_norm_residual_workspace_bytes(int64_t rows, int32_t cols) {
  if (rows < 1 || cols < 1 || cols % 8 != 0 || cols > kNormMaxCols) return 0;
  return static_cast<size_t>(norm_bwd_grid(rows, cols, host_num_sms())) * 2 * cols * 4;
}

int qlora_norm_residual_bwd(const qlora_norm* n, const void* dr, const uint16_t* dh, const void* r, const uint16_t* y,
                            const float* w_post, const float* gate, const float* w_pre, void* dx, uint16_t* dy,
                            float* dw_post, float* dgate, float* dw_pre, int32_t flags, void* ws, size_t ws_bytes,
                            qlora_stream_t stream) {
  bool f32 = false;
  const int sst = norm_shape_status(n, &f32);
  if (sst != QLORA_OK) return sst;
  if ((flags & ~QLORA_BWD_ACCUMULATE_GRADS) != 0) return QLORA_ERR_INVALID;
  if ((dw_post != nullptr && w_post == nullptr) || (dgate != nullptr && gate == nullptr) ||
      (dw_pre != nullptr && w_pre == nullptr))
    return QLORA_ERR_INVALID;
  if (!aligned16(dw_post) || !aligned16(dgate) || !aligned16(dw_pre)) return QLORA_ERR_INVALID;
  const bool weights = dw_post != nullptr || dgate != nullptr || dw_pre != nullptr;
  const bool accumulate = (flags & QLORA_BWD_ACCUMULATE_GRADS) != 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int sms = host_num_sms();
  const NormGradsParams grads{static_cast<const float*>(ws), norm_bwd_grid(n->rows, n->cols, sms), n->cols, n->scale,
                              w_post, gate, dw_post, dgate, dw_pre, accumulate ? 1 : 0};
  if (n->rows == 0)       // sums over no rows
    return weights && !accumulate ? cuda_status(launch_norm_grads(grads, st)) : QLORA_OK;
  if ((w_pre == nullptr) != (dh == nullptr) || (dh == nullptr && dr == nullptr)) return QLORA_ERR_INVALID;
  if (y == nullptr && (w_post != nullptr || gate != nullptr || dy != nullptr)) return QLORA_ERR_INVALID;
  if (bad_ptr(r) || bad_ptr(dx) || !aligned16(dr) || !aligned16(dh) || !aligned16(y) || !aligned16(w_post) ||
      !aligned16(gate) || !aligned16(w_pre) || !aligned16(dy))
    return QLORA_ERR_INVALID;
  if (weights && (bad_ptr(ws) || ws_bytes < qlora_norm_residual_workspace_bytes(n->rows, n->cols)))
    return QLORA_ERR_WORKSPACE;
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.rows = n->rows;
  p.cols = n->cols;
  p.eps = n->eps;
  p.scale = n->scale;
  p.x = r;
  p.dr = dr;
  p.dh = dh;
  p.y = y;
  p.w_post = w_post;
  p.gate = gate;
  p.w_pre = w_pre;
  p.dx = dx;
  p.dy = dy;
  p.part = weights ? static_cast<float*>(ws) : nullptr;
  const cudaError_t e = launch_norm_bwd(p, f32, sms, st);
  return cuda_status(e != cudaSuccess || !weights ? e : launch_norm_grads(grads, st));
}

// Checks of a call's sizes; fills the parameters that both directions share.
static int attention_params(const qlora_attention* a, AttnParams* p) {
  if (a == nullptr || a->batch < 1 || a->heads_q < 1 || a->heads_kv < 1 || a->head_dim < 1 || a->tokens_q < 0 ||
      a->tokens_k < 0 || a->window < 0)
    return QLORA_ERR_INVALID;
  if (a->heads_q % a->heads_kv != 0 || !(a->scale > 0.f) || !std::isfinite(a->scale)) return QLORA_ERR_INVALID;
  if (a->window > 0 && a->causal == 0) return QLORA_ERR_INVALID;
  if ((a->cu_q == nullptr) != (a->cu_k == nullptr)) return QLORA_ERR_INVALID;
  if (a->cu_q == nullptr && (a->tokens_q % a->batch != 0 || a->tokens_k % a->batch != 0)) return QLORA_ERR_INVALID;
  if (((reinterpret_cast<uintptr_t>(a->cu_q) | reinterpret_cast<uintptr_t>(a->cu_k)) & 3u) != 0)
    return QLORA_ERR_INVALID;
  const int64_t qw = static_cast<int64_t>(a->heads_q) * a->head_dim, kw = static_cast<int64_t>(a->heads_kv) * a->head_dim;
  if (a->ld_q < qw || a->ld_o < qw || a->ld_k < kw || a->ld_v < kw) return QLORA_ERR_INVALID;
  if (a->head_dim % 8 != 0 || a->head_dim > kAttnMaxHeadDim || a->heads_q / a->heads_kv > kAttnMaxGroup)
    return QLORA_ERR_UNSUPPORTED;
  if (((a->ld_q | a->ld_k | a->ld_v | a->ld_o) & 7) != 0) return QLORA_ERR_UNSUPPORTED;
  // 32-bit token indexes in the kernels (elements have 64), with room for a tile and a window past the end; the
  // tensor maps hold strides below 2^40 bytes
  constexpr int64_t kMost = int64_t(1) << 30;
  if (a->tokens_q > kMost || a->tokens_k > kMost || a->window > kMost) return QLORA_ERR_UNSUPPORTED;
  // A warp walks over the sequences, 32 at a time or, past empty ones, one by one, at 0.7 us a round trip, while others
  // wait for it, 2 s at most: a million one by one take 0.7 s.
  constexpr int32_t kMostSequences = 1 << 20;
  if (a->batch > kMostSequences) return QLORA_ERR_UNSUPPORTED;
  constexpr int64_t kMostLd = int64_t(1) << 38;
  if (a->ld_q > kMostLd || a->ld_k > kMostLd || a->ld_v > kMostLd || a->ld_o > kMostLd) return QLORA_ERR_UNSUPPORTED;
  const int64_t blocks = (std::max(a->tokens_q, a->tokens_k) + a->batch) * a->heads_kv * 16;
  if (blocks > INT32_MAX || a->tokens_q * a->heads_q / 16 >= INT32_MAX) return QLORA_ERR_UNSUPPORTED;
  std::memset(p, 0, sizeof(*p));
  p->batch = a->batch;
  p->heads_q = a->heads_q;
  p->heads_kv = a->heads_kv;
  p->group = a->heads_q / a->heads_kv;
  p->head_dim = a->head_dim;
  p->causal = a->causal != 0;
  p->window = a->window;
  p->scale = a->scale;
  p->scale_log2 = a->scale * 1.4426950408889634f;
  p->tokens_q = a->tokens_q;
  p->tokens_k = a->tokens_k;
  p->ld_q = a->ld_q;
  p->ld_k = a->ld_k;
  p->ld_v = a->ld_v;
  p->ld_o = a->ld_o;
  p->cu_q = a->cu_q;
  p->cu_k = a->cu_k;
  return QLORA_OK;
}

// Bytes of workspace of the forward for the checked sizes in p (a copy: the plan fills some of it).
static size_t attention_fwd_workspace(AttnParams p) {
  const size_t bytes = p.tokens_q == 0 ? 0 : attn_few_plan(p, host_num_sms());
  return bytes <= 1 ? 0 : bytes;
}

size_t qlora_attention_fwd_workspace_bytes(const qlora_attention* a) {
  AttnParams p;
  return attention_params(a, &p) == QLORA_OK ? attention_fwd_workspace(p) : 0;
}

int qlora_attention_fwd(const qlora_attention* a, const uint16_t* Q, const uint16_t* K, const uint16_t* V, uint16_t* O,
                        float* lse, void* ws, size_t ws_bytes, qlora_stream_t stream) {
  AttnParams p;
  const int st = attention_params(a, &p);
  if (st != QLORA_OK) return st;
  if (a->tokens_q == 0) return QLORA_OK;
  if (bad_ptr(Q) || bad_ptr(O) || !aligned16(lse)) return QLORA_ERR_INVALID;
  if (a->tokens_k > 0 ? (bad_ptr(K) || bad_ptr(V)) : (!aligned16(K) || !aligned16(V))) return QLORA_ERR_INVALID;
  const size_t need = attention_fwd_workspace(p);
  if (need > 0 && (bad_ptr(ws) || ws_bytes < need)) return QLORA_ERR_WORKSPACE;
  p.O = O;
  p.lse = lse;
  // without keys every row is empty: the maps point at something, and nothing is read through them
  if (a->tokens_k == 0) {
    K = V = Q;
    p.ld_k = p.ld_v = a->ld_q;
  }
  return cuda_status(launch_attn_fwd(p, Q, K, V, ws, host_num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

size_t qlora_attention_bwd_workspace_bytes(int64_t tokens_q, int32_t heads_q) {
  if (tokens_q < 0 || heads_q < 1) return 0;
  return align_up(static_cast<size_t>(tokens_q) * heads_q * 4, 16) + 16;      // delta, and the kernels' tile counters
}

int qlora_attention_bwd(const qlora_attention* a, const uint16_t* Q, const uint16_t* K, const uint16_t* V,
                        const uint16_t* O, const uint16_t* dO, const float* lse, uint16_t* dQ, uint16_t* dK,
                        uint16_t* dV, void* ws, size_t ws_bytes, qlora_stream_t stream) {
  AttnParams p;
  const int st = attention_params(a, &p);
  if (st != QLORA_OK) return st;
  // the kernels count the query rows that a key head meets in 32 bits, with room for a tile of 64 heads a token
  if (a->tokens_q * p.group > INT32_MAX - (128 << 6)) return QLORA_ERR_UNSUPPORTED;
  const bool q = a->tokens_q > 0, k = a->tokens_k > 0;
  if (!q && !k) return QLORA_OK;
  for (const void* t : {static_cast<const void*>(Q), static_cast<const void*>(O), static_cast<const void*>(dO),
                        static_cast<const void*>(lse), static_cast<const void*>(dQ)})
    if (q ? bad_ptr(t) : !aligned16(t)) return QLORA_ERR_INVALID;
  for (const void* t : {static_cast<const void*>(K), static_cast<const void*>(V), static_cast<const void*>(dK),
                        static_cast<const void*>(dV)})
    if (k ? bad_ptr(t) : !aligned16(t)) return QLORA_ERR_INVALID;
  const size_t need = qlora_attention_bwd_workspace_bytes(a->tokens_q, a->heads_q);
  if (bad_ptr(ws) || ws_bytes < need)
    return QLORA_ERR_WORKSPACE;
  p.O_in = O;
  p.dO = dO;
  p.lse_in = lse;
  p.dQ = dQ;
  p.dK = dK;
  p.dV = dV;
  // one side without tokens: the other's gradients are zero, and nothing is read through the maps
  if (!k) {
    K = V = Q;
    p.ld_k = p.ld_v = a->ld_q;
  }
  if (!q) {
    Q = K;
    p.dO = K;
    p.ld_q = p.ld_o = std::max(a->ld_k, static_cast<int64_t>(a->heads_q) * a->head_dim);
  }
  return cuda_status(launch_attn_bwd(p, Q, K, V, static_cast<float*>(ws),
                                     reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + need - 16), host_num_sms(),
                                     reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
