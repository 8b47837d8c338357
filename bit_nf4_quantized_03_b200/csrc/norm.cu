// Root-mean-square norms around a residual add (sm_100a): the norm after a block, its gate
// and residual scale, the add, and the norm before the next block, in one pass per direction.
//
//   t = y eta w_post, eta = rsqrt(mean(y^2) + eps)      (t = y without w_post)
//   r = x + s g t                                       (g = 1 without gate)
//   h = r rho w_pre, rho = rsqrt(mean(r^2) + eps)
//
// Backward, with dr what reaches r from later blocks, u = dh w_pre, n = y eta (y without w_post)
// and m = s g w_post, one vector for all three:
//   d = dr + rho u - r rho^3 mean(u r)       = dx        dw_pre  = sum_rows dh r rho
//   e = m d;  dy = eta (e - n mean(e n))                 (dy = e without w_post)
//   a = s sum_rows d n:  dgate = w_post a, dw_post = g a (one column sum for both)
//
// All of it in 32 bits; r, h, dx and dy are rounded to their type once, and h is formed from
// the unrounded r. The backward recomputes eta and rho from the r and y it reads anyway, so
// nothing but r and y is kept between the two directions.
//
// Bound by HBM: 8 bytes per element forward (bf16 stream), 12 backward (8192 x 8192, back to back: 91 us, 5.9 TB/s, and
// 158 us with all weight gradients, 5.1 TB/s). Many rows: persistent
// blocks, whose rows arrive by bulk copies into a ring of shared memory, so that the next rows'
// loads run while a row's sums make the block wait; the weight vectors sit in shared memory too
// (read from L2 for every row, they cost the backward half its time). Few rows: a block per row.
#include <algorithm>

#include "packed_f32.cuh"
#include "qlora_kernels.h"

namespace qlora {
namespace {

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void load_f8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
// eight elements of a residual-stream row (bf16 or fp32), element offset e
template <bool kF32>
__device__ __forceinline__ void load_res(const void* p, int64_t e, float (&f)[8]) {
  if (kF32) load_f8(static_cast<const float*>(p) + e, f);
  else unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e), f);
}
template <bool kF32>
__device__ __forceinline__ void store_res(void* p, int64_t e, const float (&f)[8]) {
  if (kF32) {
    float* o = static_cast<float*>(p) + e;
    __stcs(reinterpret_cast<float4*>(o), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(o + 4), make_float4(f[4], f[5], f[6], f[7]));
  } else {
    __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + e), pack8(f));
  }
}

// The threads that share a row: a block, or one of several groups of it (barrier `id`, not 0).
struct RowGroup {
  int tid, threads, id;
  __device__ __forceinline__ void sync() const { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
};

// Sums of N values over the group, in every thread, in a fixed order. `buf`: N * 32 floats
// that no earlier sum of the same row uses (one barrier per sum).
template <int N>
__device__ __forceinline__ void row_sum(const RowGroup& g, float (&v)[N], float* buf) {
  const int warp = g.tid >> 5, lane = threadIdx.x & 31, warps = g.threads >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i * 32 + warp] = v[i];
  g.sync();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (lane < warps) ? buf[i * 32 + lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
}

// One row per block; a thread keeps its 8 * kVec elements in registers between the sums.
template <bool kF32, int kVec>
__global__ void norm_fwd_kernel(const __grid_constant__ NormParams p) {
  griddep_enter();
  __shared__ float buf[64];
  const RowGroup grp{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), 1};
  const int64_t base = static_cast<int64_t>(blockIdx.x) * p.cols;
  const float inv = 1.0f / static_cast<float>(p.cols);
  float r[kVec][8];
  uint4 y[kVec];
  const int nvec = p.cols / 8;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < nvec) {
      load_res<kF32>(p.x, base + v * 8, r[i]);
      if (p.y != nullptr) y[i] = __ldcs(reinterpret_cast<const uint4*>(p.y + base) + v);
    }
  }
  if (p.y != nullptr) {
    float eta = 1.0f;
    if (p.w_post != nullptr) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (threadIdx.x + i * blockDim.x < nvec) {
          float t[8];
          unpack8(y[i], t);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[0] += t[j] * t[j];
        }
      row_sum(grp, s, buf);
      eta = rsqrtf(s[0] * inv + p.eps);
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        float t[8], w[8];
        unpack8(y[i], t);
        if (p.w_post != nullptr) {
          load_f8(p.w_post + v * 8, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) t[j] *= eta * w[j];
        }
        if (p.gate != nullptr) {
          load_f8(p.gate + v * 8, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) t[j] *= w[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] += p.scale * t[j];
        if (p.r != nullptr) store_res<kF32>(p.r, base + v * 8, r[i]);
      }
    }
  }
  if (p.w_pre == nullptr) return;
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    if (threadIdx.x + i * blockDim.x < nvec)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += r[i][j] * r[i][j];
  row_sum(grp, s, buf + 32);
  const float rho = rsqrtf(s[0] * inv + p.eps);
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < nvec) {
      float w[8];
      load_f8(p.w_pre + v * 8, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] *= r[i][j] * rho;
      __stcs(reinterpret_cast<uint4*>(p.h + base) + v, pack8(w));
    }
  }
}

// A group's ring of rows in shared memory, fed by bulk copies of up to four inputs. The group's
// thread 0 feeds it. A wait that gives up (2 s) leaves `alive` false: the group then goes on
// through its barriers without waiting or storing, so that every thread reaches every barrier.
constexpr int kMaxStages = 4;
constexpr int kMaxGroups = 8;

struct RowRing {
  const uint8_t* src[4];     // null: not part of the call
  uint32_t bytes[4];         // of one row
  uint32_t stage_bytes;
  uint8_t* base;
  uint64_t* full;
  int stages;
  int64_t row, stride, rows; // the group's current row, the step to its next, all rows
  int s;
  uint32_t phase;
  bool feeds, alive;

  __device__ __forceinline__ void fetch(int64_t r, int stage) const {
    uint8_t* dst = base + stage * stage_bytes;
    mbar_arrive_expect_tx(&full[stage], stage_bytes);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (src[i] != nullptr) {
        bulk_load(dst, src[i] + r * bytes[i], bytes[i], &full[stage]);
        dst += bytes[i];
      }
  }
  __device__ __forceinline__ void start() const {
    if (feeds)
      for (int i = 0; i < stages; ++i)
        if (row + i * stride < rows) fetch(row + i * stride, i);
  }
  __device__ __forceinline__ const uint8_t* wait() {
    alive = alive && mbar_wait(&full[s], phase);
    return base + s * stage_bytes;
  }
  // behind a barrier after which nobody reads the current row any more
  __device__ __forceinline__ void refill() const {
    if (feeds && alive && row + stages * stride < rows) fetch(row + stages * stride, s);
  }
  // behind a barrier after which nobody reads the row before any more
  __device__ __forceinline__ void refill_before(bool first) const {
    if (feeds && alive && !first && row + (stages - 1) * stride < rows)
      fetch(row + (stages - 1) * stride, s == 0 ? stages - 1 : s - 1);
  }
  __device__ __forceinline__ void advance() {
    row += stride;
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
};

// Copies a weight vector to shared memory (kShared) in two planes: the first and the second half of
// every eight values, so that a warp's 16-byte reads meet no bank twice (side by side they did, for
// a third of the kernels' shared-memory time). Returns where it is read from.
template <bool kShared>
__device__ __forceinline__ const float* stage_weights(const float* w, int cols, uint8_t*& to) {
  if (!kShared || w == nullptr) return w;
  const int nvec = cols / 8;
  const float* r = reinterpret_cast<const float*>(to);
  for (int i = threadIdx.x; i < nvec * 2; i += blockDim.x)
    reinterpret_cast<float4*>(to)[(i & 1) * nvec + (i >> 1)] = __ldg(reinterpret_cast<const float4*>(w) + i);
  to += static_cast<size_t>(cols) * 4;
  return r;
}

// m = scale * gate * w_post, as above, when it is kept in shared memory and not a constant.
__device__ __forceinline__ const float* stage_mix(const float* gate, const float* w_post, float scale, int cols,
                                                  uint8_t*& to) {
  if (gate == nullptr && w_post == nullptr) return nullptr;
  const int nvec = cols / 8;
  const float* r = reinterpret_cast<const float*>(to);
  for (int i = threadIdx.x; i < nvec * 2; i += blockDim.x) {
    float4 m = make_float4(scale, scale, scale, scale);
    for (const float* w : {gate, w_post})
      if (w != nullptr) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(w) + i);
        m = make_float4(m.x * f.x, m.y * f.y, m.z * f.z, m.w * f.w);
      }
    reinterpret_cast<float4*>(to)[(i & 1) * nvec + (i >> 1)] = m;
  }
  to += static_cast<size_t>(cols) * 4;
  return r;
}

// Four pairs of a row, from bf16 or fp32 in shared memory.
template <bool kF32>
__device__ __forceinline__ void load_pairs(const uint8_t* row, int v, uint64_t (&x)[4]) {
  if (kF32) {
    const ulonglong2 a = reinterpret_cast<const ulonglong2*>(row)[2 * v], b = reinterpret_cast<const ulonglong2*>(row)[2 * v + 1];
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  } else {
    const uint4 w = reinterpret_cast<const uint4*>(row)[v];
    x[0] = pair_bf16(w.x); x[1] = pair_bf16(w.y); x[2] = pair_bf16(w.z); x[3] = pair_bf16(w.w);
  }
}
template <bool kShared>
__device__ __forceinline__ void load_weights(const float* w, int v, int nvec, uint64_t (&x)[4]) {
  const ulonglong2* p = reinterpret_cast<const ulonglong2*>(w) + (kShared ? v : 2 * v);
  const ulonglong2 a = p[0], b = p[kShared ? nvec : 1];
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
template <bool kShared>
__device__ __forceinline__ void load_mix(const NormParams& p, const float* mix, int v, int nvec, uint64_t scale,
                                         uint64_t (&x)[4]) {
  if (kShared && mix != nullptr) {
    load_weights<true>(mix, v, nvec, x);
    return;
  }
  x[0] = x[1] = x[2] = x[3] = scale;
  if (kShared) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float* w = k == 0 ? p.gate : p.w_post;
    if (w == nullptr) continue;
    uint64_t f[4];
    load_weights<false>(w, v, nvec, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = mul_f32x2(x[j], f[j]);
  }
}
__device__ __forceinline__ uint4 pack_pairs(const uint64_t (&x)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpair_f32(x[i], f[2 * i], f[2 * i + 1]);
  return pack8(f);
}
template <bool kF32>
__device__ __forceinline__ void store_pairs(void* p, int64_t e, const uint64_t (&x)[4]) {
  if (kF32) {
    float* o = static_cast<float*>(p) + e;
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpair_f32(x[i], f[2 * i], f[2 * i + 1]);
    __stcs(reinterpret_cast<float4*>(o), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(o + 4), make_float4(f[4], f[5], f[6], f[7]));
  } else {
    __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + e), pack_pairs(x));
  }
}
__device__ __forceinline__ float sum_pair(uint64_t x) {
  float a, b;
  unpair_f32(x, a, b);
  return a + b;
}
__device__ __forceinline__ uint64_t both(float x) { return pair_f32(x, x); }

// Four vectors of eight per thread; several groups of threads share a block, each with rows of its
// own, so that one group's loads and sums run under the others' arithmetic.
template <bool kF32>
__global__ void __launch_bounds__(768) norm_fwd_ring_kernel(const __grid_constant__ NormParams p, int threads,
                                                            int stages) {
  constexpr int kVec = 4;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float bufs[kMaxGroups][2][64];   // by the row's parity: a late warp still reads the row before's
  __shared__ uint64_t full[kMaxGroups][kMaxStages];
  const int nvec = p.cols / 8, group = static_cast<int>(threadIdx.x) / threads;
  const int groups = static_cast<int>(blockDim.x) / threads;
  const RowGroup grp{static_cast<int>(threadIdx.x) - group * threads, threads, 1 + group};
  const int tid = grp.tid;
  float(&buf)[2][64] = bufs[group];
  RowRing ring{};
  ring.src[0] = static_cast<const uint8_t*>(p.x);
  ring.src[1] = reinterpret_cast<const uint8_t*>(p.y);
  ring.bytes[0] = static_cast<uint32_t>(p.cols) * (kF32 ? 4 : 2);
  ring.bytes[1] = static_cast<uint32_t>(p.cols) * 2;
  ring.stage_bytes = ring.bytes[0] + (p.y != nullptr ? ring.bytes[1] : 0);
  ring.full = full[group];
  ring.stages = stages;
  ring.row = static_cast<int64_t>(group) * gridDim.x + blockIdx.x;
  ring.stride = static_cast<int64_t>(groups) * gridDim.x;
  ring.rows = p.rows;
  ring.feeds = tid == 0;
  ring.alive = true;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&ring.full[s], 1);
    fence_mbar_init();
  }
  griddep_enter();
  uint8_t* at = smem;
  const float* mix = stage_mix(p.gate, p.w_post, p.scale, p.cols, at);
  const float* w_pre = stage_weights<true>(p.w_pre, p.cols, at);
  ring.base = at + static_cast<size_t>(group) * stages * ring.stage_bytes;
  __syncthreads();
  ring.start();
  const uint64_t scale2 = both(p.scale);
  const float inv = 1.0f / static_cast<float>(p.cols);
  for (int it = 0; ring.row < p.rows; ++it, ring.advance()) {
    const uint8_t* st = ring.wait();
    const uint8_t* st_y = st + ring.bytes[0];
    const int64_t base = ring.row * p.cols;
    uint64_t r[kVec][4];
    float eta = 1.0f;
    if (p.w_post != nullptr) {
      uint64_t acc = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int v = tid + i * threads;
        if (v < nvec) {
          load_pairs<false>(st_y, v, r[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc = fma_f32x2(r[i][j], r[i][j], acc);
        }
      }
      float sum[1] = {sum_pair(acc)};
      row_sum(grp, sum, buf[it & 1]);
      eta = rsqrtf(sum[0] * inv + p.eps);
    }
    const uint64_t eta2 = both(eta);
    uint64_t acc = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = tid + i * threads;
      if (v < nvec) {
        load_pairs<kF32>(st, v, r[i]);
        if (p.y != nullptr) {
          uint64_t t[4], m[4];
          load_pairs<false>(st_y, v, t);
          load_mix<true>(p, mix, v, nvec, scale2, m);
#pragma unroll
          for (int j = 0; j < 4; ++j) r[i][j] = fma_f32x2(mul_f32x2(t[j], eta2), m[j], r[i][j]);
          if (p.r != nullptr && ring.alive) store_pairs<kF32>(p.r, base + v * 8, r[i]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = fma_f32x2(r[i][j], r[i][j], acc);
      }
    }
    float sum[1] = {sum_pair(acc)};
    row_sum(grp, sum, buf[it & 1] + 32);
    ring.refill();
    if (w_pre != nullptr) {
      const uint64_t rho2 = both(rsqrtf(sum[0] * inv + p.eps));
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int v = tid + i * threads;
        if (v < nvec) {
          uint64_t w[4];
          load_weights<true>(w_pre, v, nvec, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = mul_f32x2(mul_f32x2(r[i][j], rho2), w[j]);
          if (ring.alive) __stcs(reinterpret_cast<uint4*>(p.h + base) + v, pack_pairs(w));
        }
      }
    }
  }
}

// Backward. With weight gradients (kGrads) the column sums stay in registers over a block's rows, one
// partial per block at the end (norm_grads_kernel adds them in a fixed order: the same bits on
// every call); their registers leave room for one group of threads per block. A frozen norm's
// backward has the forward's several.
template <bool kF32, int kVec, bool kGrads, bool kShared>
__global__ void __launch_bounds__(kGrads ? 512 : 768, kGrads && kVec == 1 ? 2 : 1)
    norm_bwd_kernel(const __grid_constant__ NormParams p, int threads, int stages) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kGroups = kGrads ? 1 : kMaxGroups;
  __shared__ float bufs[kGroups][2][128];     // by the row's parity: a late warp still reads the row before's
  __shared__ uint64_t full[kGroups][kMaxStages];
  const int nvec = p.cols / 8, group = kGrads ? 0 : static_cast<int>(threadIdx.x) / threads;
  const int groups = kGrads ? 1 : static_cast<int>(blockDim.x) / threads;
  const RowGroup grp{static_cast<int>(threadIdx.x) - group * threads, threads, 1 + group};
  const int tid = grp.tid;
  float(&buf)[2][128] = bufs[group];
  const uint32_t res_bytes = static_cast<uint32_t>(p.cols) * (kF32 ? 4 : 2), bf_bytes = static_cast<uint32_t>(p.cols) * 2;
  RowRing ring{};
  ring.src[0] = static_cast<const uint8_t*>(p.x);
  ring.src[1] = static_cast<const uint8_t*>(p.dr);
  ring.src[2] = reinterpret_cast<const uint8_t*>(p.dh);
  ring.src[3] = reinterpret_cast<const uint8_t*>(p.y);
  ring.bytes[0] = ring.bytes[1] = res_bytes;
  ring.bytes[2] = ring.bytes[3] = bf_bytes;
  const uint32_t off_dr = res_bytes;
  const uint32_t off_dh = off_dr + (p.dr != nullptr ? res_bytes : 0);
  const uint32_t off_y = off_dh + (p.dh != nullptr ? bf_bytes : 0);
  ring.stage_bytes = off_y + (p.y != nullptr ? bf_bytes : 0);
  ring.full = full[group];
  ring.stages = stages;
  ring.row = static_cast<int64_t>(group) * gridDim.x + blockIdx.x;
  ring.stride = static_cast<int64_t>(groups) * gridDim.x;
  ring.rows = p.rows;
  ring.feeds = tid == 0;
  ring.alive = true;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&ring.full[s], 1);
    fence_mbar_init();
  }
  griddep_enter();
  uint8_t* at = smem;
  const float* mix = kShared ? stage_mix(p.gate, p.w_post, p.scale, p.cols, at) : nullptr;
  const float* w_pre = stage_weights<kShared>(p.w_pre, p.cols, at);
  ring.base = at + static_cast<size_t>(group) * stages * ring.stage_bytes;
  __syncthreads();
  ring.start();

  uint64_t g_mix[kVec][4], g_pre[kVec][4];
#pragma unroll
  for (int i = 0; i < kVec; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) g_mix[i][j] = g_pre[i][j] = 0;
  const uint64_t scale2 = both(p.scale);
  const float inv = 1.0f / static_cast<float>(p.cols);
  for (int it = 0; ring.row < p.rows; ++it, ring.advance()) {
    const uint8_t* st = ring.wait();
    uint64_t s_rr = 0, s_ur = 0, s_yy = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = tid + i * threads;
      if (v < nvec) {
        if (p.dh != nullptr) {
          uint64_t r[4], u[4], w[4];
          load_pairs<kF32>(st, v, r);
          load_pairs<false>(st + off_dh, v, u);
          load_weights<kShared>(w_pre, v, nvec, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s_rr = fma_f32x2(r[j], r[j], s_rr);
            s_ur = fma_f32x2(mul_f32x2(u[j], w[j]), r[j], s_ur);
          }
        }
        if (p.w_post != nullptr) {
          uint64_t y[4];
          load_pairs<false>(st + off_y, v, y);
#pragma unroll
          for (int j = 0; j < 4; ++j) s_yy = fma_f32x2(y[j], y[j], s_yy);
        }
      }
    }
    float sum[3] = {sum_pair(s_rr), sum_pair(s_ur), sum_pair(s_yy)};
    row_sum(grp, sum, buf[it & 1]);
    if (stages > 1) ring.refill_before(it == 0);
    const float rho = rsqrtf(sum[0] * inv + p.eps);
    const float eta = (p.w_post != nullptr) ? rsqrtf(sum[2] * inv + p.eps) : 1.0f;
    const uint64_t rho2 = both(rho), c_r = both(-rho * rho * rho * (sum[1] * inv)), eta2 = both(eta);
    uint64_t e[kVec][4];
    uint64_t s_en = 0;
    const int64_t base = ring.row * p.cols;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = tid + i * threads;
      if (v < nvec) {
        uint64_t(&d)[4] = e[i];
        if (p.dr != nullptr) load_pairs<kF32>(st + off_dr, v, d);
        else d[0] = d[1] = d[2] = d[3] = 0;
        if (p.dh != nullptr) {
          uint64_t r[4], u[4], w[4];
          load_pairs<kF32>(st, v, r);
          load_pairs<false>(st + off_dh, v, u);
          load_weights<kShared>(w_pre, v, nvec, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t ru = mul_f32x2(u[j], rho2);
            d[j] = fma_f32x2(r[j], c_r, fma_f32x2(ru, w[j], d[j]));
            if (kGrads) g_pre[i][j] = fma_f32x2(ru, r[j], g_pre[i][j]);
          }
        }
        if (ring.alive) store_pairs<kF32>(p.dx, base + v * 8, d);
        if (p.y != nullptr) {
          uint64_t y[4], m[4];
          load_pairs<false>(st + off_y, v, y);
          load_mix<kShared>(p, mix, v, nvec, scale2, m);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t n = mul_f32x2(y[j], eta2);
            if (kGrads) g_mix[i][j] = fma_f32x2(d[j], n, g_mix[i][j]);
            d[j] = mul_f32x2(d[j], m[j]);
            s_en = fma_f32x2(d[j], n, s_en);
          }
        }
      }
    }
    if (p.dy != nullptr) {
      float dot[1] = {sum_pair(s_en)};
      if (p.w_post != nullptr) row_sum(grp, dot, buf[it & 1] + 96);
      const uint64_t c_y = both(-eta * eta * (dot[0] * inv));
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int v = tid + i * threads;
        if (v < nvec) {
          if (p.w_post != nullptr) {
            uint64_t y[4];
            load_pairs<false>(st + off_y, v, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) e[i][j] = fma_f32x2(y[j], c_y, mul_f32x2(e[i][j], eta2));
          }
          if (ring.alive) __stcs(reinterpret_cast<uint4*>(p.dy + base) + v, pack_pairs(e[i]));
        }
      }
    }
    if (stages == 1) {
      grp.sync();
      ring.refill();
    }
  }
  if (kGrads) {
    float* out = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.cols;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = tid + i * threads;
      if (v < nvec) {
        store_pairs<true>(out, v * 8, g_mix[i]);
        store_pairs<true>(out + p.cols, v * 8, g_pre[i]);
      }
    }
  }
}

// The weight gradients from the blocks' column sums part[block][a, dw_pre][c]: 32 columns per
// block, eight runs of partials each, joined in order.
__global__ void __launch_bounds__(256) norm_grads_kernel(const __grid_constant__ NormGradsParams p) {
  griddep_enter();
  __shared__ float buf[8][33];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int c = static_cast<int>(blockIdx.x) * 32 + lane;
  const int which = blockIdx.y;
  if (which == 0 ? (p.dw_post == nullptr && p.dgate == nullptr) : p.dw_pre == nullptr) return;
  float s = 0.f;
  if (c < p.cols) {
#pragma unroll 8
    for (int i = run; i < p.parts; i += 8) s += __ldcg(p.part + (static_cast<int64_t>(i) * 2 + which) * p.cols + c);
  }
  buf[run][lane] = s;
  __syncthreads();
  if (run != 0 || c >= p.cols) return;
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) t += buf[i][lane];
  auto put = [&](float* out, float x) { out[c] = p.accumulate ? out[c] + x : x; };
  if (which == 1) {
    put(p.dw_pre, t);
    return;
  }
  t *= p.scale;
  if (p.dgate != nullptr) put(p.dgate, p.w_post != nullptr ? t * p.w_post[c] : t);
  if (p.dw_post != nullptr) put(p.dw_post, p.gate != nullptr ? t * p.gate[c] : t);
}

int round32(int x) { return (x + 31) / 32 * 32; }

// With weight gradients, vectors of eight per thread, at most 512 threads: 16 column sums per vector live in registers.
int grads_vec(int cols) { return cols <= 4096 ? 1 : cols <= 8192 ? 2 : 4; }
int threads_of(int cols, int vec) { return round32((cols / 8 + vec - 1) / vec); }

// A block of the persistent kernels: `groups` groups of `threads` threads, each with a ring of `stages` rows, `per_sm`
// blocks on an SM; the weight vectors in shared memory if they leave every group two rows, or one where there are several
// groups or where without them no more would fit. The rule was measured on the bf16 stream. An fp32 stream's rows are longer
// and it serves them less well: of the copy's rate, 8192 rows back to back, 2048 and 4096 columns 85 and 87% with one frozen
// norm and 61 and 65% with both norms' gradients; 8192 columns, whose weights it leaves in L2, 96% with the pre-norm's
// gradient, 64 with both norms', and 67 and 46% frozen (one norm, both), where a block has one group of 8 warps.
constexpr size_t kSmemMost = 232448;
constexpr size_t smem_static(int groups) { return 512 + static_cast<size_t>(groups > 1 ? kMaxGroups : 1) * 1088; }
struct RingPlan {
  int threads, groups, per_sm, stages;
  bool shared;
  size_t bytes, most;      // of dynamic shared memory: of this launch, and what the kernel may ever have
};

RingPlan ring_plan(const NormParams& p, size_t stage, int threads, int groups, int per_sm, bool grads = false) {
  const size_t fixed = smem_static(grads ? 1 : kMaxGroups);
  const size_t weights = static_cast<size_t>(p.cols) * 4 *
                         ((p.w_post != nullptr || p.gate != nullptr ? 1 : 0) + (p.w_pre != nullptr ? 1 : 0));
  // 228 KB per SM, 1 KB of it reserved per block, and the kernels' static shared memory
  const size_t share = std::min<size_t>(kSmemMost, 233472 / per_sm - 1024) - fixed;
  RingPlan r{threads, groups, per_sm, 0, false, 0, kSmemMost - fixed};
  // as many groups as have room for a row each
  while (r.groups > 1 && share < weights + stage * r.groups) --r.groups;
  const size_t with = share > weights ? (share - weights) / (stage * r.groups) : 0, without = share / (stage * r.groups);
  r.shared = with >= 2 || (with >= 1 && (without < 2 || r.groups > 1));
  r.stages = static_cast<int>(std::min<size_t>(kMaxStages, r.shared ? with : without));
  r.bytes = r.stages * stage * r.groups + (r.shared ? weights : 0);
  return r;
}

template <typename K>
cudaError_t launch_ring(K kernel, const NormParams& p, const RingPlan& r, int num_sms, cudaStream_t st) {
  // the same limit whatever the size: calls on two host threads may set it at once
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(r.most));
  if (e != cudaSuccess) return e;
  const int64_t blocks = (p.rows + r.groups - 1) / r.groups;
  const int grid = static_cast<int>(std::min<int64_t>(blocks, static_cast<int64_t>(num_sms) * r.per_sm));
  return launch_pdl(kernel, grid, r.threads * r.groups, r.bytes, st, 1, p, r.threads, r.stages);
}

template <bool kGrads, bool kF32>
cudaError_t launch_bwd(const NormParams& p, int vec, const RingPlan& r, int num_sms, cudaStream_t st) {
  if (r.shared) {
    if (vec == 1) return launch_ring(norm_bwd_kernel<kF32, 1, kGrads, true>, p, r, num_sms, st);
    if (vec == 2) return launch_ring(norm_bwd_kernel<kF32, 2, kGrads, true>, p, r, num_sms, st);
    return launch_ring(norm_bwd_kernel<kF32, 4, kGrads, true>, p, r, num_sms, st);
  }
  // rows too long for the weights beside two of them; a frozen norm's are only above 6144 columns
  if constexpr (kGrads) {
    if (vec == 1) return launch_ring(norm_bwd_kernel<kF32, 1, kGrads, false>, p, r, num_sms, st);
    if (vec == 2) return launch_ring(norm_bwd_kernel<kF32, 2, kGrads, false>, p, r, num_sms, st);
  }
  if (vec != 4) return cudaErrorInvalidConfiguration;
  return launch_ring(norm_bwd_kernel<kF32, 4, kGrads, false>, p, r, num_sms, st);
}

int grads_per_sm(int cols) {
  return std::max(1, std::min(8, (grads_vec(cols) == 1 ? 1024 : 512) / threads_of(cols, grads_vec(cols))));
}

}  // namespace

cudaError_t launch_norm_fwd(const NormParams& p, bool f32, int num_sms, cudaStream_t st) {
  const int nvec = p.cols / 8;
  // Many rows: persistent blocks, where each of at least two groups finds room for a row, from a row per group on (8192 x
  // 8192: 94 us, a block per row 110; 1500 x 4096: 9.0 and 9.9; 600 x 4096: 5.7 and 4.8).
  const int threads = threads_of(p.cols, 4);
  const size_t stage = static_cast<size_t>(p.cols) * ((f32 ? 4 : 2) + (p.y != nullptr ? 2 : 0));
  const RingPlan ring = ring_plan(p, stage, threads, std::min(kMaxGroups, 768 / threads), 1);
  if (ring.shared && ring.stages >= 1 && ring.groups >= 2 && p.rows >= static_cast<int64_t>(num_sms) * ring.groups)
    return f32 ? launch_ring(norm_fwd_ring_kernel<true>, p, ring, num_sms, st)
               : launch_ring(norm_fwd_ring_kernel<false>, p, ring, num_sms, st);
  // Otherwise a block per row, with as many threads as the row has vectors, for the shortest chain (16 x 8192: 2.7 us, with
  // four vectors per thread 3.8; 600 x 4096: 4.8 and 5.5).
  const int vec = nvec <= 1024 ? 1 : 2;
  const dim3 grid(static_cast<unsigned>(p.rows));
  auto go = [&](auto kernel) { return launch_pdl_grid(kernel, grid, threads_of(p.cols, vec), 0, st, 1, p); };
  if (f32) return vec == 1 ? go(norm_fwd_kernel<true, 1>) : go(norm_fwd_kernel<true, 2>);
  return vec == 1 ? go(norm_fwd_kernel<false, 1>) : go(norm_fwd_kernel<false, 2>);
}

int norm_bwd_grid(int64_t rows, int32_t cols, int num_sms) {
  return static_cast<int>(std::min<int64_t>(rows, static_cast<int64_t>(num_sms) * grads_per_sm(cols)));
}

cudaError_t launch_norm_bwd(const NormParams& p, bool f32, int num_sms, cudaStream_t st) {
  const int res = f32 ? 4 : 2;
  const size_t stage = static_cast<size_t>(p.cols) *
                       (res + (p.dr != nullptr ? res : 0) + (p.dh != nullptr ? 2 : 0) + (p.y != nullptr ? 2 : 0));
  if (p.part == nullptr) {
    // frozen: two vectors per thread, as many groups as 768 threads hold (4096 x 4096, bf16: 35 us, with one vector 44), four
    // above 6144 columns, where two would leave room for one group. Few rows: one vector, as with weight gradients up to
    // 4096 columns, whose sums are then in the same order (16 x 4096: 3.4 us either way, 296 x 4096 4.9 and 4.5).
    const int vec = p.rows <= 2 * num_sms && p.cols <= 6144 ? 1 : p.cols <= 6144 ? 2 : 4;
    const int threads = threads_of(p.cols, vec);
    const int wanted = static_cast<int>(std::min<int64_t>(kMaxGroups, (p.rows + num_sms - 1) / num_sms));
    const RingPlan ring = ring_plan(p, stage, threads, std::min(wanted, 768 / threads), 1);
    if (ring.stages < 1) return cudaErrorInvalidConfiguration;
    return f32 ? launch_bwd<false, true>(p, vec, ring, num_sms, st) : launch_bwd<false, false>(p, vec, ring, num_sms, st);
  }
  const int vec = grads_vec(p.cols);
  const RingPlan ring = ring_plan(p, stage, threads_of(p.cols, vec), 1, grads_per_sm(p.cols), true);
  if (ring.stages < 1) return cudaErrorInvalidConfiguration;
  return f32 ? launch_bwd<true, true>(p, vec, ring, num_sms, st) : launch_bwd<true, false>(p, vec, ring, num_sms, st);
}

cudaError_t launch_norm_grads(const NormGradsParams& p, cudaStream_t st) {
  return launch_pdl_grid(norm_grads_kernel, dim3(static_cast<unsigned>((p.cols + 31) / 32), 2), 256, 0, st, 1, p);
}

}  // namespace qlora
