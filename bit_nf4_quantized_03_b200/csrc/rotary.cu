// Rotary positions of queries and keys (sm_100a), forward and backward.
//
// Pair i of a head (elements i and i + rot/2, or 2i and 2i + 1) is turned by the angle
// a = 2 pi pos turns[i]:  (u, v) -> mag (u cos a - v sin a, v cos a + u sin a); the
// backward pass is the transposed map, the same with -a.
//
// The angle is formed in 64 bits: pos * turns[i], less its nearest whole number, is exact
// to 2^-53 of the position's turns, where a 32-bit angle at position 10^5 would already be
// off by 2^-8 radians. What remains lies in [-1/2, 1/2] and goes to sincospi in 32 bits.
// Values are turned in 32 bits and rounded to bf16 once.
//
// Bound by HBM: 4 bytes per element, read and written once. 4096 tokens of 64 heads of 128 (134 MB) take 30 us (4.5 TB/s)
// behind a gigabyte of writes that has to leave the L2 cache first, and 20 back to back, where part of the data is still
// there (so above the copy's rate). The times in launch_rotary are back to back. A thread owns kPairs pairs of one token
// and walks over a run of heads, so the 64-bit product and the sine are paid once per run (launch_rotary chooses its
// length) and the loads of four heads are in flight at a time.
#include <algorithm>

#include "qlora_kernels.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float2 unpack(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// kPairs pairs as two runs of kPairs elements: (u ..., v ...) for the half layout, or
// (u v u v ...) over both runs for the interleaved one.
template <int kPairs>
struct Run;
template <>
struct Run<8> {
  using Vec = uint4;
};
template <>
struct Run<4> {
  using Vec = uint2;
};

// Heads a thread has in flight: their loads are issued before the first is turned and stored (the
// outputs may be the inputs, so the compiler could not move a load over a store itself).
constexpr int kBatch = 4;

template <int kPairs, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 3) rotary_kernel(const __grid_constant__ RotaryParams p) {
  griddep_enter();
  using Vec = typename Run<kPairs>::Vec;
  constexpr int kWords = kPairs / 2;
  const int groups = p.turn_groups + p.copy_groups;
  const int per_block = kThreads / groups;
  const int local = static_cast<int>(threadIdx.x) / groups;
  const int grp = static_cast<int>(threadIdx.x) - local * groups;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * per_block + local;
  if (local >= per_block || tok >= p.m) return;
  // runs of heads: first those of q, then those of k
  const int runs_q = (p.heads_q + p.heads_per_run - 1) / p.heads_per_run;
  const bool of_q = static_cast<int>(blockIdx.y) < runs_q;
  const int h0 = (of_q ? blockIdx.y : blockIdx.y - runs_q) * p.heads_per_run;
  const int n = min(p.heads_per_run, (of_q ? p.heads_q : p.heads_k) - h0);
  const int64_t first = static_cast<int64_t>(h0) * p.head_dim;
  const uint16_t* src = (of_q ? p.q + tok * p.ld_q : p.k + tok * p.ld_k) + first;
  uint16_t* dst = (of_q ? p.q_out + tok * p.ld_q_out : p.k_out + tok * p.ld_k_out) + first;

  if (grp >= p.turn_groups) {
    // the part of a head that is not turned: 16 elements per thread at most, skipped in place
    if (src == dst) return;
    const int e = p.rot_dim + (grp - p.turn_groups) * 16;
    const bool two = e + 8 < p.head_dim;
    for (int h = 0; h < n; h += kBatch) {
      uint4 a[kBatch], b[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (h + u < n) {
          a[u] = __ldcs(reinterpret_cast<const uint4*>(src + (h + u) * p.head_dim + e));
          if (two) b[u] = __ldcs(reinterpret_cast<const uint4*>(src + (h + u) * p.head_dim + e + 8));
        }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (h + u < n) {
          *reinterpret_cast<uint4*>(dst + (h + u) * p.head_dim + e) = a[u];
          if (two) *reinterpret_cast<uint4*>(dst + (h + u) * p.head_dim + e + 8) = b[u];
        }
    }
    return;
  }

  union Words {
    Vec v;
    uint32_t w[kWords];
  };
  const int e0 = kInterleaved ? grp * 2 * kPairs : grp * kPairs;
  const int e1 = kInterleaved ? e0 + kPairs : e0 + p.rot_dim / 2;
  Words a[kBatch], b[kBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (h + u < n) {
        a[u].v = __ldcs(reinterpret_cast<const Vec*>(src + (h + u) * p.head_dim + e0));
        b[u].v = __ldcs(reinterpret_cast<const Vec*>(src + (h + u) * p.head_dim + e1));
      }
  };
  load(0);                       // on their way while the angles are formed
  float c[kPairs], s[kPairs];
  const double pos = static_cast<double>(__ldg(p.positions + tok));
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const double t = pos * p.turns[grp * kPairs + i];
    float sn, cs;
    sincospif(static_cast<float>(2.0 * (t - rint(t))), &sn, &cs);
    c[i] = cs * p.magnitude;
    s[i] = p.transpose ? -sn * p.magnitude : sn * p.magnitude;
  }
  for (int h = 0; h < n; h += kBatch) {
    if (h > 0) load(h);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (h + u >= n) continue;
      Words ya, yb;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const float2 x = unpack(a[u].w[i]), z = unpack(b[u].w[i]);
        if (kInterleaved) {
          const int j = i + kWords;
          ya.w[i] = pack_bf16x2(x.x * c[i] - x.y * s[i], x.y * c[i] + x.x * s[i]);
          yb.w[i] = pack_bf16x2(z.x * c[j] - z.y * s[j], z.y * c[j] + z.x * s[j]);
        } else {
          const int j = 2 * i;
          ya.w[i] = pack_bf16x2(x.x * c[j] - z.x * s[j], x.y * c[j + 1] - z.y * s[j + 1]);
          yb.w[i] = pack_bf16x2(z.x * c[j] + x.x * s[j], z.y * c[j + 1] + x.y * s[j + 1]);
        }
      }
      *reinterpret_cast<Vec*>(dst + (h + u) * p.head_dim + e0) = ya.v;
      *reinterpret_cast<Vec*>(dst + (h + u) * p.head_dim + e1) = yb.v;
    }
  }
}

}  // namespace

cudaError_t launch_rotary(RotaryParams p, bool interleaved, int num_sms, cudaStream_t st) {
  // 8 pairs per thread (two 16-byte runs) where they tile the rotated part, else 4 (256 tokens of 64 heads, one a thread:
  // 5.1 us with 8, 7.1 with 4; 4096: 19.9 and 20.5)
  const int pairs = (p.rot_dim % 16 == 0) ? 8 : 4;
  p.turn_groups = p.rot_dim / (2 * pairs);
  const bool in_place = p.q == p.q_out && (p.heads_k == 0 || p.k == p.k_out);
  p.copy_groups = in_place ? 0 : (p.head_dim - p.rot_dim + 15) / 16;
  const int groups = p.turn_groups + p.copy_groups;
  const int per_block = kThreads / groups;
  const int64_t blocks = (p.m + per_block - 1) / per_block;
  // Heads per thread: 8 where that leaves a third of the SMs a block (256 tokens of 64 heads: 3.7 us, with one head 5.1;
  // 4096: 20 and 51), else fewer; a run of one head pays the angle for each head, which is what a few tokens need to
  // spread out (16 tokens: 2.2 us, with 8 heads 2.9).
  const int64_t want = num_sms / 3;
  auto runs = [&](int run) { return (p.heads_q + run - 1) / run + (p.heads_k + run - 1) / run; };
  int run = 8;
  while (run > 1 && blocks * runs(run) < want) run /= 2;
  p.heads_per_run = run;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(runs(run)));
  auto go = [&](auto kernel) { return launch_pdl_grid(kernel, grid, kThreads, 0, st, 1, p); };
  if (pairs == 8) return interleaved ? go(rotary_kernel<8, true>) : go(rotary_kernel<8, false>);
  return interleaved ? go(rotary_kernel<4, true>) : go(rotary_kernel<4, false>);
}

}  // namespace qlora
