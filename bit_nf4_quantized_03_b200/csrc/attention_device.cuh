// What the attention kernels share (sm_100a): the problem's description, the decoding of a
// block's work from the sequences' offsets, and the few tcgen05 forms that only they use.
#pragma once

#include "attention.h"
#include "packed_f32.cuh"
#include "qlora_device.cuh"

namespace qlora {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Seq {
  int32_t q0, nq, k0, nk;   // first token and length, queries and keys
  int32_t off;              // query i stands at key i + off
};

// Offsets outside the tensors are clamped, so that no access follows a bad one.
__device__ __forceinline__ void seq_range(const int32_t* cu, int64_t tokens, int batch, int b, int32_t& start,
                                          int32_t& len) {
  if (cu == nullptr) {
    len = static_cast<int32_t>(tokens / batch);
    start = b * len;
    return;
  }
  const int32_t t = static_cast<int32_t>(tokens);
  const int32_t a = min(max(__ldg(cu + b), 0), t);
  const int32_t e = min(max(__ldg(cu + b + 1), a), t);
  start = a;
  len = e - a;
}

// Tile `idx` of the sequences' tiles in a row (`per` tokens each, of the keys or the queries):
// its sequence and its place there; false past the last one, and idx is then how far past. Whole
// warps call it; both offset arrays are read in one round trip.
template <bool kByKeys>
__device__ __forceinline__ bool find_tile(const AttnParams& p, int per, int64_t& idx, Seq& sq, int& t) {
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < p.batch; base += 32) {
    int32_t q0 = 0, nq = 0, k0 = 0, nk = 0;
    if (base + lane < p.batch) {
      seq_range(p.cu_q, p.tokens_q, p.batch, base + lane, q0, nq);
      seq_range(p.cu_k, p.tokens_k, p.batch, base + lane, k0, nk);
    }
    const int n = ((kByKeys ? nk : nq) + per - 1) / per;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, idx < sum);
    if (past != 0) {
      const int l = __ffs(past) - 1;
      t = static_cast<int>(idx) - (__shfl_sync(0xFFFFFFFFu, sum, l) - __shfl_sync(0xFFFFFFFFu, n, l));
      sq.q0 = __shfl_sync(0xFFFFFFFFu, q0, l);
      sq.nq = __shfl_sync(0xFFFFFFFFu, nq, l);
      sq.k0 = __shfl_sync(0xFFFFFFFFu, k0, l);
      sq.nk = __shfl_sync(0xFFFFFFFFu, nk, l);
      sq.off = sq.nk - sq.nq;
      return true;
    }
    idx -= __shfl_sync(0xFFFFFFFFu, sum, 31);
  }
  return false;
}

// Block index -> (tile, key head). Heads are walked in runs of head_run whose keys and values
// fit the L2 cache together; within a run tiles go from the last to the first when the last
// ones see the most keys (`down`), so that the longest blocks start first.
__device__ __forceinline__ void decode_block(const AttnParams& p, uint32_t blk, bool down, int64_t& tile, int& head) {
  const uint32_t tiles = static_cast<uint32_t>(p.tiles), run = static_cast<uint32_t>(p.head_run);
  const uint32_t which = blk / (tiles * run);
  const uint32_t in = blk - which * tiles * run;
  const uint32_t h0 = which * run;
  const uint32_t n = min(run, static_cast<uint32_t>(p.heads_kv) - h0);
  const uint32_t t = in / n;
  tile = down ? tiles - 1 - t : t;
  head = static_cast<int>(h0 + (in - t * n));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z) {
  if (!qlora_check(x >= 0 && (x & 7) == 0 && y >= 0 && z >= 0 && (smem_u32(smem_dst) & 15u) == 0, 120)) return;
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// One lane of the warp, chosen by hardware. The MMA warps of these kernels run their loops with
// all lanes and predicate only the issuing instructions: descriptors then stay in uniform
// registers, where an issuing thread alone in a branch took 1700 cycles for 16 MMAs (900 so).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// D (+)= A B^T, both operands in shared memory, issued by the lane with go != 0.
__device__ __forceinline__ void umma_bf16_if(uint32_t go, uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, g;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 g, %5, 0;\n\t"
      "@g tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(go)
      : "memory");
}
// The same with A in tensor memory: row i of A in lane i, two consecutive bf16 per column.
__device__ __forceinline__ void umma_bf16_ts_if(uint32_t go, uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, g;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 g, %5, 0;\n\t"
      "@g tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(go)
      : "memory");
}
__device__ __forceinline__ void umma_commit_if(uint32_t go, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred g;\n\tsetp.ne.b32 g, %1, 0;\n\t"
      "@g tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(go)
      : "memory");
}
// A value the whole warp agrees on, in a form the compiler knows to be uniform.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The larger of two, NaN if either is (fmaxf takes the other one then).
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Store kVecs 16-byte pieces of each lane's row (row: its address, null for a row that is not
// stored; pieces at or past `vecs` are not either). Four lanes trade pieces first, so that each
// store covers 64 contiguous bytes of eight rows: a lane storing its own row piece by piece
// touched 32 rows at a time, and a tile's end took 8100 cycles.
template <int kVecs>
__device__ __forceinline__ void store_rows(uint16_t* row, uint4 (&v)[kVecs], int vecs) {
  static_assert(kVecs % 4 == 0, "four lanes, four pieces");
  const int lane = threadIdx.x & 31;
  const bool odd1 = lane & 1, odd2 = lane & 2;
  const uint64_t mine = reinterpret_cast<uint64_t>(row);
  auto trade = [&](uint4& a, uint4& b, bool odd, int mask) {
    const uint4 send = odd ? a : b;
    uint4 got;
    got.x = __shfl_xor_sync(0xFFFFFFFFu, send.x, mask);
    got.y = __shfl_xor_sync(0xFFFFFFFFu, send.y, mask);
    got.z = __shfl_xor_sync(0xFFFFFFFFu, send.z, mask);
    got.w = __shfl_xor_sync(0xFFFFFFFFu, send.w, mask);
    if (odd) a = got;
    else b = got;
  };
#pragma unroll
  for (int c = 0; c < kVecs; c += 4) {
    trade(v[c], v[c + 1], odd1, 1);
    trade(v[c + 2], v[c + 3], odd1, 1);
    trade(v[c], v[c + 2], odd2, 2);
    trade(v[c + 1], v[c + 3], odd2, 2);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t* to = reinterpret_cast<uint16_t*>(__shfl_sync(0xFFFFFFFFu, mine, (lane & ~3) + i));
    if (to == nullptr) continue;
#pragma unroll
    for (int c = 0; c < kVecs; c += 4) {
      const int piece = c + (lane & 3);
      if (piece < vecs) *reinterpret_cast<uint4*>(to + piece * 8) = v[c + i];
    }
  }
}

// 2^a and 2^b without the special-function unit, whose 16 results a cycle would bound the softmax:
// x = n + f with n the nearest whole number (the addition of 1.5 * 2^23 leaves it in the low
// bits), 2^f by a polynomial of degree 4 interpolated at Chebyshev nodes on [-1/2, 1/2] (relative
// error 3.7e-6, a thousandth of the bf16 step the result is rounded to), times 2^n, whose bits are
// n's moved into the exponent. Below -126 the result is 2^-126. NaN stays NaN: the maximum keeps it
// and so does the product (n added to 2^f's own exponent bits would make a number of it).
__device__ __forceinline__ void ex2_poly(uint64_t x, float& a, float& b) {
  float x0, x1;
  unpair_f32(x, x0, x1);
  x = pair_f32(max_nan(x0, -126.0f), max_nan(x1, -126.0f));
  const uint64_t big = pair_f32(12582912.0f, 12582912.0f), unbig = pair_f32(-12582912.0f, -12582912.0f);
  const uint64_t minus = pair_f32(-1.0f, -1.0f);
  const uint64_t r = add_f32x2(x, big);
  const uint64_t f = fma_f32x2(add_f32x2(r, unbig), minus, x);
  uint64_t y = fma_f32x2(f, pair_f32(0.009676037356257439f, 0.009676037356257439f),
                         pair_f32(0.05592203512787819f, 0.05592203512787819f));
  y = fma_f32x2(y, f, pair_f32(0.2402210682630539f, 0.2402210682630539f));
  y = fma_f32x2(y, f, pair_f32(0.6931210160255432f, 0.6931210160255432f));
  y = fma_f32x2(y, f, pair_f32(1.0000001192092896f, 1.0000001192092896f));
  float r0, r1;
  unpair_f32(r, r0, r1);
  constexpr uint32_t kOne = 0x3F800000u;
  unpair_f32(mul_f32x2(y, pair_f32(__uint_as_float((__float_as_uint(r0) << 23) + kOne),
                                   __uint_as_float((__float_as_uint(r1) << 23) + kOne))), a, b);
}

// A ring's place and phase, moved on by `by` of `size` entries.
struct RingPos {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void move(int by, int size) {
    at += by;
    if (at >= size) {
      at -= size;
      phase ^= 1;
    }
  }
  __device__ __forceinline__ void skip(int by, int size) {
    const int to = at + by;
    phase ^= (to / size) & 1;
    at = to % size;
  }
};

// Zero one 128-byte row of every 64-column chunk of a swizzled tile (chunks `chunk_bytes`
// apart; a row's 16-byte pieces stay inside the row whatever the swizzle).
template <int kChunks>
__device__ __forceinline__ void zero_tile_row(uint8_t* tile, int row, int chunk_bytes) {
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    uint4* r = reinterpret_cast<uint4*>(tile + c * chunk_bytes + row * 128);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// One step of 64 keys of a row's softmax. S of the row stands in tensor memory at src (64 columns); P takes its place
// as bf16, the A operand of the product with V, rounded once (half a step, 2^-8 of each probability) because the tensor
// core takes it so. [clo, chi): the step's columns that the row sees. m_ref, l: the row's reference maximum and sum of
// exponentials, in 32 bits. The reference is raised only when the running maximum has outgrown it by a factor of 2^8 (the
// sum then stays within 32 bits' range by far); only then is the row's accumulator (t_o; none before the `first` step)
// read back and scaled, behind wait_o(), the end of the product that added to it last. Whole warps call it.
constexpr float kRescaleAt = 8.0f;      // log2 of the growth a row's reference maximum tolerates
constexpr int kFwdStep = 64;            // keys per step

template <int kHD, typename WaitO>
__device__ __forceinline__ bool softmax_step(uint32_t src, uint32_t t_o, float c, int clo, int chi, bool exists, bool first,
                                             float& m_ref, float& l, WaitO wait_o) {
  uint32_t x[2][32];
#pragma unroll
  for (int q = 0; q < 2; ++q) tmem_ld_32x32b_x32(src + q * 32, x[q]);
  tmem_ld_wait();
  if (__any_sync(0xFFFFFFFFu, clo > 0 || chi < kFwdStep)) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (q * 32 + e < clo || q * 32 + e >= chi) x[q][e] = 0xFF800000u;
  }
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < 32; e += 4)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      mx[q] = max3(mx[q], __uint_as_float(x[q & 1][e + (q & 2)]), __uint_as_float(x[q & 1][e + (q & 2) + 1]));
  const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  // (-inf) - (-inf) is NaN and compares false: a row that has seen nothing asks for nothing
  const bool grow = exists && (m - m_ref) * c > kRescaleAt;
  if (__any_sync(0xFFFFFFFFu, grow)) {
    const float f = grow ? ex2((m_ref - m) * c) : 1.0f;      // 0 for the first keys a row sees
    if (!first) {
      if (!wait_o()) return false;
      tc_fence_after();
#pragma unroll 1
      for (int q = 0; q < kHD / 16; ++q) {
        uint32_t o[16];
        tmem_ld_32x32b_x16(t_o + q * 16, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tmem_st_32x32b_x16(t_o + q * 16, o);
      }
    }
    l *= f;
    if (grow) m_ref = m;
  }
  const float shift = m_ref == -INFINITY ? 0.f : -m_ref * c;
  const uint64_t c2 = pair_f32(c, c), shift2 = pair_f32(shift, shift);
  uint64_t sum[2] = {0, 0};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float a, z;
      const uint64_t arg = fma_f32x2(pair_f32(__uint_as_float(x[q][e]), __uint_as_float(x[q][e + 1])), c2, shift2);
      unpair_f32(arg, a, z);
      a = ex2(a);
      z = ex2(z);
      sum[q] = add_f32x2(sum[q], pair_f32(a, z));
      pk[e / 2] = pack_bf16x2(a, z);
    }
    tmem_st_32x32b_x16(src + q * 16, pk);
  }
  float a, z;
  unpair_f32(add_f32x2(sum[0], sum[1]), a, z);
  l += a + z;
  tmem_st_wait();
  return true;
}

// The end of a row: O = accumulator / l (zero for a row that has seen nothing, whose l is 0), rounded once. out: the
// row's place, null for a row that does not exist. kTrade: full tiles, whose lanes trade pieces for wider stores.
template <int kHD, bool kTrade>
__device__ __forceinline__ void store_output(uint32_t t_o, float l, uint16_t* out, int head_dim) {
  const float inv = l != 0.f ? 1.0f / l : 0.f;
#pragma unroll
  for (int q = 0; q < kHD / 32; ++q) {
    uint32_t o[32];
    tmem_ld_32x32b_x32(t_o + q * 32, o);
    tmem_ld_wait();
    uint4 v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = l != 0.f ? __uint_as_float(o[x * 8 + e]) * inv : 0.f;
      v[x] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
    if (kTrade) {
      store_rows(out == nullptr ? nullptr : out + q * 32, v, min(4, head_dim / 8 - q * 4));
    } else if (out != nullptr) {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (q * 32 + x * 8 < head_dim) *reinterpret_cast<uint4*>(out + q * 32 + x * 8) = v[x];
    }
  }
}
__device__ __forceinline__ float row_lse(float m_ref, float l, float scale) {
  return l != 0.f ? m_ref * scale + logf(l) : -INFINITY;
}

// Keys that some query of `tokens` tokens from ta on sees: [lo, hi), 0, 0 if none.
__device__ __forceinline__ void visible_keys(const AttnParams& p, const Seq& sq, int ta, int tokens, int& lo, int& hi) {
  lo = p.window > 0 ? max(0, ta + sq.off - p.window + 1) : 0;
  hi = p.causal ? min(sq.nk, ta + tokens + sq.off) : sq.nk;
  if (tokens <= 0 || hi <= lo) lo = hi = 0;
}

}  // namespace qlora
