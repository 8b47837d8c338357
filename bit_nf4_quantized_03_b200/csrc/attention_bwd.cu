// Softmax attention, backward (sm_100a): the probabilities are recomputed from lse.
//   P = exp(scale Q K^T - lse),  dP = dO V^T,  dS = P * (dP - delta),  delta = rowsum(dO * O)
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
//
// Two kernels from one template, each with one operand pair resident and the other streamed:
//   keys    128 keys of a key head stay (K, V), 128 query rows a step stream by (Q, dO):
//           S^T = K Q^T, dP^T = V dO^T;  dV += P^T dO, dK += dS^T Q
//   queries 128 query rows stay (Q, dO), 128 keys a step stream by (K, V):
//           S = Q K^T, dP = dO V^T;  dQ += dS K
// Every gradient is summed in tensor memory by the one block that owns it, in a fixed order,
// and rounded once: no atomics, no 32-bit dQ in memory, the same bits on every call; the price
// is S and dP a second time, 7 products instead of 5. A tile's P and dS go back to tensor
// memory as bf16 and are the A operand of the second products, so they never touch shared
// memory. Query heads of a shared key head are rows of the same tile (AttnParams), so their sum
// costs nothing.
//
// A step's products are 128 wide: 64-wide ones (M = 128, both operands in shared memory) took as
// long each, 1560 cycles a step of 64 where the queries' kernel now takes less for 128.
//
// A block: 16 warps exponentiate and form dS (a thread owns a row of the resident tile and a
// quarter of a step's columns), one warp issues the MMAs, one feeds the tiles by TMA, one brings
// lse and delta of the streamed rows, one finds the next tile's place. The tensor core and the
// 16 warps work on alternate halves of a step: keys: dV of a step and S of the next while dS is
// formed, dK and the next dP while the next S is exponentiated; queries: S is two steps ahead
// (two buffers; dS goes back over S, so that dP's columns are free as soon as they are read).
// Measured (heads of 128): 4 x 2048 tokens, 64 heads, causal 990 us a call by itself at 1.97 GHz, 1169 back to back for a
// second, where the power cap leaves 1.52. Back to back, 8192 tokens, 16 heads: causal 941 us (1.57 GHz), not causal 1681
// (1.49 GHz; 1145 TFLOP/s of the 7 products). Tensor pipe 54 to 57% busy, issue 47%: the 16 warps' two phases of a step wait
// for one another's products. The keys' kernel spills 12 bytes at its 96 registers.
// Blocks are persistent, so that a tile's loads and first products run under the end of the tile
// before. (As a block per tile, 16,000 of a tile's 47,000 cycles were its beginning and its end.)
#include <algorithm>
#include <climits>
#include <cstring>

#include "attention_device.cuh"
#include "qlora_kernels.h"

namespace qlora {
namespace {

constexpr int kStep = 128;            // streamed rows per step
constexpr int kMathWarps = 16;
// Of four exponentials, those by polynomial (back to back, 4 causal sequences of 2048 tokens, 64 heads of 128: 1175 us with
// none, 1169 with one, 1196 with two, 1244 with three; 8192 tokens of 32 heads: 1864, 1829, 1895, 1971).
constexpr int kPolyOf4 = 1;
constexpr int kBwdThreads = (kMathWarps + 4) * 32;

template <int kHD, bool kKeys>
struct BwdCfg {
  static constexpr int kChunks = kHD / 64;
  static constexpr int kTileBytes = 128 * kHD * 2;         // a resident or streamed tile
  // rings of the streamed tiles: first (Q or K: read by S and, last, by the gradient) and second (dO or V). The
  // queries' kernel reads V once, long before the next is due, but K from two steps ahead to the gradient.
  static constexpr int kRing1 = kHD == 128 ? (kKeys ? 2 : 3) : 4;
  static constexpr int kRing2 = kHD == 128 ? (kKeys ? 2 : 1) : (kKeys ? 4 : 2);
  // tensor memory: the gradients from column 0 (dV, dK or dQ), S in one or two buffers, dP
  static constexpr int kBufs = kKeys ? 1 : 2;
  static constexpr int kColS = kKeys ? 256 : 128;
  static constexpr int kColDp = 384;
  static constexpr int kStatBytes = kRing1 * 2 * kStep * 4;
  static constexpr int kSmem = (2 + kRing1 + kRing2) * kTileBytes + kStatBytes + 1024 + 512;
  static_assert((kKeys ? 2 : 1) * kHD <= kColS && kColS + kBufs * kStep <= kColDp, "tensor memory");
  static_assert(kSmem <= 232448 - 256, "shared memory budget");
};

// What a block has to know about a tile.
struct BwdWork {
  Seq sq;
  int32_t live;          // 0: no more tiles
  int32_t head;          // key head
  int32_t ta, tokens;    // resident tokens of the sequence
  int32_t s0;            // first streamed token
  int32_t n;             // steps
};

// mbar_wait for the warp that hands out tiles, two ahead: the others may be at a tile of `steps` steps all the while. A
// step takes about 2 us, so a tile of a million takes as long as any other wait may (2 s): 20 us a step on top.
__device__ __forceinline__ bool wait_for_a_tile(uint64_t* bar, uint32_t parity, int steps) {
  const uint32_t at = smem_u32(bar);
  if (mbar_try_wait(at, parity)) return true;
  const uint64_t t0 = globaltimer_ns(), limit = kWaitLimitNs + static_cast<uint64_t>(steps) * 20000u;
  uint32_t tries = 0;
  while (true) {
    if (mbar_try_wait_suspend(at, parity, kSuspendHintNs)) return true;
    if ((++tries & 15u) == 0 && globaltimer_ns() - t0 > limit) {
      atomicCAS(&g_device_error, kErrNone, kErrWaitTimeout);
      return false;
    }
  }
}

template <int kHD, bool kKeys>
__global__ void __launch_bounds__(kBwdThreads, 1)
    attn_bwd_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnMaps maps) {
  using C = BwdCfg<kHD, kKeys>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* sRes = smem;                                     // K, V or Q, dO
  uint8_t* sOne = smem + 2 * C::kTileBytes;                 // ring of Q or K
  uint8_t* sTwo = sOne + C::kRing1 * C::kTileBytes;         // ring of dO or V
  float* sStat = reinterpret_cast<float*>(sTwo + C::kRing2 * C::kTileBytes);   // ring of -(lse, delta), kKeys only
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sStat) + C::kStatBytes);
  uint64_t* res_full = bars;                  // resident pair
  uint64_t* res_empty = bars + 1;             // no product reads it any more
  uint64_t* acc_full = bars + 2;              // a tile's gradients are complete
  uint64_t* acc_empty = bars + 3;             // and read
  uint64_t* work_full = bars + 4;             // [2]
  uint64_t* work_empty = bars + 6;            // [2]
  uint64_t* s_full = bars + 8;                // [kBufs] S of a step
  uint64_t* p_full = bars + 10;               // P of a step is back (kKeys)
  uint64_t* dp_full = bars + 11;              // dP of a step
  uint64_t* ds_full = bars + 12;              // dS of a step is back
  uint64_t* one_full = bars + 13;             // [kRing1]
  uint64_t* one_empty = one_full + C::kRing1;
  uint64_t* two_full = one_empty + C::kRing1; // [kRing2]
  uint64_t* two_empty = two_full + C::kRing2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(two_empty + C::kRing2);
  __shared__ BwdWork work[2];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int per_res = kKeys ? 128 : 128 / p.group;          // tokens per resident tile
  const int per_str = kKeys ? kStep / p.group : kStep;      // tokens per step
  const int str_rows = kKeys ? per_str * p.group : kStep;   // rows of a step that a load writes
  if (threadIdx.x == 0) {
    mbar_init(res_full, 1);
    mbar_init(res_empty, 1);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, kMathWarps);
    mbar_init(p_full, kMathWarps);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, kMathWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&work_full[i], 1);
      mbar_init(&work_empty[i], kMathWarps + (kKeys ? 3 : 2));
    }
    for (int i = 0; i < C::kBufs; ++i) mbar_init(&s_full[i], 1);
    for (int i = 0; i < C::kRing1; ++i) {
      mbar_init(&one_full[i], kKeys ? 2 : 1);      // the TMA's and, with statistics, that warp's
      mbar_init(&one_empty[i], 1);
    }
    for (int i = 0; i < C::kRing2; ++i) {
      mbar_init(&two_full[i], 1);
      mbar_init(&two_empty[i], 1);
    }
    fence_mbar_init();
  }
  if constexpr (kKeys) {
    // rows of a step that no load writes are rows of the reduction: zero once
    const int gap = kStep - str_rows;
    for (int x = threadIdx.x; x < (C::kRing1 + C::kRing2) * gap; x += kBwdThreads)
      zero_tile_row<C::kChunks>(sOne + (x / gap) * C::kTileBytes, str_rows + x % gap, kStep * 128);
    fence_proxy_async_smem();
  }
  if (warp == kMathWarps) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // The queries' kernel reads nothing that the keys' kernel writes, and its blocks start only once every block of that
  // one is past its own wait, that is, behind delta. So they fill the SMs that the last tiles of the keys leave, and
  // wait for that grid at their end (without keys there is none: then delta is the grid before).
  if (kKeys || p.tokens_k == 0) griddep_wait();
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // every role but the scheduler walks over the tiles with this: false after the last one
  RingPos wk;
  auto take = [&](BwdWork& w) {
    if (!mbar_wait(&work_full[wk.at], wk.phase)) return false;
    w = work[wk.at];
    __syncwarp();
    if (lane == 0) mbar_arrive(&work_empty[wk.at]);
    wk.move(1, 2);
    return w.live != 0;
  };

  if (warp == kMathWarps + 3) {
    // ------------------------------------------------------------ scheduler
    const int64_t items = static_cast<int64_t>(p.tiles) * p.heads_kv;
    // Tiles there are at most, and exactly once a search has gone past the last one. Later items there are passed over
    // without another search: with tens of thousands of sequences one takes half a millisecond, and the others, whose
    // wait for a tile has a limit, gave up behind thousands of them.
    int64_t tiles = p.tiles;
    RingPos at;
    int published = 0;
    int n[3] = {0, 0, 0};            // steps of the last three tiles handed out, the oldest first
    bool ok = true;
    // Tiles are handed out longest first, one counter for all blocks: which block sums a tile changes nothing in it.
    // (Dealt out beforehand, causal sequences left a sixth of the time to the unlucky blocks.)
    while (ok) {
      uint32_t got = 0;
      if (lane == 0) got = atomicAdd(p.counter, 1u);
      const int64_t item = __shfl_sync(0xFFFFFFFFu, got, 0);
      const bool last = item >= items;
      BwdWork w;
      w.live = 0;
      if (!last) {
        int64_t tile;
        int t = 0;
        decode_block(p, static_cast<uint32_t>(item), !kKeys && p.causal != 0, tile, w.head);
        const int64_t which = tile;
        if (which >= tiles) {
          // there are a few items more than tiles
        } else if (!find_tile<kKeys>(p, per_res, tile, w.sq, t)) {
          tiles = which - tile;
        } else {
          w.live = 1;
          w.ta = t * per_res;
          w.tokens = min(per_res, (kKeys ? w.sq.nk : w.sq.nq) - w.ta);
          int s1;
          if (kKeys) {        // queries that see some key of [ta, ta + tokens)
            w.s0 = p.causal ? max(0, w.ta - w.sq.off) : 0;
            s1 = p.window > 0 ? min(w.sq.nq, w.ta + w.tokens - 1 - w.sq.off + p.window) : w.sq.nq;
          } else {            // keys that some query of [ta, ta + tokens) sees
            w.s0 = p.window > 0 ? max(0, w.ta + w.sq.off - p.window + 1) : 0;
            s1 = p.causal ? min(w.sq.nk, w.ta + w.tokens + w.sq.off) : w.sq.nk;
          }
          w.n = s1 > w.s0 ? (s1 - w.s0 + per_str - 1) / per_str : 0;
        }
      }
      if (w.live == 0 && !last) continue;
      // the place is free once every role has taken n[1]'s tile, behind the end of n[0]'s
      if (published >= 2) ok = wait_for_a_tile(&work_empty[at.at], at.phase ^ 1, n[0]);
      if (!ok) break;
      if (lane == 0) {
        work[at.at] = w;
        mbar_arrive(&work_full[at.at]);
      }
      if (last) break;
      at.move(1, 2);
      ++published;
      n[0] = n[1];
      n[1] = n[2];
      n[2] = w.n;
    }
  } else if (warp == kMathWarps + 1) {
    // ------------------------------------------------------------ TMA producer
    const CUtensorMap* m0 = kKeys ? &maps.k : &maps.q;
    const CUtensorMap* m1 = kKeys ? &maps.v : &maps.dO;
    const CUtensorMap* n0 = kKeys ? &maps.q : &maps.k;
    const CUtensorMap* n1 = kKeys ? &maps.dO : &maps.v;
    if (lane == 0) {
      tma_prefetch_desc(m0);
      tma_prefetch_desc(m1);
      tma_prefetch_desc(n0);
      tma_prefetch_desc(n1);
    }
    const int res_rows = kKeys ? 128 : per_res * p.group;
    BwdWork w;
    RingPos one, two;
    uint32_t res_phase = 1;          // the first wait finds the memory free
    int steps = 0;
    bool ok = true;
    while (ok && take(w)) {
      if (w.n == 0) continue;
      const int res_head = kKeys ? w.head : w.head * p.group, str_head = kKeys ? w.head * p.group : w.head;
      const int res_tok = (kKeys ? w.sq.k0 : w.sq.q0) + w.ta, str_tok = (kKeys ? w.sq.q0 : w.sq.k0) + w.s0;
      auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int hd, int tok) {
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c) tma_load_3d(dst + c * 16384, map, bar, c * 64, hd, tok);
      };
      ok = mbar_wait(res_empty, res_phase);
      res_phase ^= 1;
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(res_full, static_cast<uint32_t>(res_rows) * 128 * C::kChunks * 2);
        load(sRes, m0, res_full, res_head, res_tok);
        load(sRes + C::kTileBytes, m1, res_full, res_head, res_tok);
      }
      for (int j = 0; j < w.n; ++j) {
        const uint32_t bytes = static_cast<uint32_t>(str_rows) * 128 * C::kChunks;
        ok = mbar_wait(&one_empty[one.at], one.phase ^ 1);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&one_full[one.at], bytes);
          load(sOne + one.at * C::kTileBytes, n0, &one_full[one.at], str_head, str_tok + j * per_str);
        }
        one.move(1, C::kRing1);
        ok = mbar_wait(&two_empty[two.at], two.phase ^ 1);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&two_full[two.at], bytes);
          load(sTwo + two.at * C::kTileBytes, n1, &two_full[two.at], str_head, str_tok + j * per_str);
        }
        two.move(1, C::kRing2);
        ++steps;
      }
    }
    // the MMAs' last releases have landed before the block ends: the release of every slot's last use, if it had one
    auto drain = [&](RingPos at, int size, uint64_t* empty) {
      for (int i = 0; ok && i < size; ++i) {
        if (steps >= size || at.at < steps) ok = mbar_wait(&empty[at.at], steps >= size ? at.phase ^ 1 : 0);
        at.move(1, size);
      }
    };
    drain(one, C::kRing1, one_empty);
    drain(two, C::kRing2, two_empty);
    if (ok && steps > 0) mbar_wait(res_empty, res_phase);
  } else if (warp == kMathWarps + 2) {
    // ------------------------------------------------------------ statistics of the streamed rows
    if (kKeys) {
      // requested kAhead steps before they are stored: waiting for each step's in turn, with their way from memory,
      // held the whole block to one step per 2000 cycles
      constexpr int kAhead = 2;
      BwdWork w;
      RingPos str;
      bool ok = true;
      while (ok && take(w)) {
        float lse[kAhead][4], delta[kAhead][4];
        const float* base_l = p.lse_in + static_cast<int64_t>(w.sq.q0) * p.heads_q + w.head * p.group;
        const float* base_d = p.delta + static_cast<int64_t>(w.sq.q0) * p.heads_q + w.head * p.group;
        int tok_of[4], head_of[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          tok_of[h] = w.s0 + (h * 32 + lane) / p.group;
          head_of[h] = (h * 32 + lane) % p.group;
        }
        auto request = [&](int j, float (&l)[4], float (&d)[4]) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int tok = tok_of[h] + j * per_str;
            l[h] = -INFINITY;                             // exp2(S - inf) = 0: no row here
            d[h] = 0.f;
            if (j < w.n && h * 32 + lane < str_rows && tok < w.sq.nq) {
              const int64_t at = static_cast<int64_t>(tok) * p.heads_q + head_of[h];
              l[h] = -__ldg(base_l + at);
              d[h] = -__ldg(base_d + at);
            }
          }
        };
#pragma unroll
        for (int u = 0; u < kAhead; ++u) request(u, lse[u], delta[u]);
        for (int j0 = 0; j0 < w.n && ok; j0 += kAhead) {
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            if (j0 + u >= w.n || !ok) break;
            ok = mbar_wait(&one_empty[str.at], str.phase ^ 1);
            if (!ok) break;
            float* st = sStat + str.at * 2 * kStep;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              st[h * 32 + lane] = lse[u][h] * kLog2e;
              st[kStep + h * 32 + lane] = delta[u][h];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&one_full[str.at]);
            str.move(1, C::kRing1);
            request(j0 + u + kAhead, lse[u], delta[u]);
          }
        }
      }
    }
  } else if (warp == kMathWarps) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = umma_idesc_bf16(kStep, false, false);
    constexpr uint32_t idesc_g = umma_idesc_bf16(kHD, false, true);
    constexpr uint32_t kTile = C::kTileBytes >> 4;
    const uint32_t go = elect_one();
    const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
    const uint64_t d_res = umma_desc_sw128(smem_u32(sRes), 16, 1024);
    const uint64_t d_one = umma_desc_sw128(smem_u32(sOne), 16, 1024);                // as B of S
    const uint64_t d_two = umma_desc_sw128(smem_u32(sTwo), 16, 1024);                // as B of dP
    const uint64_t r_one = umma_desc_sw128(smem_u32(sOne), kStep * 128, 1024);       // as B of dK or dQ
    const uint64_t r_two = umma_desc_sw128(smem_u32(sTwo), kStep * 128, 1024);       // as B of dV
    BwdWork w;
    // places in the rings of the next S, dP, dV and dK (or dQ); S buffers of the next S and the next dQ
    RingPos s_one, dp_two, g_two, g_one, s_buf, g_buf;
    uint32_t res_phase = 0, acc_phase = 1, p_phase = 0, ds_phase = 0;
    bool ok = true;
    auto product = [&](uint32_t dst, uint64_t a, uint64_t b) {
#pragma unroll
      for (int kk = 0; kk < kHD / 16; ++kk) {
        const uint32_t o = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
        umma_bf16_if(go, dst, a + o, b + o, idesc_s, kk > 0 ? 1u : 0u);
      }
    };
    auto gradient = [&](uint32_t dst, uint32_t a, uint64_t b, bool first) {
#pragma unroll
      for (int kk = 0; kk < kStep / 16; ++kk)      // each quarter of a step packs into the start of its own columns
        umma_bf16_ts_if(go, dst, a + (kk >> 1) * 32 + (kk & 1) * 8, b + (kk * 2048 >> 4), idesc_g,
                        (first && kk == 0) ? 0u : 1u);
    };
    auto issue_s = [&]() {
      ok = ok && mbar_wait(&one_full[s_one.at], s_one.phase);
      if (!ok) return;
      tc_fence_after();
      product(tm + C::kColS + s_buf.at * kStep, d_res, d_one + static_cast<uint32_t>(s_one.at * kTile));
      umma_commit_if(go, &s_full[s_buf.at]);
      s_one.move(1, C::kRing1);
      s_buf.move(1, C::kBufs);
    };
    auto issue_dp = [&](bool last) {
      ok = ok && mbar_wait(&two_full[dp_two.at], dp_two.phase);
      if (!ok) return;
      tc_fence_after();
      product(tm + C::kColDp, d_res + kTile, d_two + static_cast<uint32_t>(dp_two.at * kTile));
      umma_commit_if(go, dp_full);
      if (!kKeys) umma_commit_if(go, &two_empty[dp_two.at]);
      if (last) umma_commit_if(go, res_empty);      // S of the last step is issued before its dP
      dp_two.move(1, C::kRing2);
    };
    while (ok && take(w)) {
      const int n = uniform(w.n);
      if (n == 0) continue;
      ok = mbar_wait(res_full, res_phase);
      res_phase ^= 1;
      issue_s();
      if (!kKeys && n > 1) {
        issue_dp(false);
        issue_s();
      } else {
        issue_dp(n == 1);
      }
      for (int j = 0; j < n && ok; ++j) {
        if (j == 0) {
          ok = mbar_wait(acc_empty, acc_phase);
          acc_phase ^= 1;
        }
        if (kKeys) {
          ok = ok && mbar_wait(p_full, p_phase);
          p_phase ^= 1;
          if (!ok) break;
          tc_fence_after();
          gradient(tm, tm + C::kColS, r_two + static_cast<uint32_t>(g_two.at * kTile), j == 0);
          umma_commit_if(go, &two_empty[g_two.at]);
          g_two.move(1, C::kRing2);
          if (j + 1 < n) issue_s();
        }
        ok = ok && mbar_wait(ds_full, ds_phase);
        ds_phase ^= 1;
        if (!ok) break;
        tc_fence_after();
        if (!kKeys && j + 1 < n) issue_dp(j + 2 == n);
        if (!ok) break;
        gradient(tm + (kKeys ? kHD : 0), tm + (kKeys ? C::kColDp : C::kColS + g_buf.at * kStep),
                 r_one + static_cast<uint32_t>(g_one.at * kTile), j == 0);
        umma_commit_if(go, &one_empty[g_one.at]);
        g_one.move(1, C::kRing1);
        g_buf.move(1, C::kBufs);
        if (kKeys && j + 1 < n) issue_dp(j + 2 == n);
        if (!kKeys && j + 2 < n) issue_s();
      }
      if (ok) umma_commit_if(go, acc_full);
    }
  } else {
    // ------------------------------------------------------------ P and dS
    const int quarter = warp >> 2;                        // of a step's columns
    const int row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int scale_rows = kKeys ? p.group : 1;
    const uint64_t c2 = pair_f32(p.scale_log2, p.scale_log2);
    const int col0 = quarter * 32;
    const int row_tok = kKeys ? row : row / p.group, row_head = kKeys ? 0 : row - row_tok * p.group;
    BwdWork w;
    RingPos one, two, buf;
    uint32_t dp_phase = 0, acc_phase = 0;
    bool ok = true;
    while (ok && take(w)) {
      const int tok = w.ta + row_tok;
      const bool exists = kKeys ? row < w.tokens : row < w.tokens * p.group;
      // streamed rows this row meets, as an interval from s0
      int lo, hi;
      if (kKeys) {
        lo = p.causal ? max(0, tok - w.sq.off) : 0;
        hi = p.window > 0 ? min(w.sq.nq, tok - w.sq.off + p.window) : w.sq.nq;
      } else {
        lo = p.window > 0 ? max(0, tok + w.sq.off - p.window + 1) : 0;
        hi = p.causal ? min(w.sq.nk, tok + w.sq.off + 1) : w.sq.nk;
      }
      if (!exists) lo = hi = w.s0;
      lo = (lo - w.s0) * scale_rows;
      hi = (hi - w.s0) * scale_rows;
      float lse_r = 0.f, delta_r = 0.f;
      if (!kKeys && exists) {
        const int64_t at = (static_cast<int64_t>(w.sq.q0) + tok) * p.heads_q + w.head * p.group + row_head;
        lse_r = -__ldcg(p.lse_in + at) * kLog2e;      // not from this SM's L1: no wait stands before these
        delta_r = -__ldcg(p.delta + at);
      }
      const uint64_t lse_2 = pair_f32(lse_r, lse_r), delta_2 = pair_f32(delta_r, delta_r);
      for (int j = 0; j < w.n; ++j) {
        if (!mbar_wait(&s_full[buf.at], buf.phase)) { ok = false; break; }
        if (kKeys && !mbar_wait(&one_full[one.at], one.phase)) { ok = false; break; }   // the statistics
        tc_fence_after();
        // what stands behind the sequence's end may be anything: as rows of the reduction it must be zero
        const int left = (kKeys ? w.sq.nq : w.sq.nk) - (w.s0 + j * per_str);
        if (left < per_str) {
          if (kKeys && !mbar_wait(&two_full[two.at], two.phase)) { ok = false; break; }
          const int x = left * scale_rows + row;
          if (x < str_rows) {
            if (quarter == 0) zero_tile_row<C::kChunks>(sOne + one.at * C::kTileBytes, x, kStep * 128);
            if (kKeys && quarter == 1) zero_tile_row<C::kChunks>(sTwo + two.at * C::kTileBytes, x, kStep * 128);
          }
          fence_proxy_async_smem();
        }
        const float* st = sStat + one.at * 2 * kStep + col0;
        const int clo = lo - j * str_rows - col0, chi = hi - j * str_rows - col0;
        const bool edge = __any_sync(0xFFFFFFFFu, clo > 0 || chi < 32);
        const uint32_t t_s = tmem + C::kColS + buf.at * kStep + col0 + lanes, t_dp = tmem + C::kColDp + col0 + lanes;
        uint32_t s[32];                                    // S, then P in 32 bits
        tmem_ld_32x32b_x32(t_s, s);
        tmem_ld_wait();
        {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            uint64_t lse[2] = {lse_2, lse_2};
            if (kKeys) {
              const float4 a = *reinterpret_cast<const float4*>(st + e);
              lse[0] = pair_f32(a.x, a.y);
              lse[1] = pair_f32(a.z, a.w);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int i = e + 2 * x;
              float p0, p1;
              const uint64_t arg = fma_f32x2(pair_f32(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2, lse[x]);
              if (kPolyOf4 > (i / 2) % 4) {
                ex2_poly(arg, p0, p1);
              } else {
                unpair_f32(arg, p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
              }
              if (edge) {
                if (i < clo || i >= chi) p0 = 0.f;
                if (i + 1 < clo || i + 1 >= chi) p1 = 0.f;
              }
              s[i] = __float_as_uint(p0);
              s[i + 1] = __float_as_uint(p1);
              if (kKeys) pk[i / 2] = pack_bf16x2(p0, p1);
            }
          }
          if (kKeys) {
            tmem_st_32x32b_x16(t_s, pk);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
          }
        }
        if (!mbar_wait(dp_full, dp_phase)) { ok = false; break; }
        dp_phase ^= 1;
        tc_fence_after();
        uint32_t d[32];
        tmem_ld_32x32b_x32(t_dp, d);
        tmem_ld_wait();
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          uint64_t delta[2] = {delta_2, delta_2};
          if (kKeys) {
            const float4 z = *reinterpret_cast<const float4*>(st + kStep + e);
            delta[0] = pair_f32(z.x, z.y);
            delta[1] = pair_f32(z.z, z.w);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int i = e + 2 * x;
            float d0, d1;
            unpair_f32(mul_f32x2(pair_f32(__uint_as_float(s[i]), __uint_as_float(s[i + 1])),
                                 add_f32x2(pair_f32(__uint_as_float(d[i]), __uint_as_float(d[i + 1])), delta[x])), d0, d1);
            if (edge) {                                    // dP may be anything there
              if (i < clo || i >= chi) d0 = 0.f;
              if (i + 1 < clo || i + 1 >= chi) d1 = 0.f;
            }
            pk[i / 2] = pack_bf16x2(d0, d1);
          }
        }
        tmem_st_32x32b_x16(kKeys ? t_dp : t_s, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
        one.move(1, C::kRing1);
        two.move(1, C::kRing2);
        buf.move(1, C::kBufs);
      }
      if (!ok) break;
      // a quarter of each gradient's columns
      constexpr int kCols = kHD / 4;
      const int64_t g = static_cast<int64_t>(kKeys ? w.sq.k0 : w.sq.q0) + tok;
      const int64_t out_head = kKeys ? w.head : w.head * p.group + row_head;
      if (w.n > 0) {
        ok = mbar_wait(acc_full, acc_phase);
        acc_phase ^= 1;
        if (!ok) break;
        tc_fence_after();
      }
      uint4 v[kKeys ? 2 : 1][4];
#pragma unroll
      for (int y = 0; y < (kKeys ? 2 : 1); ++y) {
        const float f = (kKeys && y == 0) ? 1.0f : p.scale;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          v[y][2 * q] = v[y][2 * q + 1] = make_uint4(0u, 0u, 0u, 0u);
          if (q * 16 >= kCols || w.n == 0) continue;
          uint32_t o[16];
          tmem_ld_32x32b_x16(tmem + lanes + y * kHD + quarter * kCols + q * 16, o);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 2; ++x)
            v[y][q * 2 + x] = make_uint4(
                pack_bf16x2(__uint_as_float(o[x * 8]) * f, __uint_as_float(o[x * 8 + 1]) * f),
                pack_bf16x2(__uint_as_float(o[x * 8 + 2]) * f, __uint_as_float(o[x * 8 + 3]) * f),
                pack_bf16x2(__uint_as_float(o[x * 8 + 4]) * f, __uint_as_float(o[x * 8 + 5]) * f),
                pack_bf16x2(__uint_as_float(o[x * 8 + 6]) * f, __uint_as_float(o[x * 8 + 7]) * f));
        }
      }
      if (w.n > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty);
      }
      const int vecs = min(kCols / 8, (p.head_dim - quarter * kCols) / 8);
      const int64_t h = out_head * p.head_dim + quarter * kCols;
      if (kKeys) {
        store_rows(exists ? p.dV + g * p.ld_v + h : nullptr, v[0], vecs);
        store_rows(exists ? p.dK + g * p.ld_k + h : nullptr, v[kKeys ? 1 : 0], vecs);
      } else {
        store_rows(exists ? p.dQ + g * p.ld_q + h : nullptr, v[0], vecs);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMathWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (!kKeys) griddep_wait();           // what comes behind this grid comes behind the keys' too
}

// delta[token, head] = sum over the head of dO * O, in 32 bits: 16 lanes per row, 8 elements a lane,
// four rows' loads in flight.
constexpr int kDeltaRows = 64;       // per block
__global__ void __launch_bounds__(256) attn_delta_kernel(const uint16_t* __restrict__ O, const uint16_t* __restrict__ dO,
                                                         int64_t ld, int64_t rows, uint32_t heads, int head_dim,
                                                         float* __restrict__ delta, uint32_t* __restrict__ counters) {
  griddep_enter();
  if (blockIdx.x == 0 && threadIdx.x < 2) counters[threadIdx.x] = 0;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kDeltaRows + (threadIdx.x >> 4);
  const int e = (threadIdx.x & 15) * 8;
  uint4 a[4], z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = first + i * 16;
    a[i] = z[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row < rows && e < head_dim) {
      const int64_t tok = row < UINT32_MAX ? static_cast<uint32_t>(row) / heads : row / heads;
      const int64_t at = tok * ld + (row - tok * heads) * head_dim + e;
      a[i] = __ldcs(reinterpret_cast<const uint4*>(O + at));
      z[i] = *reinterpret_cast<const uint4*>(dO + at);          // read again by the kernels behind this one
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t aw[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, zw[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
    uint64_t s2 = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) s2 = fma_f32x2(pair_bf16(aw[k]), pair_bf16(zw[k]), s2);
    float lo, hi;
    unpair_f32(s2, lo, hi);
    float s = lo + hi;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const int64_t row = first + i * 16;
    if (row < rows && (threadIdx.x & 15) == 0) delta[row] = s;
  }
}

template <int kHD, bool kKeys>
cudaError_t launch(AttnParams p, const AttnMaps& maps, int num_sms, cudaStream_t st) {
  using C = BwdCfg<kHD, kKeys>;
  const int64_t tokens = kKeys ? p.tokens_k : p.tokens_q;
  const int64_t per = kKeys ? 128 : 128 / p.group;
  const int64_t tiles = (kKeys ? p.cu_k : p.cu_q) == nullptr ? p.batch * ((tokens / p.batch + per - 1) / per)
                                                             : std::min<int64_t>(tokens, tokens / per + p.batch);
  p.tiles = static_cast<int32_t>(tiles);
  // heads walked together: those whose streamed tensors (of a mean sequence) share a quarter of the L2 cache (back to
  // back, 8192 tokens, 64 heads: 3609 us, one at a time 3667, all 4076; 32 heads: 1829, 1871, 1901; 4 x 2048, 64 heads: 1169,
  // 1177, 1184)
  const int64_t bytes = std::max<int64_t>(1, (kKeys ? p.tokens_q * p.group : p.tokens_k) / p.batch) * p.head_dim * 4;
  p.head_run = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(p.heads_kv, (int64_t(32) << 20) / bytes)));
  const int64_t blocks = tiles * p.heads_kv;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  if (blocks == 0) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(attn_bwd_kernel<kHD, kKeys>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_bwd_kernel<kHD, kKeys>, static_cast<int>(std::min<int64_t>(blocks, num_sms)), kBwdThreads,
                    C::kSmem, st, 1, p, maps);
}

}  // namespace

cudaError_t launch_attn_bwd(AttnParams p, const uint16_t* Q, const uint16_t* K, const uint16_t* V, float* delta,
                            uint32_t* counters, int num_sms, cudaStream_t st) {
  // both kernels' tiles and steps are 128 rows: the same boxes
  static_assert(kStep == 128, "one set of maps");
  AttnMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  const int64_t tq = std::max<int64_t>(p.tokens_q, 1), tk = std::max<int64_t>(p.tokens_k, 1);
  const int per = kStep / p.group;
  const bool ok = attn_map(&maps.k, K, tk, p.ld_k, p.heads_kv, p.head_dim, 1, kStep) &&
                  attn_map(&maps.v, V, tk, p.ld_v, p.heads_kv, p.head_dim, 1, kStep) &&
                  attn_map(&maps.q, Q, tq, p.ld_q, p.heads_q, p.head_dim, p.group, per) &&
                  attn_map(&maps.dO, p.dO, tq, p.ld_o, p.heads_q, p.head_dim, p.group, per);
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  const int64_t rows = p.tokens_q * p.heads_q;
  if (rows / 16 >= INT32_MAX) return cudaErrorInvalidValue;
  e = launch_pdl(attn_delta_kernel, static_cast<int>(std::max<int64_t>(1, (rows + kDeltaRows - 1) / kDeltaRows)), 256, 0, st,
                 1, p.O_in, p.dO, p.ld_o, rows, static_cast<uint32_t>(p.heads_q), static_cast<int>(p.head_dim), delta,
                 counters);
  p.delta = delta;
  p.counter = counters;
  if (e == cudaSuccess) e = p.head_dim <= 64 ? launch<64, true>(p, maps, num_sms, st) : launch<128, true>(p, maps, num_sms, st);
  p.counter = counters + 1;
  if (e == cudaSuccess) e = p.head_dim <= 64 ? launch<64, false>(p, maps, num_sms, st) : launch<128, false>(p, maps, num_sms, st);
  return e;
}

}  // namespace qlora
