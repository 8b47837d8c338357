// Softmax attention, forward (sm_100a): O = softmax(scale Q K^T over the visible keys) V and
// lse = log sum exp of the scaled logits, one pass over the keys with the running maximum and
// sum of the softmax. Packed sequences, causal and windowed masks, shared key heads.
//
// This kernel is for sequences of more rows than a tile has; attention_few.cu takes the shorter ones.
//
// A block works two tiles of 128 rows (see AttnParams on rows) against the same keys, 64 at a
// time:
//   4 warps a tile  softmax: a thread owns a row (softmax_step). S comes from tensor memory, P goes
//                   back there as bf16 (over S) and is the A operand of P V, so neither S nor P
//                   touches shared memory; rows' sums stay in 32 bits.
//   1 warp a tile   issues the tile's MMAs: P V of a step, then S of the step after the next into
//                   the same columns. Two S buffers per tile keep the softmax from ever waiting
//                   for the tensor core's round trip: with one buffer of 128 keys a step of both
//                   tiles took 4040 cycles, 2550 of them softmax and 1480 the way from P over
//                   P V to the next S.
//   1 warp          finds the block's place, then feeds Q, and K and V through a ring each, by TMA.
// The output accumulates in tensor memory and is rescaled there, which few tiles ever ask for.
//
// Bound by the exponentials and the products in turns: a step of 2100 cycles holds 1050 of each (exp unit 52% busy, tensor
// pipe 51%). 64 heads of 128, causal, 2 x 4096 tokens: 541 us (1017 TFLOP/s) a call by itself at 1.97 GHz, 623 (882) back to
// back for a second, where the power cap leaves 1.63. 16 heads, 8192 tokens, back to back: 285 us (965 TFLOP/s, 1.65 GHz), not
// causal 566 (971, 1.72).
#include <algorithm>
#include <climits>
#include <cstring>

#include "attention_device.cuh"
#include "qlora_kernels.h"

namespace qlora {
namespace {

constexpr int kStep = kFwdStep;
constexpr int kTiles = 2;               // of a block

template <int kHD>
struct FwdCfg {
  static constexpr int kChunks = kHD / 64;                 // 64-column chunks of a row
  static constexpr int kTileBytes = 128 * kHD * 2;         // one Q tile
  static constexpr int kKeyBytes = kStep * kHD * 2;        // one K or V tile
  static constexpr int kSlots = 4 * (128 / kHD);           // of the K ring, and of the V ring
  static constexpr int kSmem = kTiles * kTileBytes + 2 * kSlots * kKeyBytes + 1024 + 512;
  static constexpr int kSoftmax = 4 * kTiles;              // warps
  static constexpr int kThreads = (kSoftmax + kTiles + 1) * 32;
  static constexpr int kTmemCols = 512;                    // S of the tiles (two buffers each), then their O
  static constexpr int kColO = 128 * kTiles;
  static_assert(kSmem <= 232448 - 1536, "shared memory budget");
};

// What a block has to know about its tiles.
struct FwdWork {
  Seq sq;
  int32_t live;             // 0: nothing (the grid covers a few tiles more than there are)
  int32_t head;             // key head
  int32_t base, last, n;    // keys [base, last) that some row sees, in n steps
  struct {
    int32_t ta, rows;       // first token of the tile in its sequence, rows that exist
    int32_t j0, j1;         // steps with keys that some of its rows sees
  } tile[2];
};

template <int kHD>
__global__ void __launch_bounds__(FwdCfg<kHD>::kThreads, 1)
    attn_fwd_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnMaps maps) {
  using C = FwdCfg<kHD>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sK = smem + kTiles * C::kTileBytes;
  uint8_t* sV = sK + C::kSlots * C::kKeyBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + C::kSlots * C::kKeyBytes);
  uint64_t* q_full = bars;                       // [tile]
  uint64_t* s_full = bars + 2;                   // [tile][buffer] S of a step is in tensor memory
  uint64_t* p_full = bars + 6;                   // [tile][buffer] P of a step is, and O may be added to
  uint64_t* o_full = bars + 10;                  // [tile] P V of a step is done
  uint64_t* o_done = bars + 12;                  // [tile] the tile's last P V is
  uint64_t* k_full = bars + 14;                  // [kSlots] each
  uint64_t* k_empty = k_full + C::kSlots;
  uint64_t* v_full = k_empty + C::kSlots;
  uint64_t* v_empty = v_full + C::kSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_empty + C::kSlots);
  __shared__ FwdWork w;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int per_tile = p.per_tile;
  if (warp == 0) {
    if (lane < 2) {
      mbar_init(&q_full[lane], 1);
      mbar_init(&o_full[lane], 1);
      mbar_init(&o_done[lane], 1);
    } else if (lane < 6) {
      mbar_init(&s_full[lane - 2], 1);
      mbar_init(&p_full[lane - 2], 4);
    } else if (lane < 6 + C::kSlots) {
      mbar_init(&k_full[lane - 6], 1);
      mbar_init(&k_empty[lane - 6], kTiles);
      mbar_init(&v_full[lane - 6], 1);
      mbar_init(&v_empty[lane - 6], kTiles);
    }
    fence_mbar_init();
  }
  if (warp == C::kSoftmax) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == C::kSoftmax + kTiles && lane == 0) {
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  griddep_enter();
  constexpr int kTmaWarp = C::kSoftmax + kTiles;
  if (warp == kTmaWarp) {            // the block's place, found while the others set up
    FwdWork mine;
    mine.live = 0;
    int64_t tile;
    int t = 0;
    decode_block(p, blockIdx.x, p.causal != 0, tile, mine.head);
    if (find_tile<false>(p, kTiles * per_tile, tile, mine.sq, t)) {    // there are a few items more than tiles
      mine.live = 1;
      int klo[kTiles], khi[kTiles];
      int base = INT_MAX, end = 0;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const int ta = (t * kTiles + i) * per_tile;
        const int tokens = max(0, min(per_tile, mine.sq.nq - ta));
        mine.tile[i].ta = ta;
        mine.tile[i].rows = tokens * p.group;
        visible_keys(p, mine.sq, ta, tokens, klo[i], khi[i]);
        if (khi[i] > klo[i]) base = min(base, klo[i]);
        end = max(end, khi[i]);
      }
      if (end == 0) base = 0;
      mine.base = base;
      mine.last = end;
      mine.n = end > base ? (end - base + kStep - 1) / kStep : 0;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const int lo = max(klo[i], base), hi = min(khi[i], end);
        mine.tile[i].j0 = hi > lo ? (lo - base) / kStep : 0;
        mine.tile[i].j1 = hi > lo ? (hi - base + kStep - 1) / kStep : 0;
      }
    }
    if (lane == 0) w = mine;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (w.live == 0) {
    // nothing here
  } else if (warp == kTmaWarp) {
    // ------------------------------------------------------------ TMA producer
    const uint32_t q_bytes = static_cast<uint32_t>(per_tile * p.group) * 128 * C::kChunks;
    RingPos kr, vr;
    bool ok = true;
    auto load_q = [&](int i) {
      if (lane != 0 || w.tile[i].j1 <= w.tile[i].j0) return;
      mbar_arrive_expect_tx(&q_full[i], q_bytes);
#pragma unroll
      for (int c = 0; c < C::kChunks; ++c)
        tma_load_3d(sQ + i * C::kTileBytes + c * 128 * 128, &maps.q, &q_full[i], c * 64, w.head * p.group,
                    w.sq.q0 + w.tile[i].ta);
    };
    auto load_kv = [&](uint8_t* ring, const CUtensorMap* map, uint64_t* full, uint64_t* empty, RingPos& r, int j) {
      ok = ok && mbar_wait(&empty[r.at], r.phase ^ 1);
      if (ok && lane == 0) {
        mbar_arrive_expect_tx(&full[r.at], C::kKeyBytes);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
          tma_load_3d(ring + r.at * C::kKeyBytes + c * kStep * 128, map, &full[r.at], c * 64, w.head,
                      w.sq.k0 + w.base + j * kStep);
      }
      r.move(1, C::kSlots);
    };
    const int n = w.n;
    if (n > 0) {
      load_q(0);
      load_kv(sK, &maps.k, k_full, k_empty, kr, 0);
      load_q(1);
      // in the order the MMAs ask for them: K runs two steps ahead of V
      if (n > 1) load_kv(sK, &maps.k, k_full, k_empty, kr, 1);
      for (int j = 0; j < n && ok; ++j) {
        load_kv(sV, &maps.v, v_full, v_empty, vr, j);
        if (j + 2 < n) load_kv(sK, &maps.k, k_full, k_empty, kr, j + 2);
      }
    }
    // the MMAs' last releases have landed before the block ends: those of every slot's last use, if it had one
    auto drain = [&](RingPos r, uint64_t* empty) {
      for (int i = 0; ok && i < C::kSlots; ++i) {
        if (n >= C::kSlots || r.at < n) ok = mbar_wait(&empty[r.at], n >= C::kSlots ? r.phase ^ 1 : 0);
        r.move(1, C::kSlots);
      }
    };
    drain(kr, k_empty);
    drain(vr, v_empty);
  } else if (warp >= C::kSoftmax) {
    // ------------------------------------------------------------ MMA issuer of tile i
    const int i = uniform(warp - C::kSoftmax);
    constexpr uint32_t idesc_s = umma_idesc_bf16(kStep, false, false);
    constexpr uint32_t idesc_o = umma_idesc_bf16(kHD, false, true);
    const uint32_t go = elect_one();
    const uint32_t tm = static_cast<uint32_t>(uniform(static_cast<int>(tmem)));
    const uint32_t t_s = tm + i * 128, t_o = tm + C::kColO + i * kHD;
    const uint64_t dq = umma_desc_sw128(smem_u32(sQ) + i * C::kTileBytes, 16, 1024);
    const uint64_t dk = umma_desc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dv = umma_desc_sw128(smem_u32(sV), kStep * 128, 1024);
    RingPos kr, vr, sb, ob;          // rings of K and V; S buffers of the next S and the next P V
    bool ok = true;
    const int n = uniform(w.n);
    const int j0 = uniform(i == 0 ? w.tile[0].j0 : w.tile[1].j0), j1 = uniform(i == 0 ? w.tile[0].j1 : w.tile[1].j1);
    // K of step j: S, if the tile sees the step; the slot is freed once it holds the step, so that no release counts
    // for an earlier one
    auto take_k = [&](int j) {
      ok = ok && mbar_wait(&k_full[kr.at], kr.phase);
      if (!ok) return;
      if (j >= j0 && j < j1) {
        tc_fence_after();
        const uint64_t b = dk + static_cast<uint32_t>(kr.at * (C::kKeyBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < kHD / 16; ++kk)
          umma_bf16_if(go, t_s + sb.at * kStep, dq + (((kk >> 2) * 128 * 128 + (kk & 3) * 32) >> 4),
                       b + (((kk >> 2) * kStep * 128 + (kk & 3) * 32) >> 4), idesc_s, kk > 0 ? 1u : 0u);
        umma_commit_if(go, &s_full[i * 2 + sb.at]);
        sb.move(1, 2);
      }
      umma_commit_if(go, &k_empty[kr.at]);
      kr.move(1, C::kSlots);
    };
    if (j1 > j0) ok = mbar_wait(&q_full[i], 0);
    for (int j = 0; j < 2 && j < n; ++j) take_k(j);
    for (int j = 0; j < n && ok; ++j) {
      ok = mbar_wait(&v_full[vr.at], vr.phase);
      if (ok && j >= j0 && j < j1) {
        ok = mbar_wait(&p_full[i * 2 + ob.at], ob.phase);
        if (!ok) break;
        tc_fence_after();
        const uint64_t b = dv + static_cast<uint32_t>(vr.at * (C::kKeyBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          umma_bf16_ts_if(go, t_o, t_s + ob.at * kStep + kk * 8, b + kk * (2048 >> 4), idesc_o,
                          (j > j0 || kk > 0) ? 1u : 0u);
        umma_commit_if(go, &o_full[i]);
        if (j + 1 == j1) umma_commit_if(go, &o_done[i]);
        ob.move(1, 2);
      }
      if (ok) umma_commit_if(go, &v_empty[vr.at]);
      vr.move(1, C::kSlots);
      if (j + 2 < n) take_k(j + 2);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int i = warp >> 2;
    const int row = threadIdx.x & 127;
    const int row_tok = row / p.group, row_head = row - row_tok * p.group;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + i * 128 + lanes, t_o = tmem + C::kColO + i * kHD + lanes;
    const float c = p.scale_log2;
    RingPos sb, vj;                  // S buffer and V's slot of the next step
    int steps = 0;                   // done
    bool ok = true;
    const auto r = i == 0 ? w.tile[0] : w.tile[1];
    const int tok = r.ta + row_tok;                      // in the sequence
    const bool exists = row < r.rows;
    const bool warp_works = (row & ~31) < r.rows;        // a warp without rows only keeps the barriers going
    // keys this row sees, from the block's first
    int lo = p.window > 0 ? max(0, tok + w.sq.off - p.window + 1) : 0;
    int hi = p.causal ? min(w.sq.nk, tok + w.sq.off + 1) : w.sq.nk;
    hi = min(hi, w.last);
    lo -= w.base;
    hi -= w.base;
    if (!exists) {                   // a row that nobody looks at asks for no masking either
      lo = 0;
      hi = INT_MAX;
    }
    float m_ref = -INFINITY, l = 0.f;
    vj.skip(r.j0, C::kSlots);
    for (int j = r.j0; j < r.j1; ++j) {
      if (!mbar_wait(&s_full[i * 2 + sb.at], sb.phase)) { ok = false; break; }
      tc_fence_after();
      // values behind the sequence's last key may be anything: 0 * NaN must not reach O
      const int left = w.sq.nk - w.base - j * kStep;
      if (left < kStep) {
        if (!mbar_wait(&v_full[vj.at], vj.phase)) { ok = false; break; }
        if (row >= left && row < kStep) zero_tile_row<C::kChunks>(sV + vj.at * C::kKeyBytes, row, kStep * 128);
        fence_proxy_async_smem();
      }
      vj.move(1, C::kSlots);
      if (warp_works) {
        ok = softmax_step<kHD>(t_s + sb.at * kStep, t_o, c, lo - j * kStep, hi - j * kStep, exists, j == r.j0, m_ref, l,
                               [&]() { return mbar_wait(&o_full[i], (steps - 1) & 1); });
        if (!ok) break;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[i * 2 + sb.at]);
      sb.move(1, 2);
      ++steps;
    }
    const bool any = r.j1 > r.j0;
    // a barrier of its own: the softmax may be up to two products ahead here, and a parity tells neighbouring phases
    // apart only
    ok = ok && (!any || mbar_wait(&o_done[i], 0));
    tc_fence_after();
    const int gh = w.head * p.group + row_head;
    const int64_t gtok = static_cast<int64_t>(w.sq.q0) + tok;
    if (ok && warp_works) {
      if (exists && p.lse != nullptr) p.lse[gtok * p.heads_q + gh] = row_lse(m_ref, l, p.scale);
      uint16_t* out = exists ? p.O + gtok * p.ld_o + static_cast<int64_t>(gh) * p.head_dim : nullptr;
      store_output<kHD, true>(t_o, any ? l : 0.f, out, p.head_dim);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kSoftmax) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int kHD>
cudaError_t launch(const AttnParams& p, const AttnMaps& maps, int64_t blocks, cudaStream_t st) {
  using C = FwdCfg<kHD>;
  auto kernel = attn_fwd_kernel<kHD>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, static_cast<int>(blocks), C::kThreads, C::kSmem, st, 1, p, maps);
}

}  // namespace

bool attn_map(CUtensorMap* m, const void* base, int64_t tokens, int64_t ld, int heads, int head_dim, int box_heads,
              int box_tokens) {
  return tmap_3d_bf16(m, base, static_cast<uint64_t>(head_dim), static_cast<uint64_t>(heads),
                      static_cast<uint64_t>(tokens), static_cast<uint64_t>(head_dim) * 2, static_cast<uint64_t>(ld) * 2,
                      64, static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_tokens));
}

cudaError_t launch_attn_fwd(AttnParams p, const uint16_t* Q, const uint16_t* K, const uint16_t* V, void* ws, int num_sms,
                            cudaStream_t st) {
  AttnMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  const bool few = attn_few_plan(p, num_sms) > 0;
  const int most = 128 / p.group;
  if (!few) p.per_tile = most;
  if (!attn_map(&maps.q, Q, p.tokens_q, p.ld_q, p.heads_q, p.head_dim, p.group, p.per_tile) ||
      !attn_map(&maps.k, K, std::max<int64_t>(p.tokens_k, 1), p.ld_k, p.heads_kv, p.head_dim, 1, kStep) ||
      !attn_map(&maps.v, V, std::max<int64_t>(p.tokens_k, 1), p.ld_v, p.heads_kv, p.head_dim, 1, kStep))
    return cudaErrorInvalidValue;
  if (few) return launch_attn_few(p, maps, static_cast<float*>(ws), st);
  p.tiles = static_cast<int32_t>(attn_tiles(p, 2 * most));
  // heads walked together: those whose keys and values (of a mean sequence) share a quarter of the L2 cache (2 x 4096 tokens,
  // 64 heads, in turns in one run: 520 us; one head at a time 541, all 547)
  const int64_t kv = std::max<int64_t>(1, p.tokens_k / p.batch) * p.head_dim * 4;
  p.head_run = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(p.heads_kv, (int64_t(32) << 20) / kv)));
  const int64_t blocks = static_cast<int64_t>(p.tiles) * p.heads_kv;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return p.head_dim <= 64 ? launch<64>(p, maps, blocks, st) : launch<128>(p, maps, blocks, st);
}

}  // namespace qlora
