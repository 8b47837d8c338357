// Softmax attention, forward, for sequences of few rows (sm_100a): generation, where one or a few
// new tokens meet long caches, short samples, and problems whose tiles would not fill the SMs.
// The formulas, and a tile's steps, are those of attention_fwd.cu; what differs is how the work is
// dealt out.
//
// All tiles' steps (64 keys of one tile of at most 128 rows: a key head's query heads side by side)
// stand in one line, sequence after sequence, and every block takes an equal run of the line: two
// blocks per SM, all resident at once, so that the keys and values, which bound such calls, stream
// through every SM until the end whatever the sequences' lengths. A run may begin and end inside a
// tile; a tile cut that way leaves unnormalised outputs with their maxima and sums in the workspace,
// and a second kernel, which starts under the end of the first, joins them in a fixed order: no
// atomics, the same bits on every call.
//
// Measured back to back (8 key heads of 128, 4 query heads each, one query a sequence; keys and values
// at the copy's rate would take): 16 ragged sequences of 28,900 keys 29.3 us (18.0), 16 of 4096 51.0
// (40.9), 16 of 8192 92.5 (81.7), 19 of 1811 32.9 (21.5), one of 16384 20.1 (10.2). Of a call 6 us are
// its beginning and end (finding the run 1, first loads 1.5), 2 to 3 the second kernel. A cluster of
// blocks per tile that joined its results in shared memory took 34.5, 50, 89, 54 and 22 us in a run in
// which this form took 28.4, 49.5, 89, 32 and 20: blocks of unequal length, a second round of them (4
// us), and 4 us to join.
//
// A block: 4 warps softmax, 1 warp MMAs, 1 warp that finds the segments of the run and feeds Q, and K
// and V through a ring each, by TMA. Loads and first products of a segment run under the end of the
// one before.
#include <algorithm>
#include <climits>

#include "attention_device.cuh"
#include "qlora_kernels.h"

namespace qlora {
namespace {

constexpr int kStep = kFwdStep;
// What a tile's beginning and end cost, in steps. Back to back, the ragged sequences above: 38.3 us with 0, 31.1 with 1, 30.6
// with 2, 30.1 with 3, 30.5 with 5; 300 sequences of 130 to 1200 keys: 192.7, 167.8, 157.6, 154.6, 153.9. Equal sequences,
// whose runs cut them alike, move by 7% at most.
constexpr int kSwitch = 3;
// Tiles of so many steps stay whole (16 sequences of 256 keys: 11.5 us, from 2 steps on cut 13.0; 300 of 130 to 1200: 154.6 and
// 152.9), and all tiles where none can have
// more than kAllWhole: the second launch and its workspace cost a caller 5 us. Others are not cut closer than kSnap steps
// to their ends.
constexpr int kWhole = 4, kAllWhole = 16, kSnap = 2;

template <int kHD, int kRows>
struct FewCfg {
  static constexpr int kChunks = kHD / 64;                 // 64-column chunks of a row
  // Of a tile with at most 32 rows only those have memory: the MMA reads 128 rows from there on, and what stands behind
  // them (the K ring) gives rows of S that nobody looks at.
  static constexpr int kTileBytes = kRows * kHD * 2;
  static constexpr int kKeyBytes = kStep * kHD * 2;        // one K or V tile
  static constexpr int kSlots = (kRows == 128 ? 2 : 3) * (128 / kHD);      // of the K ring, and of the V ring
  static constexpr int kSmem = kTileBytes + 2 * kSlots * kKeyBytes + 1024 + 512;
  static constexpr int kThreads = 6 * 32;
  static constexpr int kTmemCols = 256;                    // two S buffers, then O
  static constexpr int kColO = 128;
  static_assert(kSmem <= 232448 / 2 - 1536, "shared memory budget of two blocks per SM");
  static_assert(kChunks * kRows * 128 + 16384 <= kTileBytes + 2 * kSlots * kKeyBytes, "a Q operand's 128 rows are inside");
};

// Floats of one cut tile's partial result: [head_dim / 4][rows][4] outputs, then [rows][2] maximum and sum.
__host__ __device__ inline int64_t part_floats(int head_dim, int rows) {
  return (static_cast<int64_t>(rows) * (head_dim + 2) + 3) / 4 * 4;
}

// ---------------------------------------------------------------- the line of all tiles' steps
// A tile's steps (one where no key is visible), and their cost in the line.
__device__ __forceinline__ int tile_steps(const AttnParams& p, const Seq& sq, int t, int& lo, int& hi) {
  const int ta = t * p.per_tile;
  visible_keys(p, sq, ta, min(p.per_tile, sq.nq - ta), lo, hi);
  return max(1, (hi - lo + kStep - 1) / kStep);
}
__device__ __forceinline__ void load_seq(const AttnParams& p, int b, Seq& sq) {
  seq_range(p.cu_q, p.tokens_q, p.batch, b, sq.q0, sq.nq);
  seq_range(p.cu_k, p.tokens_k, p.batch, b, sq.k0, sq.nk);
  sq.off = sq.nk - sq.nq;
}
// What a sequence takes of the line, all heads.
__device__ __forceinline__ int seq_cost(const AttnParams& p, const Seq& sq) {
  if (sq.nq <= 0) return 0;
  int lo, hi, sum = tile_steps(p, sq, 0, lo, hi) + kSwitch;
  if (sq.nq > p.per_tile) {
    const int tiles = (sq.nq + p.per_tile - 1) / p.per_tile;
    if (!p.causal) sum *= tiles;
    else
      for (int t = 1; t < tiles; ++t) sum += tile_steps(p, sq, t, lo, hi) + kSwitch;
  }
  return sum * p.heads_kv;
}

struct Place {              // a tile of the line
  Seq sq;
  int32_t b, t, head;
  int32_t n, lo, hi;        // steps, visible keys
  int32_t c0;               // where it begins in the line
};
struct Run {                // block i of the line's equal runs
  int32_t each, more;       // the first `more` runs are one longer
  __device__ __forceinline__ int begin(int i) const { return each * i + min(i, more); }
  // the first run that begins at x > 0 or behind it (past the last: any number above)
  __device__ __forceinline__ int at_or_after(int x) const {
    const int longer = (each + 1) * more;
    if (x <= longer) return (x + each) / (each + 1);
    return each > 0 ? more + (x - longer + each - 1) / each : INT_MAX;
  }
};

// The line's division, and the tile at the beginning of run i (false: the run is empty). Whole warps call it, one
// sequence a lane at a time; up to 32 sequences are read once. (Cold code that runs once bounds this: as 64-bit sums of
// four sequences a lane it took 9 us; a shorter way for many sequences cost calls with 16 of them 2 to 8 us, out of line
// calls with 64 of them 6, and saved 13 of 245 for 1024.)
__device__ __forceinline__ bool find_run(const AttnParams& p, int i, Run& run, Place& at) {
  const int lane = threadIdx.x & 31;
  Seq sq;
  int cost = 0, total = 0;
  auto read = [&](int base) {
    cost = 0;
    if (base + lane < p.batch) {
      load_seq(p, base + lane, sq);
      cost = seq_cost(p, sq);
    }
  };
  for (int base = 0; base < p.batch; base += 32) {
    read(base);
    total += __reduce_add_sync(0xFFFFFFFFu, cost);
  }
  run.each = static_cast<int>(static_cast<uint32_t>(total) / static_cast<uint32_t>(p.blocks));
  run.more = total - run.each * p.blocks;
  const int pos = run.begin(i);
  if (pos >= total || run.begin(i + 1) == pos) return false;
  int before = 0;
  for (int base = 0; base < p.batch; base += 32) {
    if (p.batch > 32) read(base);
    int sum = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, pos < before + sum);
    if (past == 0) {
      before += __shfl_sync(0xFFFFFFFFu, sum, 31);
      continue;
    }
    const int l = __ffs(past) - 1;
    at.b = base + l;
    at.c0 = __shfl_sync(0xFFFFFFFFu, before + sum - cost, l);
    at.sq.q0 = __shfl_sync(0xFFFFFFFFu, sq.q0, l);
    at.sq.nq = __shfl_sync(0xFFFFFFFFu, sq.nq, l);
    at.sq.k0 = __shfl_sync(0xFFFFFFFFu, sq.k0, l);
    at.sq.nk = __shfl_sync(0xFFFFFFFFu, sq.nk, l);
    at.sq.off = at.sq.nk - at.sq.nq;
    for (at.t = 0;; ++at.t) {
      at.n = tile_steps(p, at.sq, at.t, at.lo, at.hi);
      const int all = (at.n + kSwitch) * p.heads_kv;
      if (pos < at.c0 + all || (at.t + 1) * static_cast<int64_t>(p.per_tile) >= at.sq.nq) break;
      at.c0 += all;
    }
    at.head = min(static_cast<int>(static_cast<uint32_t>(pos - at.c0) / static_cast<uint32_t>(at.n + kSwitch)), p.heads_kv - 1);
    at.c0 += at.head * (at.n + kSwitch);
    return true;
  }
  return false;
}
// The next tile; false after the last.
__device__ __forceinline__ bool next_place(const AttnParams& p, Place& at) {
  at.c0 += at.n + kSwitch;
  if (++at.head < p.heads_kv) return true;
  at.head = 0;
  if ((++at.t) * static_cast<int64_t>(p.per_tile) >= at.sq.nq) {
    at.t = 0;
    do {
      if (++at.b >= p.batch) return false;
      load_seq(p, at.b, at.sq);
    } while (at.sq.nq == 0);
  }
  at.n = tile_steps(p, at.sq, at.t, at.lo, at.hi);
  return true;
}
// Where a run's boundary, x behind a tile's beginning in the line, cuts the tile's n steps: 0 and n are no cuts.
__device__ __forceinline__ int cut_at(const AttnParams& p, int x, int n) {
  const int s = x - kSwitch;
  if (n <= p.whole) return s >= (n + 1) / 2 ? n : 0;
  return s < kSnap ? 0 : s > n - kSnap ? n : s;
}

// A segment: steps of one tile that a block takes.
struct FewWork {
  Seq sq;
  int32_t live;             // 0: no more
  int32_t head;             // key head
  int32_t ta, rows;         // first token of the tile in its sequence, rows that exist
  int32_t base, last, n;    // keys [base, last) in n >= 1 steps
  int32_t part;             // its place in the workspace, -1: the whole tile
};
constexpr int kQueue = 4;   // the S products run two steps, so at most two segments, ahead of the others

template <int kHD, int kRows>
__global__ void __launch_bounds__(FewCfg<kHD, kRows>::kThreads, 2)
    attn_few_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ AttnMaps maps, float* parts) {
  using C = FewCfg<kHD, kRows>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::kTileBytes;
  uint8_t* sV = sK + C::kSlots * C::kKeyBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + C::kSlots * C::kKeyBytes);
  uint64_t* q_full = bars;                       // Q of a segment
  uint64_t* q_empty = bars + 1;                  // no product reads it any more
  uint64_t* o_full = bars + 2;                   // P V of a step is done
  uint64_t* o_done = bars + 3;                   // a segment's last P V is
  uint64_t* s_full = bars + 4;                   // [2] S of a step is in tensor memory
  uint64_t* p_full = bars + 6;                   // [2] P of a step is, and O may be added to
  uint64_t* work_full = bars + 8;                // [kQueue]
  uint64_t* work_empty = work_full + kQueue;     // [kQueue]
  uint64_t* k_full = work_empty + kQueue;        // [kSlots] each
  uint64_t* k_empty = k_full + C::kSlots;
  uint64_t* v_full = k_empty + C::kSlots;
  uint64_t* v_empty = v_full + C::kSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_empty + C::kSlots);
  __shared__ FewWork work[kQueue];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  constexpr int kMmaWarp = 4, kTmaWarp = 5;
  if (warp == 0) {
    if (lane < 4) {
      mbar_init(&bars[lane], 1);
    } else if (lane < 6) {
      mbar_init(&s_full[lane - 4], 1);
      mbar_init(&p_full[lane - 4], 4);
    } else if (lane < 6 + kQueue) {
      mbar_init(&work_full[lane - 6], 1);
      mbar_init(&work_empty[lane - 6], 6);       // four softmax warps, and the MMA warp for S and for P V
    } else if (lane < 6 + kQueue + C::kSlots) {
      const int i = lane - 6 - kQueue;
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  griddep_enter();
  // the block's run of the line and its first tile, found while the others set up
  Place at;
  Run run;
  bool more = false;
  if (warp == kTmaWarp) more = find_run(p, static_cast<int>(blockIdx.x), run, at);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // the consumers walk over the segments with this: false after the last one
  auto take = [&](RingPos& pos, FewWork& w) {
    if (!mbar_wait(&work_full[pos.at], pos.phase)) return false;
    w = work[pos.at];
    __syncwarp();
    if (lane == 0) mbar_arrive(&work_empty[pos.at]);
    pos.move(1, kQueue);
    return w.live != 0;
  };

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ segments, TMA producer
    const uint32_t q_bytes = static_cast<uint32_t>(p.per_tile * p.group) * 128 * C::kChunks;
    RingPos kr, vr, qr;
    uint32_t q_phase = 1;            // the first wait finds the memory free
    int published = 0, steps = 0;
    bool ok = true;
    auto publish = [&](const FewWork& w) {
      if (published >= kQueue) ok = ok && mbar_wait(&work_empty[qr.at], qr.phase ^ 1);
      if (ok && lane == 0) {
        work[qr.at] = w;
        mbar_arrive(&work_full[qr.at]);
      }
      qr.move(1, kQueue);
      ++published;
    };
    auto load_kv = [&](uint8_t* ring, const CUtensorMap* map, uint64_t* full, uint64_t* empty, RingPos& r, int head, int tok) {
      ok = ok && mbar_wait(&empty[r.at], r.phase ^ 1);
      if (ok && lane == 0) {
        mbar_arrive_expect_tx(&full[r.at], C::kKeyBytes);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
          tma_load_3d(ring + r.at * C::kKeyBytes + c * kStep * 128, map, &full[r.at], c * 64, head, tok);
      }
      r.move(1, C::kSlots);
    };
    const int from = more ? run.begin(static_cast<int>(blockIdx.x)) : 0, to = more ? run.begin(static_cast<int>(blockIdx.x) + 1) : 0;
    for (; more && ok && at.c0 < to; more = next_place(p, at)) {
      const int s0 = cut_at(p, from - at.c0, at.n), s1 = cut_at(p, to - at.c0, at.n);
      if (s1 <= s0) continue;
      FewWork w;
      w.sq = at.sq;
      w.live = 1;
      w.head = at.head;
      w.ta = at.t * p.per_tile;
      w.rows = min(p.per_tile, at.sq.nq - w.ta) * p.group;
      if (at.hi <= at.lo) {          // rows that see no key
        for (int r = 0; r < w.rows; ++r) {
          const int64_t tok = static_cast<int64_t>(at.sq.q0) + w.ta + r / p.group;
          const int head = at.head * p.group + r % p.group;
          if (lane * 8 < p.head_dim)
            *reinterpret_cast<uint4*>(p.O + tok * p.ld_o + static_cast<int64_t>(head) * p.head_dim + lane * 8) =
                make_uint4(0u, 0u, 0u, 0u);
          if (lane == 0 && p.lse != nullptr) p.lse[tok * p.heads_q + head] = -INFINITY;
        }
        continue;
      }
      w.n = s1 - s0;
      w.base = at.lo + s0 * kStep;
      w.last = min(at.hi, at.lo + s1 * kStep);
      w.part = s0 == 0 && s1 == at.n ? -1 : static_cast<int>(2 * blockIdx.x) + (s0 == 0 ? 1 : 0);
      publish(w);
      ok = ok && mbar_wait(q_empty, q_phase);
      q_phase ^= 1;
      if (ok && lane == 0) {
        mbar_arrive_expect_tx(q_full, q_bytes);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
          tma_load_3d(sQ + c * kRows * 128, &maps.q, q_full, c * 64, w.head * p.group, w.sq.q0 + w.ta);
      }
      // in the order the MMAs ask for them: K runs two steps ahead of V
      const int tok = w.sq.k0 + w.base;
      auto load_k = [&](int j) { load_kv(sK, &maps.k, k_full, k_empty, kr, w.head, tok + j * kStep); };
      load_k(0);
      if (w.n > 1) load_k(1);
      for (int j = 0; j < w.n && ok; ++j) {
        load_kv(sV, &maps.v, v_full, v_empty, vr, w.head, tok + j * kStep);
        if (j + 2 < w.n) load_k(j + 2);
      }
      steps += w.n;
    }
    FewWork none;
    none.live = 0;
    publish(none);
    // the MMAs' last releases have landed before the block ends: those of every slot's last use, if it had one
    auto drain = [&](RingPos r, uint64_t* empty) {
      for (int i = 0; ok && i < C::kSlots; ++i) {
        if (steps >= C::kSlots || r.at < steps) ok = mbar_wait(&empty[r.at], steps >= C::kSlots ? r.phase ^ 1 : 0);
        r.move(1, C::kSlots);
      }
    };
    drain(kr, k_empty);
    drain(vr, v_empty);
    if (ok && steps > 0) mbar_wait(q_empty, q_phase);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = umma_idesc_bf16(kStep, false, false);
    constexpr uint32_t idesc_o = umma_idesc_bf16(kHD, false, true);
    const uint32_t go = elect_one();
    const uint32_t t_s = static_cast<uint32_t>(uniform(static_cast<int>(tmem))), t_o = t_s + C::kColO;
    const uint64_t dq = umma_desc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dk = umma_desc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dv = umma_desc_sw128(smem_u32(sV), kStep * 128, 1024);
    RingPos kr, vr, sb, ob, ws, wo;  // rings of K and V; S buffers of the next S and the next P V; segments of both
    FewWork w;
    int s_left = 0;                  // steps of the S products' segment to come
    uint32_t q_phase = 0;
    bool ok = true, s_more = true;
    // S of the next step of all segments
    auto next_s = [&]() {
      if (!ok || !s_more) return;
      if (s_left == 0) {
        s_more = take(ws, w);
        if (!s_more) return;
        s_left = uniform(w.n);
        ok = mbar_wait(q_full, q_phase);
        q_phase ^= 1;
      }
      ok = ok && mbar_wait(&k_full[kr.at], kr.phase);
      if (!ok) return;
      tc_fence_after();
      const uint64_t b = dk + static_cast<uint32_t>(kr.at * (C::kKeyBytes >> 4));
#pragma unroll
      for (int kk = 0; kk < kHD / 16; ++kk)
        umma_bf16_if(go, t_s + sb.at * kStep, dq + (((kk >> 2) * kRows * 128 + (kk & 3) * 32) >> 4),
                     b + (((kk >> 2) * kStep * 128 + (kk & 3) * 32) >> 4), idesc_s, kk > 0 ? 1u : 0u);
      umma_commit_if(go, &s_full[sb.at]);
      umma_commit_if(go, &k_empty[kr.at]);
      if (--s_left == 0) umma_commit_if(go, q_empty);
      sb.move(1, 2);
      kr.move(1, C::kSlots);
    };
    next_s();
    next_s();
    while (ok && take(wo, w)) {
      const int n = uniform(w.n);
      for (int j = 0; j < n && ok; ++j) {
        ok = mbar_wait(&v_full[vr.at], vr.phase) && mbar_wait(&p_full[ob.at], ob.phase);
        if (!ok) break;
        tc_fence_after();
        const uint64_t b = dv + static_cast<uint32_t>(vr.at * (C::kKeyBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk)
          umma_bf16_ts_if(go, t_o, t_s + ob.at * kStep + kk * 8, b + kk * (2048 >> 4), idesc_o,
                          (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit_if(go, o_full);
        if (j + 1 == n) umma_commit_if(go, o_done);
        umma_commit_if(go, &v_empty[vr.at]);
        ob.move(1, 2);
        vr.move(1, C::kSlots);
        next_s();
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int row = threadIdx.x;
    const int row_tok = row / p.group, row_head = row - row_tok * p.group;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t t_s = tmem + lanes, t_o = tmem + C::kColO + lanes;
    RingPos sb, vr, wr;              // S buffer and V's slot of the next step; the next segment
    uint32_t steps = 0, o_phase = 0;
    bool ok = true;
    FewWork w;
    while (ok && take(wr, w)) {
      const int tok = w.ta + row_tok;                      // in the sequence
      const bool exists = row < w.rows;
      const bool warp_works = (row & ~31) < w.rows;        // a warp without rows only keeps the barriers going
      // keys this row sees, from the segment's first
      int lo = (p.window > 0 ? max(0, tok + w.sq.off - p.window + 1) : 0) - w.base;
      int hi = min(w.last, p.causal ? min(w.sq.nk, tok + w.sq.off + 1) : w.sq.nk) - w.base;
      if (!exists) {                 // a row that nobody looks at asks for no masking either
        lo = 0;
        hi = INT_MAX;
      }
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < w.n; ++j) {
        ok = mbar_wait(&s_full[sb.at], sb.phase);
        if (!ok) break;
        tc_fence_after();
        // values behind the sequence's last key may be anything: 0 * NaN must not reach O
        const int left = w.sq.nk - w.base - j * kStep;
        if (left < kStep) {
          ok = mbar_wait(&v_full[vr.at], vr.phase);
          if (!ok) break;
          if (row >= left && row < kStep) zero_tile_row<C::kChunks>(sV + vr.at * C::kKeyBytes, row, kStep * 128);
          fence_proxy_async_smem();
        }
        vr.move(1, C::kSlots);
        if (warp_works) {
          ok = softmax_step<kHD>(t_s + sb.at * kStep, t_o, p.scale_log2, lo - j * kStep, hi - j * kStep, exists, j == 0,
                                 m_ref, l, [&]() { return mbar_wait(o_full, (steps - 1) & 1); });
          if (!ok) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sb.at]);
        sb.move(1, 2);
        ++steps;
      }
      ok = ok && mbar_wait(o_done, o_phase);
      o_phase ^= 1;
      if (!ok || !warp_works) continue;
      tc_fence_after();
      if (w.part >= 0) {
        const int rows = p.per_tile * p.group;
        float* part = parts + w.part * part_floats(kHD, rows);
#pragma unroll 1
        for (int q = 0; q < kHD / 32; ++q) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(t_o + q * 32, o);
          tmem_ld_wait();
          if (exists)
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + (static_cast<int64_t>(q * 8 + e / 4) * rows + row) * 4) =
                  make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
        if (exists)
          *reinterpret_cast<float2*>(part + static_cast<int64_t>(rows) * kHD + row * 2) = make_float2(m_ref, l);
      } else {
        const int gh = w.head * p.group + row_head;
        const int64_t gtok = static_cast<int64_t>(w.sq.q0) + tok;
        if (exists && p.lse != nullptr) p.lse[gtok * p.heads_q + gh] = row_lse(m_ref, l, p.scale);
        uint16_t* out = exists ? p.O + gtok * p.ld_o + static_cast<int64_t>(gh) * p.head_dim : nullptr;
        store_output<kHD, kRows == 128>(t_o, l, out, p.head_dim);
      }
      tc_fence_before();             // the next segment's first P V, behind p_full, overwrites O
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Joins the pieces of the tile that the beginning of run blockIdx.x + 1 cuts:
//   O = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s, m = max m_s, in a fixed order.
// The blocks whose runs cut the same tile share its rows; in a block, groups of threads share the pieces.
// kMany: tiles of more than 32 rows, whose pieces may be many items for each thread (the shorter code for the others is
// worth 2 us: it runs once, cold).
constexpr int kJoinThreads = 256;
template <int kHD, bool kMany>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnParams p, const float* parts) {
  __shared__ float4 sO[kJoinThreads];
  __shared__ float2 sMl[kJoinThreads];
  __shared__ Place sAt;
  __shared__ int sCuts[2];          // runs first .. end cut the tile: blocks first - 1 .. end have a piece
  // One warp finds the tile (all of them doing it took most of a call with long tiles). The offsets were written before
  // the grid before this one passed its own wait, so they may be read under its end.
  const int g = static_cast<int>(blockIdx.x) + 1;
  if (threadIdx.x < 32) {
    Run run;
    Place at;
    int first = 0, end = -1;
    if (find_run(p, g, run, at)) {
      const int c = cut_at(p, run.begin(g) - at.c0, at.n);
      if (c > 0 && c < at.n) {
        // (within the workspace also where overlapping sequences, from bad offsets, make the line longer than 32 bits)
        first = max(1, run.at_or_after(at.c0 + kSwitch + kSnap));
        end = min(p.blocks, run.at_or_after(at.c0 + kSwitch + at.n - kSnap + 1)) - 1;
      }
      if (threadIdx.x == 0) sAt = at;
    }
    if (threadIdx.x == 0) {
      sCuts[0] = first;
      sCuts[1] = end;
    }
  }
  // also where nothing is to do: the grid behind this one relies on the one before
  griddep_enter();
  __syncthreads();
  const int first = sCuts[0], end = sCuts[1];
  if (end < first) return;
  const Place& at = sAt;
  const int ta = at.t * p.per_tile;
  const int stride = p.per_tile * p.group, rows = min(p.per_tile, at.sq.nq - ta) * p.group;
  const int64_t size = part_floats(kHD, stride);
  const int vecs = p.head_dim / 4, items = rows * vecs;
  // Each block takes `share` of the items (four columns of a row). Few of them: groups of threads share the pieces too.
  // A thread has kAhead requests under way: of as many pieces, or, where its group takes all pieces, of as many items.
  constexpr int kAhead = 4;
  const int sharers = end - first + 1, pieces = sharers + 1, share = (items + sharers - 1) / sharers;
  int groups = 1;
  while (groups < 8 && groups < pieces && kJoinThreads / (2 * groups) >= max(32, share)) groups *= 2;
  const bool wide = kMany && share > kJoinThreads;
  constexpr int kSets = kMany ? kAhead : 1;
  const int each = kJoinThreads / groups, mine_group = threadIdx.x / each, mine_item = threadIdx.x - mine_group * each;
  const int per_round = wide ? kAhead * kJoinThreads : each;
  for (int x0 = (g - first) * per_round; x0 < items; x0 += sharers * per_round) {
    float m[kSets] = {}, l[kSets] = {};
    float4 o[kSets] = {};
    auto add = [&](int u, float2 ml, float4 os) {
      const float top = fmaxf(m[u], ml.x);
      const float f = m[u] == -INFINITY ? 0.f : ex2((m[u] - top) * p.scale_log2);
      const float fs = ml.x == -INFINITY ? 0.f : ex2((ml.x - top) * p.scale_log2);
      m[u] = top;
      l[u] = l[u] * f + ml.y * fs;
      o[u].x = o[u].x * f + os.x * fs;
      o[u].y = o[u].y * f + os.y * fs;
      o[u].z = o[u].z * f + os.z * fs;
      o[u].w = o[u].w * f + os.w * fs;
    };
    int v[kSets], row[kSets];
#pragma unroll
    for (int u = 0; u < kSets; ++u) {
      const int x = x0 + mine_item + (wide ? u * kJoinThreads : 0);
      v[u] = x / rows;
      row[u] = x - v[u] * rows;
      if (x >= items) v[u] = -1;
      m[u] = -INFINITY;
      l[u] = 0.f;
      o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int stride_i = wide ? 1 : kAhead * groups;
    for (int i0 = first - 1 + mine_group; i0 <= end; i0 += stride_i) {
      float2 ml[kAhead];
      float4 os[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + (wide ? 0 : u * groups);
        ml[u] = make_float2(-INFINITY, 0.f);
        os[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int k = u % kSets;
        if (v[k] < 0 || i > end) continue;
        const float* from = parts + (2 * static_cast<int64_t>(i) + (i == first - 1 ? 1 : 0)) * size;
        ml[u] = __ldcg(reinterpret_cast<const float2*>(from + stride * kHD + row[k] * 2));
        os[u] = __ldcg(reinterpret_cast<const float4*>(from + (v[k] * stride + row[k]) * 4));
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) add(u % kSets, ml[u], os[u]);
    }
    auto store = [&](int u) {
      const float inv = l[u] != 0.f ? 1.0f / l[u] : 0.f;
      const int tok = row[u] / p.group, gh = at.head * p.group + row[u] - tok * p.group;
      const int64_t gtok = static_cast<int64_t>(at.sq.q0) + ta + tok;
      *reinterpret_cast<uint2*>(p.O + gtok * p.ld_o + static_cast<int64_t>(gh) * p.head_dim + v[u] * 4) =
          make_uint2(pack_bf16x2(o[u].x * inv, o[u].y * inv), pack_bf16x2(o[u].z * inv, o[u].w * inv));
      if (v[u] == 0 && p.lse != nullptr) p.lse[gtok * p.heads_q + gh] = row_lse(m[u], l[u], p.scale);
    };
    if (wide) {
#pragma unroll
      for (int u = 0; u < kSets; ++u)
        if (v[u] >= 0) store(u);
      continue;
    }
#pragma unroll
    for (int u = 1; u < kSets; ++u) add(0, make_float2(m[u], l[u]), o[u]);
    sO[threadIdx.x] = o[0];
    sMl[threadIdx.x] = make_float2(m[0], l[0]);
    __syncthreads();
    if (mine_group == 0 && v[0] >= 0) {
      for (int i = 1; i < groups; ++i) add(0, sMl[threadIdx.x + i * each], sO[threadIdx.x + i * each]);
      store(0);
    }
    __syncthreads();
  }
}

// Steps of the longest tile there can be, in a call of p's sizes.
int64_t most_steps(const AttnParams& p) {
  int64_t keys = p.cu_k == nullptr ? p.tokens_k / p.batch : p.tokens_k;
  if (p.window > 0) keys = std::min<int64_t>(keys, static_cast<int64_t>(p.window) + p.per_tile - 1);
  return std::max<int64_t>(1, (keys + kStep - 1) / kStep);
}

template <int kHD, int kRows>
cudaError_t launch(const AttnParams& p, const AttnMaps& maps, float* parts, cudaStream_t st) {
  using C = FewCfg<kHD, kRows>;
  auto kernel = attn_few_kernel<kHD, kRows>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e == cudaSuccess) e = launch_pdl(kernel, p.blocks, C::kThreads, C::kSmem, st, 1, p, maps, parts);
  if (e != cudaSuccess || p.whole == INT_MAX) return e;
  return launch_pdl(attn_join_kernel<kHD, (kRows > 32)>, p.blocks - 1, kJoinThreads, 0, st, 1, p, static_cast<const float*>(parts));
}

}  // namespace

size_t attn_few_plan(AttnParams& p, int num_sms) {
  const int most = 128 / p.group;
  const int64_t mean_q = (p.tokens_q + p.batch - 1) / p.batch;
  // Two tiles of 128 rows per block need sequences of more than one, and enough of them for every SM: 2048 tokens of 32
  // heads, causal, take 44 us there and 63 here, 4096 of 8 heads 68 there and 57 here.
  if (mean_q * p.group > 128 && attn_tiles(p, 2 * most) * p.heads_kv >= num_sms) return 0;
  p.per_tile = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(most, mean_q)));
  const int64_t line = attn_tiles(p, p.per_tile) * p.heads_kv * (most_steps(p) + kSwitch);
  if (line > INT32_MAX) return 0;            // the line is counted in 32 bits
  p.blocks = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(2 * static_cast<int64_t>(num_sms), line)));
  p.whole = p.blocks > 1 && most_steps(p) > kAllWhole ? kWhole : INT_MAX;
  if (p.whole == INT_MAX) return 1;
  return static_cast<size_t>(2 * static_cast<int64_t>(p.blocks) *
                             part_floats(p.head_dim <= 64 ? 64 : 128, p.per_tile * p.group)) * 4;
}

cudaError_t launch_attn_few(const AttnParams& p, const AttnMaps& maps, float* part, cudaStream_t st) {
  // memory for 32 rows of Q leaves a third place in the rings (the ragged sequences above: 28.5 us, with 128 rows 33.1)
  const bool few = p.per_tile * p.group <= 32;
  if (p.head_dim <= 64) return few ? launch<64, 32>(p, maps, part, st) : launch<64, 128>(p, maps, part, st);
  return few ? launch<128, 32>(p, maps, part, st) : launch<128, 128>(p, maps, part, st);
}

}  // namespace qlora
