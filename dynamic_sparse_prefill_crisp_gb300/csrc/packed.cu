// Causal GQA softmax attention over packed sequences on the 5th-generation
// tensor cores. Sequence b has the query rows [cu_q[b], cu_q[b+1]) and the key
// rows [cu_k[b], cu_k[b+1]) of packed tensors; with off = k_len - q_len its
// query i sees its keys j <= off + i.
//
// A tile is `tokens` consecutive queries of one sequence times `hp` query heads
// of one kv head (128 rows at most, token by token): a kv head's keys are read
// once for its whole group, and a short prompt fills a tile with its heads
// where rows of one head alone would leave it empty. Tiles run in the order of
// the keys they see, most first, kv head by kv head; a CTA finds its tile from
// the lengths (find_tile), so that no schedule has to be made or kept.
//
// The work on a tile is csrc/attention.cu's: 64-key sub-blocks, two score
// buffers in TMEM, the first sub-block's row maximum as the reference, two more
// passes where a row's sum passes 2^64. What differs:
//  - sub-blocks start at any key row, so the rows behind a sequence's last key
//    are another sequence's. Their scores are masked and their V rows are zeroed
//    in shared memory; elements of V that only some of the tile's rows see and
//    that are no finite number are taken out of the product and added to the
//    rows that see them at the end (0 times NaN would reach the others).
//  - when there are too few tiles for the GPU, a tile's keys are split over
//    several CTAs, whose unfinished rows a second kernel joins in a fixed order.
//
// Warp roles: 0-7 softmax + epilogue, 8 TMA producer, 9 MMA issuer (TMEM owner).
#include <algorithm>
#include <cuda_bf16.h>
#include <type_traits>

#include "attn.cuh"

namespace crisp {
using namespace ptx;

namespace {

constexpr int kSoftmaxWarps = 8;
constexpr int kWarps = kSoftmaxWarps + 2;
constexpr int kThreads = kWarps * 32;
constexpr int kTmaWarp = kSoftmaxWarps, kMmaWarp = kSoftmaxWarps + 1;
constexpr int kSubKeys = kB / 2;                          // keys per sub-block
constexpr uint32_t kTile = kB * kD * 2;                   // 32 KB bf16 tile (Q)
constexpr uint32_t kHalf = kTile / 2;                     // Q: one 64-feature half
constexpr uint32_t kSub = kTile / 2;                      // K or V: one sub-block (both feature halves)
constexpr uint32_t kSubHalf = kSub / 2;                   // 64 keys x 64 features
constexpr uint32_t kSmemBytes = 1024 + kTile + 4 * kSub;  // Q, K[2], V[2] (+ alignment slack)
constexpr uint32_t kTmemCols = 256;                       // S/P [0,64) and [64,128), O [128,256)

enum Mode : int { kFast = 0, kMaxOnly = 1, kFixed = 2 };

struct PackedArgs {
  const int32_t *cu_q, *cu_k;
  int batch, total_q, total_k, hq, group;
  int hp, chunks;         // heads of a tile; tiles that a group's heads take
  int tokens;             // queries of a tile
  uint32_t inv_tokens;    // ceil(2^32 / tokens), 0 for one token
  int bound;              // no batch of these sizes has more (sequence, tokens) tiles
  int splits, split_subs; // CTAs of a tile and sub-blocks of each (the last takes what is left)
  float c_log2;
  __nv_bfloat16* out;
  int64_t o_hs, o_ts;
  const __nv_bfloat16* v;
  int64_t v_hs, v_ts;
  float* part;            // [splits][total_q][hq][128]  unfinished rows (splits > 1)
  float2* part_ml;        // [splits][total_q][hq]       their references and sums
  DevStatus* status;
};

struct Tile {
  int q0, k0;        // the sequence's first rows
  int nq, nk;
  int t0;            // the tile's first query
  int cost;          // sub-blocks it sees
};

struct Bars {
  uint64_t q_full;
  uint64_t k_full[2], v_full[2], v_empty[2];  // a K slot is free again once s_full of its sub-block completes
  uint64_t s_full[2], p_full[2];
  uint64_t o_full, drain;
  uint64_t xbar[4];      // per lane quarter: both warps have written their partial row maxima
  uint32_t tmem_base;
  int abort;
  int redo;              // a chunk row sum passed kOverflowSum (fast pass)
  int odd_v;             // a partly seen V element is not finite
  int found;             // the CTA has a tile
  int sum[kWarps], top[kWarps], count[2][kWarps];
  Tile tile;
  float xmax[2][kB];     // [chunk][row]: partial row maxima
  float xsum[2][kB];     // [chunk][row]: partial row sums (epilogue)
};

__host__ __device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }
// x / tokens for 0 <= x < 2^25 (inv_tokens is off by less than tokens <= 2^7).
__device__ __forceinline__ int over_tokens(const PackedArgs& a, int x) {
  return a.inv_tokens == 0u ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), a.inv_tokens));
}
// Sub-blocks that the tile of queries [t0, t0 + tokens) sees.
__device__ __forceinline__ int tile_cost(int nq, int nk, int t0, int tokens) {
  const int end = nk - nq + min(t0 + tokens, nq);
  return end > 0 ? (end + kSubKeys - 1) / kSubKeys : 0;
}
__device__ __forceinline__ int tiles_of(const PackedArgs& a, int nq) { return over_tokens(a, nq + a.tokens - 1); }
// Tiles of a sequence that see c sub-blocks or more: its last ones.
__device__ __forceinline__ int tiles_from(const PackedArgs& a, int2 n, int c) {
  const int tiles = tiles_of(a, n.x);
  if (c <= 0 || tiles == 0) return tiles;
  const int keys = kSubKeys * (c - 1);  // more than these
  if (n.y <= keys) return 0;
  const int x = keys - (n.y - n.x);  // queries that see no more, if whole tiles of them
  return x <= 0 ? tiles : tiles - min(over_tokens(a, x), tiles - 1);
}

// The lengths of sequence b, or {0, 0} where cu_q or cu_k do not describe one.
__device__ __forceinline__ int2 seq_lens(const PackedArgs& a, int b, bool& ok) {
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  ok = q0 >= 0 && q1 >= q0 && q1 <= a.total_q && k0 >= 0 && k1 >= k0 && k1 <= a.total_k && q1 - q0 <= kMaxSeq &&
       k1 - k0 <= kMaxSeq;
  return ok ? make_int2(q1 - q0, k1 - k0) : make_int2(0, 0);
}

// The tile of a rank in the order of descending cost (equal costs: by sequence,
// then by query). With N(c) the tiles of cost c or more, the rank's cost is the
// largest c with N(c) > rank; each warp counts one N(c) a round, so that a
// round cuts the range to an eleventh (16k tokens, 256 costs: three rounds).
// seqs: room for the batch's lengths. All threads; the result in bars.tile
// (bars.found stays 0 where there is none).
__device__ void find_tile(const PackedArgs& a, int rank, int2* seqs, Bars& bars) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int tiles = 0, top = 0;
  for (int b = threadIdx.x; b < a.batch; b += kThreads) {
    bool ok;
    const int2 n = seq_lens(a, b, ok);
    if (!ok && blockIdx.x == 0) report_error(a.status, CRISP_ERR_BOUNDS, 0x801);
    seqs[b] = n;
    tiles += tiles_of(a, n.x);
    if (n.x > 0) top = max(top, (n.y + kSubKeys - 1) / kSubKeys);
  }
  tiles = __reduce_add_sync(0xffffffffu, tiles);
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) {
    bars.sum[warp] = tiles;
    bars.top[warp] = top;
  }
  __syncthreads();
  tiles = top = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    tiles += bars.sum[w];
    top = max(top, bars.top[w]);
  }
  if (rank >= tiles) return;
  int lo = 0, hi = top + 1, above = 0;  // N(lo) > rank >= N(hi) = above
  for (int round = 0; hi - lo > 1; ++round) {
    const int step = (hi - lo + kWarps) / (kWarps + 1), c = lo + (warp + 1) * step;
    int n = 0;
    if (c < hi)
      for (int b = lane; b < a.batch; b += 32) n += tiles_from(a, seqs[b], c);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) bars.count[round & 1][warp] = n;
    __syncthreads();
    const int lo0 = lo, hi0 = hi;
    for (int w = 0; w < kWarps; ++w) {
      const int cw = lo0 + (w + 1) * step;
      if (cw >= hi0) break;
      const int nw = bars.count[round & 1][w];
      if (nw <= rank) {
        hi = cw;
        above = nw;
        break;
      }
      lo = cw;
    }
  }
  if (warp == kTmaWarp) {
    // The rank-th of the tiles of cost lo, each lane counting neighbouring sequences.
    const int per = div_up(a.batch, 32), b0 = min(lane * per, a.batch), b1 = min(b0 + per, a.batch);
    auto of_cost = [&](int b) {
      return tiles_from(a, seqs[b], lo) - tiles_from(a, seqs[b], lo + 1);
    };
    int mine = 0;
    for (int b = b0; b < b1; ++b) mine += of_cost(b);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    int left = rank - above - (upto - mine);
    if (left >= 0 && left < mine) {
      int b = b0;
      for (; b + 1 < b1; ++b) {
        const int m = of_cost(b);
        if (left < m) break;
        left -= m;
      }
      const int2 n = seqs[b];
      Tile t;
      t.nq = n.x;
      t.nk = n.y;
      t.q0 = a.cu_q[b];
      t.k0 = a.cu_k[b];
      t.t0 = (tiles_of(a, n.x) - tiles_from(a, n, lo) + left) * a.tokens;
      t.cost = lo;
      bars.tile = t;
      bars.found = 1;
    }
  }
  __syncthreads();
}

// Keys past the row's last one (columns above lim) -> -inf.
__device__ __forceinline__ void mask_from32(int lim, uint32_t (&sv)[32]) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (e > lim) sv[e] = 0xff800000u;
}

__device__ __forceinline__ bool odd_bf16(uint32_t h) { return (h & 0x7f80u) == 0x7f80u; }

// Makes a sub-block of V (two halves of 64 keys x 64 features, each key's 128
// bytes in a row) safe to multiply with p = 0: rows from `seen_end` on are no
// keys of this tile and become zeros, and in rows from `all_end` on, which some
// of the tile's rows do not see, elements that are not finite become zero.
// Returns whether there were such elements. One warp; swizzling moves 16-byte
// pieces inside a row only.
__device__ __forceinline__ bool guard_v(uint8_t* sub, int all_end, int seen_end, int lane) {
  bool odd = false;
  for (int row = max(all_end, 0) + (lane >> 3); row < kSubKeys; row += 4) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint4* at = reinterpret_cast<uint4*>(sub + half * kSubHalf + row * 128 + (lane & 7) * 16);
      if (row >= seen_end) {
        *at = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      uint4 x = *at;
      uint32_t m = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) m = __vmaxu2(m, (&x.x)[e] & 0x7fff7fffu);
      if ((m & 0xffffu) >= 0x7f80u || (m >> 16) >= 0x7f80u) {
        odd = true;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t& w = (&x.x)[e];
          if (odd_bf16(w)) w &= 0xffff0000u;
          if (odd_bf16(w >> 16)) w &= 0x0000ffffu;
        }
        *at = x;
      }
    }
  }
  return odd;
}

__global__ void __launch_bounds__(kThreads, 2)
    packed_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv, const __grid_constant__ PackedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* sK = base + kTile;             // K sub-block slots 0, 1
  uint8_t* sV = base + kTile + 2 * kSub;  // V sub-block slots 0, 1
  __shared__ Bars bars;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    bars.abort = 0;
    bars.redo = 0;
    bars.odd_v = 0;
    bars.found = 0;
    mbar_init(&bars.q_full, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.k_full[s], 1);
      mbar_init(&bars.v_full[s], 1);
      mbar_init(&bars.v_empty[s], 1);
      mbar_init(&bars.s_full[s], 1);
      mbar_init(&bars.p_full[s], kSoftmaxWarps);
    }
    mbar_init(&bars.o_full, 1);
    mbar_init(&bars.drain, 1);
    for (int qq = 0; qq < 4; ++qq) mbar_init(&bars.xbar[qq], 64);
    fence_mbar_init();
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  grid_dep_wait();
  // blockIdx.x = ((kv head, head chunk) * bound + rank) * splits + split
  const int split = static_cast<int>(blockIdx.x) % a.splits, item = static_cast<int>(blockIdx.x) / a.splits;
  const int rank = item % a.bound, gc = item / a.bound;
  find_tile(a, rank, reinterpret_cast<int2*>(sK), bars);  // ends with a barrier
  if (bars.found == 0) return;
  const Tile tile = bars.tile;
  const int sub0 = split * a.split_subs;
  const int nsub = (split == a.splits - 1 ? tile.cost : min(tile.cost, sub0 + a.split_subs)) - sub0;
  if (split > 0 && nsub <= 0) return;
  const bool partial = min(a.splits, div_up(tile.cost, a.split_subs)) > 1;
  const int g = gc / a.chunks, hc = (gc % a.chunks) * a.hp;  // kv head; first head of the tile inside the group
  const int off = tile.nk - tile.nq;
  // the tile's first row sees the keys [0, off + t0], its last one those below kv_end
  const int kv_all = max(off + tile.t0 + 1, 0), kv_end = off + min(tile.t0 + a.tokens, tile.nq);
  // sub-blocks from here on (of this CTA's) are seen in part by some rows
  const int guarded = min(max(kv_all / kSubKeys - sub0, 0), max(nsub, 0));
  if (warp == kMmaWarp) {
    tmem_alloc(&bars.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  fence_async_shared();  // find_tile's use of the K slots comes before the copies into them
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();  // not before every CTA of this grid has its TMEM: the next kernel may ask for some
  const uint32_t tmem = bars.tmem_base;

  // Phase counters that persist across passes (each role counts its own).
  SlotCounts kn, vn;  // TMA: loads issued per slot; MMA: loads consumed per slot
  SlotCounts pn;      // MMA: p_full phases consumed per slot
  SlotCounts sn;      // softmax: s_full phases consumed per slot
  uint32_t drains = 0u, o_phase = 0u, x_phase = 0u;
  // Softmax state (per thread: one row, one 32-column chunk).
  const int quarter = warp & 3, chunk = warp >> 2;
  const int r = quarter * 32 + lane;
  const int t_row = tile.t0 + r / a.hp, h_row = hc + r % a.hp;  // query of the sequence, head of the group
  const bool live = r < a.hp * a.tokens && t_row < tile.nq && h_row < a.group;
  const int pos = live ? off + t_row : -1;  // the row's last key
  const bool warp_live = __any_sync(0xffffffffu, live);
  const int pair_bar = 1 + quarter;
  auto row_max = [&](float partial_max, float& m) -> bool {
    bars.xmax[chunk][r] = partial_max;
    mbar_arrive(&bars.xbar[quarter]);
    const bool got = warp_wait(&bars.xbar[quarter], x_phase & 1u, &bars.abort);
    ++x_phase;
    m = fmaxf(bars.xmax[0][r], bars.xmax[1][r]);
    return got;
  };
  const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
  float m_ref = 0.f, l = 0.f;
  bool ok = true;

  int mode = kFast;
  for (int pass = 0; pass < 3 && nsub > 0; ++pass) {
    mode = pass;
    if (warp == kTmaWarp) {
      if (lane == 0) {
        if (pass == 0) {
          if (CRISP_CHECK(tile.q0 + tile.t0 < a.total_q && g * a.group + hc < a.hq, a.status, 0x812)) {
            mbar_arrive_expect_tx(&bars.q_full, static_cast<uint32_t>(a.hp * a.tokens) * 256u);
            tma_load_3d(sQ, &tq, &bars.q_full, 0, g * a.group + hc, tile.q0 + tile.t0);
            tma_load_3d(sQ + kHalf, &tq, &bars.q_full, 64, g * a.group + hc, tile.q0 + tile.t0);
          } else {
            mbar_arrive(&bars.q_full);
          }
        }
        // K runs one sub-block ahead of V: the order in which the products free their slots.
        auto load = [&](bool is_k, int t) -> bool {
          const int s = t & 1;
          uint64_t* empty = is_k ? &bars.s_full[s] : &bars.v_empty[s];
          uint64_t* full = is_k ? &bars.k_full[s] : &bars.v_full[s];
          SlotCounts& cnt = is_k ? kn : vn;
          if (!mbar_wait(empty, cnt.parity(s) ^ 1u, &bars.abort)) {
            fail(&bars.abort, a.status, is_k ? 0x821 : 0x822);
            return false;
          }
          cnt.inc(s);
          uint8_t* dst = (is_k ? sK : sV) + s * kSub;
          const CUtensorMap* map = is_k ? &tk : &tv;
          const int row = tile.k0 + (sub0 + t) * kSubKeys;
          if (CRISP_CHECK(row < a.total_k && g * a.group < a.hq, a.status, 0x814)) {
            mbar_arrive_expect_tx(full, kSub);
            tma_load_3d(dst, map, full, 0, row, g);
            tma_load_3d(dst + kSubHalf, map, full, 64, row, g);
          } else {
            mbar_arrive(full);
          }
          return true;
        };
        bool go = true;
        for (int t = 0; go && t <= nsub; ++t) {
          if (t < nsub) go = load(true, t);
          if (go && t >= 1 && mode != kMaxOnly) go = load(false, t - 1);
        }
        // Every copy issued has landed before the pass ends. Bounded waits that ignore the abort flag.
        const int never = 0;
        mbar_wait(&bars.q_full, 0, &never);
        for (int s = 0; s < 2; ++s) {
          if (kn.any(s)) mbar_wait(&bars.k_full[s], kn.parity(s) ^ 1u, &never);
          if (vn.any(s)) mbar_wait(&bars.v_full[s], vn.parity(s) ^ 1u, &never);
        }
      }
    } else if (warp == kMmaWarp) {
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kSubKeys, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, 128, false, true);
      const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk0 = sdesc_sw128(smem_u32(sK), 16, 1024), dk1 = dk0 + (kSub >> 4);
      const uint64_t dv0 = sdesc_sw128(smem_u32(sV), kSubHalf, 1024), dv1 = dv0 + (kSub >> 4);
      // S_s = Q K_s^T into buffer s (the slot as a constant: its descriptors and
      // barriers then take no instruction between the products).
      auto issue_qk = [&](auto slot) -> bool {
        constexpr int s = decltype(slot)::value;
        if (!mbar_wait(&bars.k_full[s], kn.parity(s), &bars.abort)) return false;
        kn.inc(s);
        tc_fence_after();
        umma_qk_x8<(kHalf >> 4), (kSubHalf >> 4)>(tmem + s * kSubKeys, dq, s ? dk1 : dk0, idesc_qk);
        umma_commit(&bars.s_full[s]);
        return true;
      };
      // O += P_s V_s; V_s has landed.
      auto issue_pv = [&](auto slot, bool first) -> bool {
        constexpr int s = decltype(slot)::value;
        if (!mbar_wait(&bars.p_full[s], pn.parity(s), &bars.abort)) return false;
        pn.inc(s);
        tc_fence_after();
        umma_pv_x4(tmem + 128, tmem + s * kSubKeys + 16, s ? dv1 : dv0, idesc_pv, first ? 0u : 1u);
        umma_commit(&bars.v_empty[s]);
        return true;
      };
      auto wait_v = [&](int s) -> bool {
        if (!mbar_wait(&bars.v_full[s], vn.parity(s), &bars.abort)) return false;
        vn.inc(s);
        return true;
      };
      // Sub-block i's second product, then the scores of sub-block i + 2.
      auto issue_step = [&](auto slot, int i) -> bool {
        if (!issue_pv(slot, i == 0)) return false;
        return i + 2 >= nsub || issue_qk(slot);
      };
      constexpr std::integral_constant<int, 0> s0;
      constexpr std::integral_constant<int, 1> s1;
      bool go = true;
      if (lane == 0) {
        go = mbar_wait(&bars.q_full, 0, &bars.abort);
        if (!go) fail(&bars.abort, a.status, 0x823);
      }
      if (mode != kMaxOnly) {
        // QK(0) QK(1) | PV(0) QK(2) PV(1) QK(3) | ...: the QK that writes buffer s
        // is issued right behind the PV that reads P_s from it (the products of
        // one thread execute in order). The sub-blocks that every row sees whole
        // take lane 0 alone; before each of the others the warp looks through
        // its V, while the softmax warps work on its scores.
        if (lane == 0) {
          go = go && issue_qk(s0) && (nsub < 2 || issue_qk(s1));
          for (int i = 0; go && i < guarded; i += 2) {
            go = wait_v(0) && issue_step(s0, i);
            if (go && i + 1 < guarded) go = wait_v(1) && issue_step(s1, i + 1);
          }
        }
        for (int i = guarded; i < nsub; ++i) {
          const int s = i & 1;
          if (lane == 0) go = go && wait_v(s);
          go = __shfl_sync(0xffffffffu, go ? 1 : 0, 0) != 0;
          if (!go) break;
          const int key0 = (sub0 + i) * kSubKeys;
          if (guard_v(sV + s * kSub, kv_all - key0, kv_end - key0, lane)) *reinterpret_cast<volatile int*>(&bars.odd_v) = 1;
          fence_async_shared();
          __syncwarp();
          if (lane == 0) go = s ? issue_step(s1, i) : issue_step(s0, i);
        }
        if (lane == 0 && go) umma_commit(&bars.o_full);
      } else if (lane == 0) {
        // Scores only: a buffer is free again once its scores have been read.
        for (int i = 0; go && i < nsub; ++i) {
          const int s = i & 1;
          if (i >= 2) {
            go = mbar_wait(&bars.p_full[s], pn.parity(s), &bars.abort);
            if (go) pn.inc(s);
          }
          if (go) go = s ? issue_qk(s1) : issue_qk(s0);
        }
        for (int s = 0; go && s < 2 && s < nsub; ++s) {
          go = mbar_wait(&bars.p_full[s], pn.parity(s), &bars.abort);
          if (go) pn.inc(s);
        }
      }
      if (lane == 0) {
        if (!go) fail(&bars.abort, a.status, 0x824);
        // Every product issued in this pass has completed before it ends (a
        // bounded wait that ignores the abort flag: TMEM is released later).
        umma_commit(&bars.drain);
        const int never = 0;
        if (!mbar_wait(&bars.drain, drains & 1u, &never)) fail(&bars.abort, a.status, 0x826);
        ++drains;
      }
    } else {
      const uint32_t s_col = static_cast<uint32_t>(chunk * 32);
      float mx = -INFINITY;  // max-only pass: running raw max of this chunk
      if (mode != kMaxOnly) l = 0.f;
      for (int i = 0; ok && i < nsub; ++i) {
        const int s = i & 1;
        if (!warp_wait(&bars.s_full[s], sn.parity(s), &bars.abort)) {
          if (lane == 0) fail(&bars.abort, a.status, 0x827);
          ok = false;
          break;
        }
        sn.inc(s);
        if (!warp_live) {  // rows of no token: what P holds there reaches no other row
          if (lane == 0) mbar_arrive(&bars.p_full[s]);
          continue;
        }
        tc_fence_after();
        uint32_t sv[32];
        tmem_ld32(tmem + lane_addr + s * kSubKeys + s_col, sv);
        if (i >= guarded) mask_from32(pos - (sub0 + i) * kSubKeys - chunk * 32, sv);
        if (mode == kMaxOnly) {
          mx = fmaxf(mx, max32(sv));
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.p_full[s]);
          continue;
        }
        if (mode == kFast && i == 0) {
          // First sub-block: its exact row max (both chunks) is the reference.
          float m0;
          if (!row_max(max32(sv), m0)) {
            if (lane == 0) fail(&bars.abort, a.status, 0x829);
            ok = false;
            break;
          }
          m_ref = m0 > -INFINITY ? m0 * a.c_log2 : 0.f;  // a row that sees nothing here: every p is 0
        }
        uint32_t pk[16];
        float cs = 0.f;
        p_exp32(sv, a.c_log2, -m_ref, pk, cs);
        tmem_st16(tmem + lane_addr + s * kSubKeys + s_col + 16, pk);
        l += cs;
        if (mode == kFast && live && cs > kOverflowSum) *reinterpret_cast<volatile int*>(&bars.redo) = 1;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[s]);
      }
      if (mode == kMaxOnly) {
        if (warp_live) {
          float m1;
          if (!row_max(mx, m1)) {
            if (lane == 0) fail(&bars.abort, a.status, 0x82a);
            ok = false;
          }
          m_ref = m1 > -INFINITY ? m1 * a.c_log2 : 0.f;
        }
      } else if (ok) {
        // O is final once every PV of the pass has completed.
        if (!warp_wait(&bars.o_full, o_phase & 1u, &bars.abort)) {
          if (lane == 0) fail(&bars.abort, a.status, 0x828);
          ok = false;
        }
        ++o_phase;
        tc_fence_after();
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // After the fast pass, a marked CTA runs the max-only and fixed passes.
    const bool stop = *reinterpret_cast<volatile int*>(&bars.abort) != 0;
    if (stop || (pass == kFast && *reinterpret_cast<volatile int*>(&bars.redo) == 0) || pass == kFixed) break;
  }

  if (warp < kSoftmaxWarps && warp_live) {
    const uint32_t o_addr = tmem + lane_addr + 128 + chunk * 64;
    const bool have = ok && nsub > 0 && *reinterpret_cast<volatile int*>(&bars.abort) == 0;
    const bool odd = *reinterpret_cast<volatile int*>(&bars.odd_v) != 0;
    bars.xsum[chunk][r] = l;
    named_bar_sync(pair_bar, 64);
    const float l_row = have ? bars.xsum[0][r] + bars.xsum[1][r] : 0.f;
    const int tok = tile.q0 + t_row, head = g * a.group + h_row;
    const int64_t row_index = static_cast<int64_t>(tok) * a.hq + head;
    uint4* stg = reinterpret_cast<uint4*>(sK + warp * (32 * 128));  // 32 rows x 128 B
    const float inv_l = partial ? 1.f : (l_row != 0.f ? 1.0f / l_row : 0.f);
    float* part = a.part + (static_cast<int64_t>(split) * a.total_q * a.hq + row_index) * kD + chunk * 64;
#pragma unroll 1
    for (int cc = 0; cc < 2; ++cc) {
      uint32_t v[32];
      if (have) {
        tmem_ld32(o_addr + cc * 32, v);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = 0u;
      }
      if (odd && live) {
        // What guard_v took out, for the rows that see it: their p is above zero.
        const int last = min(pos, (sub0 + nsub) * kSubKeys - 1);
        for (int j = max(kv_all, sub0 * kSubKeys); j <= last; ++j) {
          const __nv_bfloat16* at = a.v + g * a.v_hs + (tile.k0 + j) * a.v_ts + chunk * 64 + cc * 32;
          for (int e = 0; e < 32; ++e) {
            const float x = __bfloat162float(at[e]);
            if (!(fabsf(x) < INFINITY)) v[e] = __float_as_uint(__uint_as_float(v[e]) + x);
          }
        }
      }
      if (partial) {
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(part + cc * 32 + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
        continue;
      }
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
        uint4 u;
        u.x = pack_bf16x2(__uint_as_float(v[q4 * 8 + 0]) * inv_l, __uint_as_float(v[q4 * 8 + 1]) * inv_l);
        u.y = pack_bf16x2(__uint_as_float(v[q4 * 8 + 2]) * inv_l, __uint_as_float(v[q4 * 8 + 3]) * inv_l);
        u.z = pack_bf16x2(__uint_as_float(v[q4 * 8 + 4]) * inv_l, __uint_as_float(v[q4 * 8 + 5]) * inv_l);
        u.w = pack_bf16x2(__uint_as_float(v[q4 * 8 + 6]) * inv_l, __uint_as_float(v[q4 * 8 + 7]) * inv_l);
        const int c16 = cc * 4 + q4;  // 16-byte chunk of this warp's 128-byte row part
        stg[lane * 8 + (c16 ^ (lane & 7))] = u;
      }
    }
    if (partial) {
      if (live && chunk == 0)
        a.part_ml[static_cast<int64_t>(split) * a.total_q * a.hq + row_index] =
            make_float2(l_row != 0.f ? m_ref : -INFINITY, l_row);
    } else {
      // Staged per warp so that each store instruction writes four 128-byte row segments.
      const int64_t at = live ? head * a.o_hs + tok * a.o_ts + chunk * 64 : -1;
      __syncwarp();
      const int c16 = lane & 7;
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int R = it * 4 + (lane >> 3);
        const int64_t to = __shfl_sync(0xffffffffu, at, R);
        // (to < 0: a row of no token)
        if (to >= 0) *reinterpret_cast<uint4*>(a.out + to + c16 * 8) = stg[R * 8 + (c16 ^ (R & 7))];
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// The rows of split tiles: out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s
// with M the largest reference m_s, in the order of the splits. A warp per row.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(kJoinWarps * 32) packed_join_kernel(const __grid_constant__ PackedArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(a.total_q) * a.hq;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  grid_dep_launch();
  grid_dep_wait();
  if (row >= rows) return;
  const int tok = static_cast<int>(row / a.hq), head = static_cast<int>(row % a.hq);
  // the last sequence that starts at or before the token
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.cu_q[mid] <= tok) lo = mid;
    else hi = mid;
  }
  bool ok;
  const int2 n = seq_lens(a, lo, ok);
  const int t = tok - a.cu_q[lo];
  if (t < 0 || t >= n.x) return;
  const int cost = tile_cost(n.x, n.y, t / a.tokens * a.tokens, a.tokens);
  const int ns = min(a.splits, div_up(cost, a.split_subs));
  if (ns <= 1) return;  // written by the tile's only CTA
  float top = -INFINITY;
  for (int s = lane; s < ns; s += 32) {
    const float2 ml = a.part_ml[s * rows + row];
    if (ml.y != 0.f) top = fmaxf(top, ml.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  const float* part = a.part + row * kD + lane * 4;
#pragma unroll 4
  for (int s = 0; s < ns; ++s) {
    const float2 ml = a.part_ml[s * rows + row];
    const float4 o = *reinterpret_cast<const float4*>(part + s * rows * kD);
    if (ml.y == 0.f) continue;
    const float w = ex2_approx(ml.x - top);
    l = fmaf(ml.y, w, l);
    acc.x = fmaf(o.x, w, acc.x);
    acc.y = fmaf(o.y, w, acc.y);
    acc.z = fmaf(o.z, w, acc.z);
    acc.w = fmaf(o.w, w, acc.w);
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<uint2*>(a.out + head * a.o_hs + tok * a.o_ts + lane * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

// Heads of a tile: all of a group where they fill 128 rows well, else the
// fewest tiles of equal parts within a tenth of the fewest rows a query can
// take (a group of 65 heads takes 5 tiles of 13 heads x 9 queries, not one of 65
// rows; one of 7 stays whole, 18 queries and 126 rows).
int tile_heads(int group) {
  auto rows = [&](int chunks) {  // tiles per query
    const int hp = div_up(group, chunks);
    return hp > kB ? 1e9 : static_cast<double>(div_up(group, hp)) / (kB / hp);
  };
  double best = 1e9;
  for (int c = 1; c <= group; ++c) best = std::min(best, rows(c));
  int c = 1;
  while (rows(c) > 1.1 * best) ++c;
  return div_up(group, c);
}

struct PackedPlan {
  int hp, chunks, tokens, bound, splits, split_subs;
};

// Tiles are split over CTAs where there are not enough of them for two CTAs on
// each SM, into parts of eight sub-blocks or more (below that the second kernel
// and a CTA's own start and end cost more than the split saves).
PackedPlan packed_plan(const crisp_packed& p) {
  PackedPlan L{};
  const int group = p.hq / p.hkv;
  L.hp = tile_heads(group);
  L.chunks = div_up(group, L.hp);
  L.tokens = kB / L.hp;
  const int64_t bound = (static_cast<int64_t>(p.total_q) + static_cast<int64_t>(p.batch) * (L.tokens - 1)) / L.tokens;
  L.bound = static_cast<int>(std::min<int64_t>(bound, p.total_q));
  const int longest = p.max_k > 0 ? std::min(p.max_k, p.total_k) : p.total_k;
  const int cost = std::max(1, div_up(std::min(longest, kMaxSeq), kSubKeys));
  const int64_t items = static_cast<int64_t>(L.bound) * L.chunks * p.hkv;
  L.splits = items > 0 ? static_cast<int>(std::min<int64_t>(std::max<int64_t>(kPackedCtas / items, 1), std::max(cost / 8, 1))) : 1;
  L.split_subs = div_up(cost, L.splits);
  L.splits = div_up(cost, L.split_subs);
  return L;
}

}  // namespace

PackedLayout packed_layout(const crisp_packed& p) {
  const PackedPlan plan = packed_plan(p);
  const size_t rows = plan.splits > 1 ? static_cast<size_t>(p.total_q) * p.hq * plan.splits : 0;
  PackedLayout L{};
  size_t o = align_up(sizeof(DevStatus));
  L.part = o;    o = align_up(o + rows * kD * sizeof(float));
  L.part_ml = o; o = align_up(o + rows * sizeof(float2));
  L.total = o;
  return L;
}

void packed_q_box(const crisp_packed& p, int* heads, int* tokens) {
  const PackedPlan L = packed_plan(p);
  *heads = L.hp;
  *tokens = L.tokens;
}

cudaError_t launch_packed(const crisp_packed& p, const TmaMaps& maps, float scale, const crisp_tokens& v,
                          const crisp_tokens& out, char* ws, cudaStream_t st) {
  const PackedPlan plan = packed_plan(p);
  const PackedLayout L = packed_layout(p);
  PackedArgs a{};
  a.cu_q = p.cu_q;
  a.cu_k = p.cu_k;
  a.batch = p.batch;
  a.total_q = p.total_q;
  a.total_k = p.total_k;
  a.hq = p.hq;
  a.group = p.hq / p.hkv;
  a.hp = plan.hp;
  a.chunks = plan.chunks;
  a.tokens = plan.tokens;
  a.inv_tokens = plan.tokens == 1 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) + plan.tokens - 1) / plan.tokens);
  a.bound = plan.bound;
  a.splits = plan.splits;
  a.split_subs = plan.split_subs;
  a.c_log2 = scale * 1.4426950408889634f;
  a.out = static_cast<__nv_bfloat16*>(const_cast<void*>(out.data));
  a.o_hs = out.head_stride;
  a.o_ts = out.tok_stride;
  a.v = static_cast<const __nv_bfloat16*>(v.data);
  a.v_hs = v.head_stride;
  a.v_ts = v.tok_stride;
  a.part = reinterpret_cast<float*>(ws + L.part);
  a.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  a.status = reinterpret_cast<DevStatus*>(ws);
  cudaError_t e = cudaFuncSetAttribute(packed_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  // (a tile holds more than 64 of at most 2^24 x 4096 rows: below 2^31)
  const unsigned grid = static_cast<unsigned>(plan.bound) * plan.chunks * p.hkv * plan.splits;
  e = launch_dependent(packed_kernel, dim3(grid), kThreads, kSmemBytes, st, maps.q, maps.k64, maps.v, a);
  if (e != cudaSuccess || plan.splits == 1) return e;
  const int64_t rows = static_cast<int64_t>(p.total_q) * p.hq;
  return launch_dependent(packed_join_kernel, dim3(static_cast<unsigned>((rows + kJoinWarps - 1) / kJoinWarps)),
                          kJoinWarps * 32, 0, st, a);
}

}  // namespace crisp
