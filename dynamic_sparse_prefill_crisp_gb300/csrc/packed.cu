// Causal GQA softmax attention over packed sequences on the 5th-generation
// tensor cores. Sequence b has the query rows [cu_q[b], cu_q[b+1]) and the key
// rows [cu_k[b], cu_k[b+1]) of packed tensors; with off = k_len - q_len its
// query i sees its keys j <= off + i.
//
// A tile is `tokens` consecutive queries of one sequence times `hp` query heads
// of one kv head (128 rows at most, token by token): a kv head's keys are read
// once for its whole group, and a short prompt fills a tile with its heads
// where rows of one head alone would leave it empty. A block of the grid stands
// for a tile (or a part of one, see below): the sequences of most keys first, each
// from its last tile to its first, the kv heads side by side or in turn
// (packed_plan). A block's tile follows from the lengths, so that no schedule has
// to be made or kept. (In the order of all tiles' keys, the search for a tile took
// 5000 cycles, four sub-blocks.)
//
// Two CTAs stay on each SM and take over blocks that have not started, one
// ahead: the next tile's Q and first K and V are on their way while this one's
// softmax and epilogue run. Short prompts need that (256 of up to 300 tokens,
// 28/4 heads: 121 us, 5.3 TB/s; a CTA per tile, whose start, loads and end came
// one after the other, 340 us).
//
// Long prompts are bound by the tensor pipe at the rate of its 64-key products (a
// product's operands come from shared memory at 128 bytes a cycle, 48 cycles where
// 64 keys' arithmetic takes 32): 16k tokens of 32/8 heads take 1.22 ms, 1800
// TFLOP/s, a sub-block 1225 cycles a CTA and 612 an SM (1.42 ms in calls back to
// back, which the power cap holds at 1.5 GHz).
//
// The products are csrc/attention.cu's: 64-key sub-blocks, two score buffers in
// TMEM, the first sub-block's row maximum as the reference. What differs:
//  - sub-blocks start at any key row, so the rows behind a sequence's last key
//    are another sequence's, and of the last ones some rows of the tile see a
//    part. Masked scores give p = 0, which leaves V out as long as V is finite: a
//    result that is not says that it may not have been, and the tile is done
//    again with such elements taken out of the product and added to the rows that
//    see them (to look through V first took 5000 cycles of a tile's 60000 in a 4k
//    prompt).
//  - a tile is done again, as two more items of the CTA, too where a row's sum
//    passes 2^64 or stays under 2^-64: the exact row maxima first, then the sums at
//    those. (A sum is small where the first sub-block's scores are all -inf, and the
//    reference 0 is none of the row's scores: exponentials below 2^-126 are zeros, of
//    a sum of 2^-64 at most 2^-42 over 2^20 keys, of a smaller one up to all of it.)
//  - when there are too few tiles for the GPU, a tile's keys are split over
//    several blocks, whose unfinished rows a second kernel joins in a fixed order.
//
// Warp roles: 0-7 softmax + epilogue, 8 finds tiles and issues TMA, 9 issues the
// products (TMEM owner).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cuda_bf16.h>

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
constexpr int kRing = 4;                                  // items on their way through a CTA
constexpr int kAskAhead = 4;                              // sub-blocks before the end at which the next block is asked for
constexpr uint32_t kTmemCols = 256;                       // S/P [0,64) and [64,128), O [128,256)

// What the CTA does with a tile: kFast; then, where a result is not finite,
// kGuarded, the same but for a look through V; and where sums left their range (or
// kGuarded's results are not finite where V is), kMaxOnly and kFixed, with that look too.
enum Mode : int { kFast, kGuarded, kMaxOnly, kFixed, kEnd };
constexpr uint32_t batch_bytes(int batch) { return batch * 6u + 8u; }  // ranks and order

constexpr float kSmallSum = 0x1p-64f;  // sum of a row that sees keys, below which the row is done again

// Room below fp32's largest number: p of a tile that is done again at its row maxima is
// at most 2^-24 (and the parts' weights of a join too), so that sums of p v over 2^20
// keys stay finite whatever finite v is. (What that takes below 2^-126 is a 2^-102 of the
// largest.)
constexpr float kHeadroom = 24.f;

enum Redo : int { kNotFinite = 1, kOverflow = 2 };

struct PackedArgs {
  const int32_t *cu_q, *cu_k;
  int batch, total_q, total_k, hq, hkv, group;
  int hp, chunks;         // heads of a tile; tiles that a group's heads take
  int tokens;             // queries of a tile
  uint32_t inv_tokens;    // ceil(2^32 / tokens), 0 for one token
  int heads_log2;         // kv heads (times chunks) that run side by side
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

// A tile, or one split of it, on its way through the CTA.
struct Item {
  int mode;
  int q0, k0;        // the sequence's first rows
  int nq, nk;
  int t0;            // the tile's first query
  int g, hc;         // kv head; first head of the tile inside its group
  int split;
  int sub0, nsub;    // sub-blocks [sub0, sub0 + nsub) of those the tile sees
  int partial;       // other splits hold the rest
};

constexpr int kTaken = 3 * kD / 32, kOddWords = kTaken + 1;

struct Shared {
  uint64_t q_full, q_empty;
  uint64_t k_full[2], v_full[2], v_empty[2];  // a K slot is free again once s_full of its sub-block completes
  uint64_t s_full[2], p_full[2];
  uint64_t o_full, o_empty;
  uint64_t item_full[kRing], item_empty[kRing];
  uint64_t next, drain;
  uint64_t xbar[4];      // per lane quarter: both warps have posted a value
  uint4 answer;          // about a block to take over
  uint32_t tmem_base;
  int abort;
  int redo[kRing];       // Redo bits: the slot's item has to be done again
  uint32_t odd_v[kRing][kOddWords];  // of the slot's item, where V was looked through: see guard_v
  Item item[kRing], again[kRing];
  float xch[2][2][kB];   // [exchange & 1][chunk][row]: partial row maxima, partial row sums
};

// The phases of the barriers of two slots, and whether a slot was used at all. (Bits,
// not counts: a CTA that stays passes any number of them.)
struct SlotPhases {
  uint32_t v = 0u;
  __device__ __forceinline__ uint32_t parity(int s) const { return v >> s & 1u; }
  __device__ __forceinline__ void inc(int s) { v = (v ^ 1u << s) | 4u << s; }
  __device__ __forceinline__ bool any(int s) const { return (v >> s & 4u) != 0u; }
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

// The lengths of sequence b, or {0, 0} where cu_q or cu_k do not describe one.
__device__ __forceinline__ int2 seq_lens(const PackedArgs& a, int b, bool& ok) {
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  ok = q0 >= 0 && q1 >= q0 && q1 <= a.total_q && k0 >= 0 && k1 >= k0 && k1 <= a.total_k && q1 - q0 <= kMaxSeq &&
       k1 - k0 <= kMaxSeq;
  return ok ? make_int2(q1 - q0, k1 - k0) : make_int2(0, 0);
}

// Whether sequence b begins before the end of an earlier one that is well-formed; then
// it counts as empty, and no row belongs to two. (Only where some are not: else all sums
// ascend.)
__device__ __noinline__ bool begins_early(const PackedArgs& a, int b) {
  for (int c = 0; c < b; ++c) {
    bool ok;
    seq_lens(a, c, ok);
    if (ok && a.cu_q[c + 1] > a.cu_q[b]) return true;
  }
  return false;
}

// Reports sums that are not well-formed, and leaves sequences out that begin early.
// All threads.
__device__ __noinline__ void drop_early(const PackedArgs& a, int* keys, int* tiles) {
  if (blockIdx.x == 0 && threadIdx.x == 0) report_error(a.status, CRISP_ERR_BOUNDS, 0x801);
  for (int b = threadIdx.x; b < a.batch; b += kThreads)
    if (tiles[b] > 0 && begins_early(a, b)) keys[b] = tiles[b] = 0;
  __syncthreads();
}

// The order in which the CTAs take the sequences, most keys first (equal ones: in
// the batch's order): order[i] the i-th one's place in the batch, ranks[i] the
// tiles of those before it, ranks[batch] all tiles. All threads; keys: room for
// the batch's key counts, tiles of each beside them (2 ints a sequence). Each is compared
// with each, full or empty: 4 tokens behind 500 take 9.6 us in a batch of 4, 14 among 256
// slots, 40 among 512, 141 among 1024.
__device__ __forceinline__ void order_sequences(const PackedArgs& a, int* keys, uint16_t* order, int* ranks) {
  const int padded = div_up(a.batch, 4) * 4;
  int* tiles = keys + padded;
  bool all_ok = true;
#pragma unroll 1
  for (int b = threadIdx.x; b < padded; b += kThreads) {
    int2 n = make_int2(0, -1);
    if (b < a.batch) {
      bool ok;
      n = seq_lens(a, b, ok);
      all_ok = all_ok && ok;
    }
    keys[b] = n.y;
    tiles[b] = over_tokens(a, n.x + a.tokens - 1);
  }
  if (__syncthreads_or(!all_ok)) drop_early(a, keys, tiles);
#pragma unroll 1
  for (int b = threadIdx.x; b < a.batch; b += kThreads) {
    const int mine = keys[b];
    int before = 0, ranked = 0;
#pragma unroll 1
    for (int c = 0; c < padded; c += 4) {
      const int4 k = *reinterpret_cast<const int4*>(keys + c), t = *reinterpret_cast<const int4*>(tiles + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int other = (&k.x)[e];
        if (other > mine || (other == mine && c + e < b)) {
          ++before;
          ranked += (&t.x)[e];
        }
      }
    }
    order[before] = static_cast<uint16_t>(b);
    ranks[before] = ranked;
    if (before == a.batch - 1) ranks[a.batch] = ranked + tiles[b];
  }
  __syncthreads();
}

// The item of a block: the tiles of a sequence in descending order of the keys
// they see. Returns false where the block has none.
__device__ __forceinline__ bool find_item(const PackedArgs& a, uint3 block, const uint16_t* order, const int* ranks,
                                          Item& it) {
  const int rank = static_cast<int>(block.x >> a.heads_log2), split = static_cast<int>(block.y);
  const int gc = static_cast<int>((block.z << a.heads_log2) + (block.x & ((1u << a.heads_log2) - 1u)));
  if (rank >= ranks[a.batch] || gc >= a.chunks * a.hkv) return false;
  int lo = 0, hi = a.batch;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ranks[mid] <= rank) lo = mid;
    else hi = mid;
  }
  const int b = order[lo];
  it.q0 = a.cu_q[b];
  it.k0 = a.cu_k[b];
  it.nq = a.cu_q[b + 1] - it.q0;
  it.nk = a.cu_k[b + 1] - it.k0;
  it.t0 = (ranks[lo + 1] - 1 - rank) * a.tokens;
  const int cost = tile_cost(it.nq, it.nk, it.t0, a.tokens);
  it.split = split;
  it.sub0 = split * a.split_subs;
  it.nsub = (split == a.splits - 1 ? cost : min(cost, it.sub0 + a.split_subs)) - it.sub0;
  it.partial = a.splits > 1 && cost > a.split_subs;
  it.g = a.chunks == 1 ? gc : gc / a.chunks;
  it.hc = (gc - it.g * a.chunks) * a.hp;
  return split == 0 || it.nsub > 0;
}

// The phase of a ring slot's barrier at its n-th item.
__device__ __forceinline__ uint32_t ring_parity(int n) { return static_cast<uint32_t>(n / kRing) & 1u; }

// The waits and what follows a failed one are calls: in line, at some thirty
// places, they made the kernel half as large again, and what a tile runs once
// (its search, its epilogue) then came from beyond the instruction cache every time.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  return mbar_wait(bar, parity, abort);
}
__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  return mbar_try_wait(bar, parity) || wait_on(bar, parity, abort);
}
__device__ __forceinline__ bool await_warp(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  return __all_sync(0xffffffffu, await(bar, parity, abort));
}
__device__ __noinline__ void give_up(int* abort, DevStatus* st, uint32_t where) { fail(abort, st, where); }

// One lane of a converged warp, and which. Code under this condition is known to
// run in one lane, and keeps descriptors in uniform registers; under `lane == 0`
// the products took longer to issue than to run (16k tokens, 8/8 heads: 320 us,
// 370 so).
__device__ __forceinline__ bool elect_lane(int& lane) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync %1|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok), "=r"(lane));
  return ok != 0u;
}
// Keys past the row's last one (columns above lim) -> -inf.
__device__ __forceinline__ void mask_from32(int lim, uint32_t (&sv)[32]) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (e > lim) sv[e] = 0xff800000u;
}

__device__ __forceinline__ bool odd_bf16(uint32_t h) { return (h & 0x7f80u) == 0x7f80u; }
// acc + 0 * w of bf16 pairs: no longer zero once a w was no finite number.
__device__ __forceinline__ void note_odd(uint32_t& acc, uint32_t w) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w), "r"(0u));
}

// Makes a sub-block of V (two halves of 64 keys x 64 features, each key's 128
// bytes in a row) safe to multiply with p = 0: rows from `seen_end` on are no
// keys of this tile and become zeros, and in rows from `all_end` on, which some
// of the tile's rows do not see, elements that are not finite become zero (then
// odd[kTaken] = 1). Bit f % 32 of odd[kind * 4 + f / 32]: a key that all rows see has an
// element of feature f that is infinity, minus infinity or NaN (kind 0, 1, 2). One warp,
// eight lanes a row, eight reads in flight; swizzling moves 16-byte pieces inside a row
// only.
__device__ __noinline__ void guard_v(uint8_t* sub, int all_end, int seen_end, int lane, uint32_t* odd) {
  uint8_t* mine = sub + (lane >> 3) * 128 + (lane & 7) * 16;
#pragma unroll 1
  for (int row0 = 0; row0 < kSubKeys; row0 += 16) {
    uint4 x[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = row0 + 4 * u + (lane >> 3);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint4* at = reinterpret_cast<uint4*>(mine + half * kSubHalf + (row0 + 4 * u) * 128);
        x[u][half] = make_uint4(0u, 0u, 0u, 0u);
        if (row >= seen_end) *at = x[u][half];
        else x[u][half] = *at;
      }
    }
    uint32_t acc = 0u;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int e = 0; e < 4; ++e) note_odd(acc, (&x[u][half].x)[e]);
    if ((acc & 0x7fff7fffu) == 0u) continue;
#pragma unroll 1
    for (int e = 0; e < 4 * 2 * 4; ++e) {  // word by word
      const int u = e >> 3, half = e >> 2 & 1, row = row0 + 4 * u + (lane >> 3);
      uint32_t* at = reinterpret_cast<uint32_t*>(mine + half * kSubHalf + (row0 + 4 * u) * 128) + (e & 3);
      uint32_t w = *at;
      const uint32_t which = (odd_bf16(w) ? 1u : 0u) | (odd_bf16(w >> 16) ? 2u : 0u);
      if (which == 0u) continue;
      if (row < all_end) {
        const int feature = half * 64 + ((lane & 7) ^ (row & 7)) * 8 + (e & 3) * 2;
        for (int x = 0; x < 2; ++x) {
          const uint32_t h = w >> 16 * x & 0xffffu;
          const int kind = (h & 0x7fu) != 0u ? 2 : static_cast<int>(h >> 15);
          if (which >> x & 1u) atomicOr(&odd[kind * 4 + feature / 32], 1u << (feature + x) % 32);
        }
        continue;
      }
      if (which & 1u) w &= 0xffff0000u;
      if (which & 2u) w &= 0x0000ffffu;
      *at = w;
      odd[kTaken] = 1u;
    }
  }
}

// out += v_j over the keys j in [from, last] and 64 columns, where v_j is not
// finite; `to`: those of a row of out, or of an unfinished row.
__device__ __noinline__ void add_odd(const PackedArgs& a, const Item& it, int64_t to, bool partial, int col0, int from,
                                     int last) {
#pragma unroll 1
  for (int j = from; j <= last; ++j) {
    const __nv_bfloat16* vj = a.v + it.g * a.v_hs + (it.k0 + j) * a.v_ts + col0;
#pragma unroll 1
    for (int e = 0; e < 64; ++e) {
      const float x = __bfloat162float(vj[e]);
      if (fabsf(x) < INFINITY) continue;
      if (partial)
        a.part[to + e] += x;
      else
        a.out[to + e] = __float2bfloat16(__bfloat162float(a.out[to + e]) + x);
    }
  }
}

// What is left of a row's 64 columns from col0 on, where its results are not all finite or
// its tile is done again. V may not be finite: the tile is looked through. Where it was,
// and a result that is not finite is not what the keys that all rows see make it
// (infinity, minus infinity, or NaN for NaN and for both), the sums have left fp32's
// range. And what guard_v took out is added for the rows that see it (their p is above
// zero): infinities and NaN, whatever the finite rest is.
__device__ __noinline__ void settle(const PackedArgs& a, const Item& it, int64_t to, int col0, int last, bool odd,
                                    Shared& sh, int slot) {
  const uint32_t* odd_v = sh.odd_v[slot];
  int* redo = &sh.redo[slot];
  const bool partial = it.partial != 0;
  if (odd && it.mode == kFast) atomicOr(redo, kNotFinite);
  if (odd && it.mode == kGuarded) {
    bool found = false;
#pragma unroll 1
    for (int e = 0; e < 64; ++e) {
      const float x = partial ? a.part[to + e] : __bfloat162float(a.out[to + e]);
      if (fabsf(x) < INFINITY) continue;
      auto seen = [&](int kind) { return (odd_v[kind * 4 + (col0 + e) / 32] >> e % 32 & 1u) != 0u; };
      const bool nan = seen(2) || (seen(0) && seen(1));
      found = found || (x != x ? !nan : nan || !seen(x > 0.f ? 0 : 1));
    }
    if (found) atomicOr(redo, kOverflow);
  }
  if (it.mode != kFast && odd_v[kTaken] != 0u)
    add_odd(a, it, to, partial, col0, max(it.nk - it.nq + it.t0 + 1, it.sub0 * kSubKeys),
            min(last, (it.sub0 + it.nsub) * kSubKeys - 1));
}

// kWide: the rows of out allow 32-byte stores.
template <bool kWide>
__global__ void __launch_bounds__(kThreads, 2)
    packed_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv, const __grid_constant__ PackedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base;
  uint8_t* sK = base + kTile;             // K sub-block slots 0, 1
  uint8_t* sV = base + kTile + 2 * kSub;  // V sub-block slots 0, 1
  int* ranks = reinterpret_cast<int*>(base + kTile + 4 * kSub);
  uint16_t* order = reinterpret_cast<uint16_t*>(ranks + a.batch + 1);
  __shared__ Shared sh;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    sh.abort = 0;
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.k_full[s], 1);
      mbar_init(&sh.v_full[s], 1);
      mbar_init(&sh.v_empty[s], 1);
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.p_full[s], kSoftmaxWarps);
    }
    for (int s = 0; s < kRing; ++s) {
      sh.redo[s] = 0;
      mbar_init(&sh.item_full[s], 1);
      mbar_init(&sh.item_empty[s], kSoftmaxWarps + 1);
    }
    mbar_init(&sh.o_full, 1);
    mbar_init(&sh.o_empty, kSoftmaxWarps);
    mbar_init(&sh.next, 1);
    mbar_init(&sh.drain, 1);
    for (int qq = 0; qq < 4; ++qq) mbar_init(&sh.xbar[qq], 64);
    fence_mbar_init();
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  grid_dep_wait();
  order_sequences(a, reinterpret_cast<int*>(sK), order, ranks);
  Item ahead;
  bool found = false;  // ahead is the next item
  // (side by side, and with no waits behind an item that is through: 7.9 us for a
  // prompt of 300 tokens, 8.5 without)
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem_base, kTmemCols);
    tmem_relinquish();
  } else if (warp == kTmaWarp) {
    found = find_item(a, blockIdx, order, ranks, ahead);
  }
  fence_async_shared();  // the K slots' use above comes before the copies into them
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();  // not before every CTA of this grid has its TMEM: the next kernel may ask for some
  const uint32_t tmem = sh.tmem_base;
  // The tile's first row sees the keys [0, all_of), its last one those below end_of.
  auto all_of = [&](const Item& it) { return max(it.nk - it.nq + it.t0 + 1, 0); };
  auto end_of = [&](const Item& it) { return it.nk - it.nq + min(it.t0 + a.tokens, it.nq); };
  // Sub-blocks of the item from here on are seen in part by some rows.
  auto guard_of = [&](const Item& it) { return min(max(all_of(it) / kSubKeys - it.sub0, 0), max(it.nsub, 0)); };

  if (warp == kTmaWarp) {
    int from;  // the lane that issues
    const bool leader = elect_lane(from);
    SlotPhases kn, vn;  // loads issued per slot
    uint32_t loads = 0u, asks = 0u;
    bool asked = false, go = true;
    bool more = true;  // no answer was no yet
    auto send = [&]() {
      mbar_arrive_expect_tx(&sh.next, 16);
      take_block(&sh.answer, &sh.next);
    };
    auto ask = [&]() {
      if (leader) send();
      ++asks;
      asked = true;
    };
    // The next item, passing over blocks that have none.
    auto look_ahead = [&]() {
      while (go && !found && asked) {
        go = await_warp(&sh.next, (asks - 1u) & 1u, &sh.abort);
        asked = false;
        if (!go) return;
        uint3 block;
        more = taken_block(&sh.answer, block);
        fence_async_shared();  // read before the next answer is written
        __syncwarp();
        if (!more) return;
        found = find_item(a, block, order, ranks, ahead);
        if (!found) ask();
      }
    };
    if (!found) ask();
    int retired = 0;  // items known to be through
    int again = 0;    // items that come back
    bool fixed_next = false;
    Item it;
    // The next item is through, and comes back if there is a reason.
    auto retire = [&]() -> bool {
      const int n = retired++;
      if (!await_warp(&sh.item_empty[n % kRing], ring_parity(n), &sh.abort)) return false;
      const int why = *reinterpret_cast<volatile int*>(&sh.redo[n % kRing]);
      if (why != 0) {
        __syncwarp();
        if (leader) {
          sh.again[again] = sh.item[n % kRing];
          sh.again[again].mode = why & kOverflow ? kMaxOnly : kGuarded;
          sh.redo[n % kRing] = 0;
        }
        ++again;
        __syncwarp();
      }
      return true;
    };
    for (int n = 0; go; ++n) {
      while (go && retired <= n - kRing) go = retire();
      if (!go) break;
      if (fixed_next) {
        it.mode = kFixed;
        fixed_next = false;
      } else {
        if (again == 0) look_ahead();
        while (go && again == 0 && !found && retired < n) go = retire();  // one of the last may come back
        if (!go) break;
        if (again > 0) {
          it = sh.again[--again];
          fixed_next = it.mode == kMaxOnly;
        } else {
          it = ahead;
          it.mode = found ? kFast : kEnd;
          found = false;
        }
      }
      if (leader) {
        sh.item[n % kRing] = it;
        if (it.mode != kFast)
          for (uint32_t& w : sh.odd_v[n % kRing]) w = 0u;
        mbar_arrive(&sh.item_full[n % kRing]);
      }
      if (it.mode == kEnd) break;
      // The next block is asked for when this item is about to end: taken earlier, it
      // would wait here while other CTAs run out of work.
      const bool ask_next = it.mode == kFast && more;
      const int ask_at = max(it.nsub - kAskAhead, 0);
      const int head = it.g * a.group + it.hc;
      // K runs one sub-block ahead of V: the order in which the products free their slots.
      auto load = [&](bool is_k, int t) -> bool {
        const int s = t & 1;
        uint64_t* empty = is_k ? &sh.s_full[s] : &sh.v_empty[s];
        uint64_t* full = is_k ? &sh.k_full[s] : &sh.v_full[s];
        SlotPhases& cnt = is_k ? kn : vn;
        if (!await(empty, cnt.parity(s) ^ 1u, &sh.abort)) {
          give_up(&sh.abort, a.status, is_k ? 0x821 : 0x822);
          return false;
        }
        cnt.inc(s);
        uint8_t* dst = (is_k ? sK : sV) + s * kSub;
        const CUtensorMap* map = is_k ? &tk : &tv;
        const int row = it.k0 + (it.sub0 + t) * kSubKeys;
        if (CRISP_CHECK(row < a.total_k && head < a.hq, a.status, 0x814)) {
          mbar_arrive_expect_tx(full, kSub);
          tma_load_3d(dst, map, full, 0, row, it.g);
          tma_load_3d(dst + kSubHalf, map, full, 64, row, it.g);
        } else {
          mbar_arrive(full);
        }
        return true;
      };
      if (leader && it.nsub > 0) {
        if (loads > 0u) go = await(&sh.q_empty, (loads - 1u) & 1u, &sh.abort);
        if (!go) {
          give_up(&sh.abort, a.status, 0x820);
        } else {
          ++loads;
          if (CRISP_CHECK(it.q0 + it.t0 < a.total_q && head < a.hq, a.status, 0x812)) {
            mbar_arrive_expect_tx(&sh.q_full, static_cast<uint32_t>(a.hp * a.tokens) * 256u);
            tma_load_3d(sQ, &tq, &sh.q_full, 0, head, it.q0 + it.t0);
            tma_load_3d(sQ + kHalf, &tq, &sh.q_full, 64, head, it.q0 + it.t0);
          } else {
            mbar_arrive(&sh.q_full);
          }
        }
      }
      // The next item is looked for before the last V is loaded (a short item's
      // first), which is when the producer would wait for the products before.
      const int look_at = it.nsub <= kAskAhead ? min(it.nsub, 1) : it.nsub;
#pragma unroll 1
      for (int t = 0; t <= it.nsub; ++t) {
        if (t == ask_at && ask_next) ask();
        if (leader && go && t < it.nsub) go = load(true, t);
        if (t == look_at) {
          go = __shfl_sync(0xffffffffu, go ? 1 : 0, from) != 0;
          if (it.mode == kFast) look_ahead();
          if (!go) break;
        }
        if (leader && go && t >= 1 && it.mode != kMaxOnly) go = load(false, t - 1);
      }
      go = __shfl_sync(0xffffffffu, go ? 1 : 0, from) != 0;
    }
    if (leader && !go) {
      give_up(&sh.abort, a.status, 0x82b);
      // Everything asked for has landed before the CTA ends (where no wait ran out, all
      // items are through). Bounded waits that ignore the abort flag.
      const int never = 0;
      if (asked) await(&sh.next, (asks - 1u) & 1u, &never);
      if (loads > 0u) await(&sh.q_full, (loads - 1u) & 1u, &never);
      for (int s = 0; s < 2; ++s) {
        if (kn.any(s)) await(&sh.k_full[s], kn.parity(s) ^ 1u, &never);
        if (vn.any(s)) await(&sh.v_full[s], vn.parity(s) ^ 1u, &never);
      }
    }
  } else if (warp == kMmaWarp) {
    int from;  // the lane that issues
    const bool leader = elect_lane(from);
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kSubKeys, false, false);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, 128, false, true);
    const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dk0 = sdesc_sw128(smem_u32(sK), 16, 1024);       // slot 0; slot 1 behind it
    const uint64_t dv0 = sdesc_sw128(smem_u32(sV), kSubHalf, 1024);
    SlotPhases kn, vn, pn;               // loads and p_full phases consumed per slot
    uint32_t q_items = 0u, o_items = 0u;  // items with products; with second products
    bool go = true;
    for (int n = 0;; ++n) {
      if (leader) go = go && await(&sh.item_full[n % kRing], ring_parity(n), &sh.abort);
      go = __shfl_sync(0xffffffffu, go ? 1 : 0, from) != 0;
      if (!go) break;
      __syncwarp();
      const Item& it = sh.item[n % kRing];
      const int mode = it.mode, nsub = it.nsub;
      if (mode == kEnd) break;
      if (nsub > 0) {
        // in the fast pass V is taken as it is
        const int kv_all = all_of(it) - it.sub0 * kSubKeys, kv_end = end_of(it) - it.sub0 * kSubKeys;
        // S_s = Q K_s^T into buffer s.
        auto issue_qk = [&](int s, int i) -> bool {
          if (!await(&sh.k_full[s], kn.parity(s), &sh.abort)) return false;
          kn.inc(s);
          tc_fence_after();
          umma_qk_x8<(kHalf >> 4), (kSubHalf >> 4)>(tmem + s * kSubKeys, dq, dk0 + s * (kSub >> 4), idesc_qk);
          umma_commit(&sh.s_full[s]);
          if (i == nsub - 1) umma_commit(&sh.q_empty);
          return true;
        };
        auto await_v = [&](int s) -> bool {
          if (!await(&sh.v_full[s], vn.parity(s), &sh.abort)) return false;
          vn.inc(s);
          return true;
        };
        auto await_p = [&](int s) -> bool {
          if (!await(&sh.p_full[s], pn.parity(s), &sh.abort)) return false;
          pn.inc(s);
          return true;
        };
        // O += P_s V_s.
        auto issue_pv = [&](int s, int i) {
          tc_fence_after();
          umma_pv_x4(tmem + 128, tmem + s * kSubKeys + 16, dv0 + s * (kSub >> 4), idesc_pv, i == 0 ? 0u : 1u);
          umma_commit(&sh.v_empty[s]);
        };
        if (leader) go = await(&sh.q_full, q_items & 1u, &sh.abort);
        ++q_items;
        // QK(0) QK(1) | PV(0) QK(2) PV(1) QK(3) | ...: the QK that writes buffer s
        // is issued right behind the PV that reads P_s from it (the products of
        // one thread execute in order).
        if (mode == kFast) {
          if (leader) {
            go = go && issue_qk(0, 0) && (nsub < 2 || issue_qk(1, 1));
            // O is the epilogue's until it has read the last item's
            if (o_items > 0u) go = go && await(&sh.o_empty, (o_items - 1u) & 1u, &sh.abort);
            for (int i = 0; go && i < nsub; ++i) {
              const int s = i & 1;
              go = await_v(s) && await_p(s);
              if (go) issue_pv(s, i);
              if (go && i + 2 < nsub) go = issue_qk(s, i + 2);
            }
          }
        } else {
          // Done again: the warp looks through V where some rows do not see all of a
          // sub-block; or scores only (a buffer is free again once they have been read).
          const bool products = mode != kMaxOnly;
          for (int j = 0; j < nsub + 2; ++j) {
            const int i = j - 2;
            if (i >= 0 && products) {
              if (leader) {
                if (i == 0 && o_items > 0u) go = go && await(&sh.o_empty, (o_items - 1u) & 1u, &sh.abort);
                go = go && await_v(i & 1);
              }
              go = __shfl_sync(0xffffffffu, go ? 1 : 0, from) != 0;
              if (!go) break;
              // every lane that reads V sees its barrier's phase for itself (its next one comes
              // no earlier than the product below)
              const uint32_t phase = __shfl_sync(0xffffffffu, vn.parity(i & 1) ^ 1u, from);
              go = await_warp(&sh.v_full[i & 1], phase, &sh.abort);
              if (!go) break;
              guard_v(sV + (i & 1) * kSub, kv_all - i * kSubKeys, kv_end - i * kSubKeys, lane, sh.odd_v[n % kRing]);
              fence_async_shared();
              __syncwarp();
            }
            if (leader && go) {
              if (i >= 0) {
                go = await_p(i & 1);
                if (go && products) issue_pv(i & 1, i);
              }
              if (go && j < nsub) go = issue_qk(j & 1, j);
            }
          }
        }
        if (mode != kMaxOnly) {
          ++o_items;
          if (leader && go) umma_commit(&sh.o_full);
        }
      }
      __syncwarp();
      if (leader) mbar_arrive(&sh.item_empty[n % kRing]);
    }
    if (leader && !go) {
      give_up(&sh.abort, a.status, 0x824);
      // Every product has completed before TMEM is released (where no wait ran out, all
      // items are through). A bounded wait that ignores the abort flag.
      umma_commit(&sh.drain);
      const int never = 0;
      if (!await(&sh.drain, 0u, &never)) give_up(&sh.abort, a.status, 0x826);
    }
  } else {
    // Softmax and epilogue: per thread one row, one 32-column chunk of the scores.
    const int quarter = warp & 3, chunk = warp >> 2;
    const int r = quarter * 32 + lane;
    const int t_row = r / a.hp, h_row = r % a.hp;  // query of the tile, head of the tile
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_col = static_cast<uint32_t>(chunk * 32);
    SlotPhases sn;  // s_full phases consumed per slot
    uint32_t o_items = 0u, x_phase = 0u;
    float m_ref = 0.f;
    bool ok = true;
    // Posts this row's value of a chunk and takes the other's: {chunk 0's, chunk 1's}.
    auto exchange = [&](float mine) -> float2 {
      // (two buffers: the other warp may not have taken the last exchange's values yet)
      float (*at)[kB] = sh.xch[x_phase & 1u];
      at[chunk][r] = mine;
      mbar_arrive(&sh.xbar[quarter]);
      if (!await_warp(&sh.xbar[quarter], x_phase & 1u, &sh.abort)) {
        if (lane == 0) give_up(&sh.abort, a.status, 0x829);
        ok = false;
      }
      ++x_phase;
      return make_float2(at[0][r], at[1][r]);
    };
    for (int n = 0;; ++n) {
      if (!await_warp(&sh.item_full[n % kRing], ring_parity(n), &sh.abort)) {
        if (lane == 0) give_up(&sh.abort, a.status, 0x825);
        break;
      }
      const Item& it = sh.item[n % kRing];
      const int mode = it.mode, nsub = it.nsub, sub0 = it.sub0;
      if (mode == kEnd) break;
      const bool live = r < a.hp * a.tokens && it.t0 + t_row < it.nq && it.hc + h_row < a.group &&
                        CRISP_CHECK(it.q0 + it.t0 + t_row < a.total_q && it.g * a.group + it.hc + h_row < a.hq &&
                                        it.split < a.splits,
                                    a.status, 0x815);
      const int pos = live ? it.nk - it.nq + it.t0 + t_row : -1;  // the row's last key
      const bool warp_live = __any_sync(0xffffffffu, live);
      const int guarded = guard_of(it);
      float mx = -INFINITY;  // running raw max of this chunk
      float l = 0.f;
      for (int i = 0; ok && i < nsub; ++i) {
        const int s = i & 1;
        if (!await_warp(&sh.s_full[s], sn.parity(s), &sh.abort)) {
          if (lane == 0) give_up(&sh.abort, a.status, 0x827);
          ok = false;
          break;
        }
        sn.inc(s);
        if (!warp_live) {  // rows of no token: what P holds there reaches no other row
          if (lane == 0) mbar_arrive(&sh.p_full[s]);
          continue;
        }
        tc_fence_after();
        uint32_t sv[32];
        tmem_ld32(tmem + lane_addr + s * kSubKeys + s_col, sv);
        if (i >= guarded) mask_from32(pos - (sub0 + i) * kSubKeys - chunk * 32, sv);
        if (mode == kMaxOnly || (mode <= kGuarded && i == 0)) {
          mx = fmaxf(mx, max32(sv));
          if (mode == kMaxOnly) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[s]);
          }
          // The reference: the row max (both chunks) of the first sub-block, or of all.
          if (mode != kMaxOnly || i == nsub - 1) {
            const float2 m = exchange(mx);
            mx = fmaxf(m.x, m.y);
            m_ref = mx > -INFINITY ? mx * a.c_log2 : 0.f;  // a row that sees nothing here: every p is 0
          }
          if (mode == kMaxOnly) continue;
        }
        uint32_t pk[16];
        float cs = 0.f;
        p_exp32(sv, a.c_log2, -m_ref, pk, cs);
        tmem_st16(tmem + lane_addr + s * kSubKeys + s_col + 16, pk);
        l += cs;
        if (mode == kFast && live && cs > kOverflowSum) atomicOr(&sh.redo[n % kRing], kOverflow);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[s]);
      }
      if (!ok) break;
      if (mode != kMaxOnly) {
        // This thread's row: its place in out (or among the unfinished rows).
        const int tok = it.q0 + it.t0 + t_row, head = it.g * a.group + it.hc + h_row;
        const int64_t row_index = static_cast<int64_t>(it.split) * a.total_q * a.hq + static_cast<int64_t>(tok) * a.hq + head;
        const bool partial = it.partial != 0;
        const int64_t to = (partial ? row_index * kD : head * a.o_hs + tok * a.o_ts) + chunk * 64;
        float l_row = 0.f;
        if (nsub > 0) {
          if (warp_live) {
            const float2 sums = exchange(l);
            l_row = sums.x + sums.y;
          }
          // O is final once every second product of the item has completed.
          if (!await_warp(&sh.o_full, o_items & 1u, &sh.abort)) {
            if (lane == 0) give_up(&sh.abort, a.status, 0x828);
            ok = false;
          }
          ++o_items;
          tc_fence_after();
        }
        if (!ok) break;
        if (warp_live) {
          uint32_t odd = 0u;  // no longer zero: the result is no finite number
          auto o_read = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.o_empty);
          };
          const uint32_t o_addr = tmem + lane_addr + 128 + chunk * 64;
          if (partial) {
            uint32_t v[2][32];
            tmem_ld32_async(o_addr, v[0]);
            tmem_ld32_async(o_addr + 32, v[1]);
            tmem_ld_wait32(v[0]);
            tmem_ld_wait32(v[1]);
            o_read();
            if (live) {
              float none = 0.f;
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                  store32(a.part + to + c * 32 + e, v[c] + e, true);
#pragma unroll
                  for (int x = 0; x < 8; ++x) none = fmaf(__uint_as_float(v[c][e + x]), 0.f, none);
                }
              odd = none == 0.f ? 0u : 1u;
              if (chunk == 0) a.part_ml[row_index] = make_float2(l_row != 0.f ? m_ref : -INFINITY, l_row);
            }
          } else {
            // (half a row after the other: both in line are code of every tile that has to
            // be fetched again, 128 us for the short prompts above)
            const float inv_l = l_row != 0.f ? 1.0f / l_row : 0.f;
#pragma unroll 1
            for (int c = 0; c < 64; c += 32) {
              uint32_t v[32], w[16];
              if (nsub > 0) {
                tmem_ld32(o_addr + c, v);
                if (c != 0) o_read();
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = 0u;
              }
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                float lo, hi;
                fmul2(lo, hi, __uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1]), inv_l, inv_l);
                w[x] = pack_bf16x2(lo, hi);
                note_odd(odd, w[x]);
              }
              if (live)
#pragma unroll
                for (int e = 0; e < 16; e += 8) store32(a.out + to + c + 2 * e, w + e, kWide);
            }
          }
          if (live && mode == kFast && l_row < kSmallSum && pos >= sub0 * kSubKeys) atomicOr(&sh.redo[n % kRing], kOverflow);
          const bool not_finite = (odd & 0x7fff7fffu) != 0u;
          if (live && (not_finite || mode != kFast))
            settle(a, it, to, chunk * 64, pos, not_finite, sh, n % kRing);
          __syncwarp();
        } else if (nsub > 0) {
          if (lane == 0) mbar_arrive(&sh.o_empty);
        }
      } else {
        m_ref += kHeadroom;  // (here: added where the maximum is taken, it made long prompts 1 to 4 % slower)
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_empty[n % kRing]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// The rows of split tiles: out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, both times 2^-24,
// with M the largest reference m_s, in the order of the splits. A warp takes kJoinRows
// rows of a token, kJoinAhead parts of each in flight: one row, or two where a warp a
// row would be more than the GPU holds at once (32k rows of whole prompts in halves: 8
// us, 11 with one).
constexpr int kJoinWarps = 4;

template <int kJoinRows, int kJoinAhead>
__global__ void __launch_bounds__(kJoinWarps * 32) packed_join_kernel(const __grid_constant__ PackedArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(a.total_q) * a.hq;
  const int groups = div_up(a.hq, kJoinRows);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  grid_dep_launch();
  grid_dep_wait();
  const int tok = static_cast<int>(unit / groups), head0 = static_cast<int>(unit % groups) * kJoinRows;
  if (tok >= a.total_q) return;
  // The parts of the token's tile, by the lane that finds the sequence that holds it:
  // all are looked at, 32 at a time, because the sums need not ascend where some are not
  // well-formed.
  int ns = -1;
  bool all_ok = true;
#pragma unroll 1
  for (int b0 = 0; ns < 0 && b0 < a.batch; b0 += 32) {
    const int b = min(b0 + lane, a.batch - 1);  // (the last one, more than once)
    bool ok;
    const int2 n = seq_lens(a, b, ok);
    const int t = ok ? tok - a.cu_q[b] : -1;
    all_ok = __all_sync(0xffffffffu, ok) && all_ok;
    const bool holds = t >= 0 && t < n.x && (all_ok || !begins_early(a, b));
    const int cost = tile_cost(n.x, n.y, t / a.tokens * a.tokens, a.tokens);
    ns = __reduce_max_sync(0xffffffffu, holds ? min(a.splits, div_up(cost, a.split_subs)) : -1);
  }
  if (ns <= 1) return;  // written by the tile's only CTA, or no sequence's
  const int64_t row0 = static_cast<int64_t>(tok) * a.hq + head0;
  const int live = min(kJoinRows, a.hq - head0);
  float top[kJoinRows], l[kJoinRows];
  float4 acc[kJoinRows];
#pragma unroll
  for (int r = 0; r < kJoinRows; ++r) {
    top[r] = -INFINITY;
    l[r] = 0.f;
    acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int s = lane; s < ns; s += 32)
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r)
      if (r < live) {
        const float2 ml = a.part_ml[s * rows + row0 + r];
        if (ml.y != 0.f) top[r] = fmaxf(top[r], ml.x);
      }
#pragma unroll
  for (int r = 0; r < kJoinRows; ++r) top[r] = warp_max(top[r]);
  for (int s0 = 0; s0 < ns; s0 += 32) {
    // each lane a part's weights, then all lanes part after part
    float w[kJoinRows];
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
      w[r] = 0.f;
      if (s0 + lane < ns && r < live) {
        const float2 ml = a.part_ml[(s0 + lane) * rows + row0 + r];
        w[r] = ml.y != 0.f ? ex2_approx(ml.x - top[r]) * 0x1p-24f : 0.f;  // kHeadroom
        l[r] += w[r] != 0.f ? ml.y * w[r] : 0.f;
      }
    }
    const float* part = a.part + (s0 * rows + row0) * kD + lane * 4;
    const int parts = min(32, ns - s0);
#pragma unroll 1
    for (int s = 0; s < parts; s += kJoinAhead) {
      float4 o[kJoinAhead][kJoinRows];
#pragma unroll
      for (int e = 0; e < kJoinAhead; ++e)
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r)
          if (s + e < parts && r < live) o[e][r] = *reinterpret_cast<const float4*>(part + ((s + e) * rows + r) * kD);
#pragma unroll
      for (int e = 0; e < kJoinAhead; ++e)
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r) {
          const float ws = __shfl_sync(0xffffffffu, w[r], (s + e) & 31);
          if (s + e < parts && r < live && ws != 0.f) {
            acc[r].x = fmaf(o[e][r].x, ws, acc[r].x);
            acc[r].y = fmaf(o[e][r].y, ws, acc[r].y);
            acc[r].z = fmaf(o[e][r].z, ws, acc[r].z);
            acc[r].w = fmaf(o[e][r].w, ws, acc[r].w);
          }
        }
    }
  }
#pragma unroll
  for (int r = 0; r < kJoinRows; ++r) {
    if (r >= live) break;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
    const float inv = l[r] != 0.f ? 1.f / l[r] : 0.f;
    *reinterpret_cast<uint2*>(a.out + (head0 + r) * a.o_hs + tok * a.o_ts + lane * 4) =
        make_uint2(pack_bf16x2(acc[r].x * inv, acc[r].y * inv), pack_bf16x2(acc[r].z * inv, acc[r].w * inv));
  }
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

}  // namespace

// A tile is split into parts of two sub-blocks or more where that makes the whole
// shorter by this estimate in us, fitted to 115 batches of 1 to 16k queries behind up
// to 130k keys, each with up to 38 parts (its choice is 0.8 % slower than the best of
// them, 50 % at worst and 7 % on average with a plainer one):
//   a sub-block          0.45 with a CTA an SM, 0.6 with two, 0.72 with CTAs that go on
//   the CTAs' chains     their longest part; with more blocks than CTAs the mean too
//   the join             0.7, 0.04 a part, 1e-4 a row and 2e-4 a part of a row
// Whole prompts have tiles of every size, of which the long ones are split: half as
// many parts. The lengths are on the device: the sizes that the host knows stand for
// them.
PackedPlan packed_plan(const crisp_packed& p) {
  PackedPlan L{};
  const int group = p.hq / p.hkv;
  L.hp = tile_heads(group);
  L.chunks = div_up(group, L.hp);
  L.tokens = kB / L.hp;
  const int64_t bound = (static_cast<int64_t>(p.total_q) + static_cast<int64_t>(p.batch) * (L.tokens - 1)) / L.tokens;
  L.bound = static_cast<int>(std::min<int64_t>(bound, p.total_q));
  const int longest = std::min(p.max_k > 0 ? std::min(p.max_k, p.total_k) : p.total_k, kMaxSeq);
  // Heads side by side as long as the keys and values of a sequence fill no more
  // than half of L2: then every head's long tiles start before any short one
  // (16k tokens, 8/8 heads: 370 us, 470 head by head).
  const int heads = L.chunks * p.hkv;
  while ((2 << L.heads_log2) <= heads && (int64_t(2) << L.heads_log2) * longest * (4 * kD) <= (int64_t(64) << 20))
    ++L.heads_log2;
  const double batch = std::max(p.batch, 1), q = p.total_q / batch, off = std::max(p.total_k - p.total_q, 0) / batch;
  const double mean = std::max((off + q / 2) / kSubKeys, 0.5), most = std::max(longest / double(kSubKeys), 1.0);
  const double tiles = static_cast<double>(L.bound) * heads, rows = static_cast<double>(p.total_q) * p.hq;
  double best = 0.0;
  L.splits = 1;
  for (int s = 1; s == 1 || (s <= kPackedCtas && most / s >= 2.0); s += 1 + s / 32) {
    const double parts = off > q ? s : (s + 1) / 2.0, part = most / s, blocks = tiles * parts;
    double us = 2 * blocks <= kPackedCtas ? 0.45 * part : 0.6 * part;
    if (blocks > kPackedCtas) us = std::max(us, 0.72 * mean * tiles / kPackedCtas);
    if (s > 1) us += 0.7 + 0.04 * s + rows * (1e-4 + 2e-4 * parts);
    if (s == 1 || us < best) {
      best = us;
      L.splits = s;
    }
  }
  const int cost = div_up(std::max(longest, 1), kSubKeys);
  L.split_subs = div_up(cost, L.splits);
  L.splits = div_up(cost, L.split_subs);
  return L;
}

PackedLayout packed_layout(const crisp_packed& p, const PackedPlan& plan) {
  const size_t rows = plan.splits > 1 ? static_cast<size_t>(p.total_q) * p.hq * plan.splits : 0;
  PackedLayout L{};
  size_t o = align_up(sizeof(DevStatus));
  L.part = o;    o = align_up(o + rows * kD * sizeof(float));
  L.part_ml = o; o = align_up(o + rows * sizeof(float2));
  L.total = o;
  return L;
}

cudaError_t launch_packed(const crisp_packed& p, const PackedPlan& plan, const TmaMaps& maps, float scale,
                          const crisp_tokens& v, const crisp_tokens& out, char* ws, cudaStream_t st) {
  const PackedLayout L = packed_layout(p, plan);
  PackedArgs a{};
  a.cu_q = p.cu_q;
  a.cu_k = p.cu_k;
  a.batch = p.batch;
  a.total_q = p.total_q;
  a.total_k = p.total_k;
  a.hq = p.hq;
  a.hkv = p.hkv;
  a.group = p.hq / p.hkv;
  a.hp = plan.hp;
  a.chunks = plan.chunks;
  a.tokens = plan.tokens;
  a.inv_tokens = plan.tokens == 1 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) + plan.tokens - 1) / plan.tokens);
  a.heads_log2 = plan.heads_log2;
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
  const bool wide = reinterpret_cast<uintptr_t>(out.data) % 32 == 0 && (p.hq == 1 || out.head_stride % 16 == 0) &&
                    (p.total_q == 1 || out.tok_stride % 16 == 0);
  const size_t smem = kSmemBytes + batch_bytes(p.batch);
  // the most that any batch takes, once a device
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if ((allowed.load(std::memory_order_relaxed) & bit) == 0) {
    for (auto* kernel : {packed_kernel<false>, packed_kernel<true>}) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(kSmemBytes + batch_bytes(kMaxBatch)));
      if (e != cudaSuccess) return e;
    }
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  // (heads side by side, tiles), parts, groups of heads; a tile holds more than 64
  // of at most 2^24 x 4096 rows
  const dim3 grid(static_cast<unsigned>(plan.bound) << plan.heads_log2, static_cast<unsigned>(plan.splits),
                  static_cast<unsigned>(div_up(plan.chunks * p.hkv, 1 << plan.heads_log2)));
  e = launch_dependent(wide ? packed_kernel<true> : packed_kernel<false>, grid, kThreads, smem, st, maps.q, maps.k64, maps.v, a);
  if (e != cudaSuccess || plan.splits == 1) return e;
  // two rows a warp where a row each would be more warps than the GPU holds at once
  const int64_t rows = static_cast<int64_t>(p.total_q) * p.hq;
  const bool two = rows > kPackedCtas * 32;
  const int64_t units = two ? static_cast<int64_t>(p.total_q) * div_up(p.hq, 2) : rows;
  const dim3 blocks(static_cast<unsigned>((units + kJoinWarps - 1) / kJoinWarps));
  return two ? launch_dependent(packed_join_kernel<2, 2>, blocks, kJoinWarps * 32, 0, st, a)
             : launch_dependent(packed_join_kernel<1, 4>, blocks, kJoinWarps * 32, 0, st, a);
}

}  // namespace crisp
