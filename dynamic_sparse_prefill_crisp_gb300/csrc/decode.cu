// Attention of a few new tokens over the paged 8-bit cache.
//
// Per kv head the rows are the G query heads times the q_len tokens, up to 32
// of them at a time. One page (128 keys) is one tile; codes kc, vc in e4m3 with
// the page's scales ks, vs:
//   S^T = Kc Q'^T        tcgen05.mma kind::f8f6f4: A = the K page (M = 128 keys, K-major), B = Q' (N = 2 x rows)
//   p   = 2^(s - m_t)    softmax warps, m_t = the row's largest s of the step
//   O^T = Vc^T P'^T      A = the V page (M = 128 features, MN-major), B = P' (N = 2 x rows, 128 keys)
//   acc = acc 2^(m - m') + O^T vs 2^(m_t - m')      fp32 registers, m' = max(m, m_t)
// K and V go from HBM by TMA to shared memory and into the tensor cores as
// they are: nothing dequantises them. The other operand is made of two e4m3
// pieces, x = hi + lo / 16 (for eight rows, columns r and 8 + r of 16). A bf16 q
// at a power-of-two row scale is exactly that sum, down to 2^-13 of the row's
// largest element (the smallest step of lo / 16 is 2^-13, the largest element
// at least 224). p, scaled to 256 at the step's maximum, goes through fp16: it
// is off by at most 2^-11 of itself for that and 2^-9 for the pieces, less than
// a bf16 p, but by no less than half of that smallest step, 2^-22 of the
// maximum: a p below 2^-14 of its step's largest has fewer bits in the product
// (in l and in the weights it has them all). What that leaves out is at most
// 2^-22 |v| a key, seen only where the large p stand before a V near zero. A
// third piece would be 32 columns where there are 16 (M = 128 takes them by
// 16), and 32 rows have all of TMEM in use. O^T is read back every tile, so
// that page scales and the running maximum act in fp32, and a step of small p
// is as exact as any other.
//
// Two tiles of an item make a step: what takes time between a step's scores and
// its P' is a chain of waits (one tile at a time took 2300 cycles, where the
// memory gives a CTA a tile every 2800), and two tiles share it. Then the
// memory bounds all but short calls: 512k tokens of 8 heads in 160 us (6.7 TB/s
// of K and V; a copy does 6.8). What it comes to elsewhere: 5 us before the
// first product (launch, lengths, page table, first pages), 4 us behind the
// last (the joining kernel), and a few waits at every item's end (1000
// sequences of up to 1000 tokens: 243 us, 153 at the copy rate). With 17 to 32
// rows one CTA of four groups has the SM; its chain of 1850 cycles a tile is
// longer than the memory's 1400 (28 rows, 128k tokens, 4 heads: 39 us against 20).
//
// The work is the list of all tiles of the batch, item (sequence, kv head, row
// chunk) by item; every CTA takes an equal run of it, so ragged batches stay
// balanced and one long sequence spreads over the chip. An item inside one
// CTA's run is finished there; the others leave (m, l, acc) per CTA and
// join_kernel adds them in CTA order: results do not depend on timing.
//
// Warps: kWG groups of four for softmax and accumulation, eight rows each
// (thread t of a group: key t of a tile, feature t of the output), then K copies,
// V copies, MMA issue (and TMEM), and the Q' operand.
//
// Every launch may start while the kernel before it ends (3 us a call saved);
// each waits (grid_dep_wait) before it touches anything of another's, and no
// thread returns without that, so that a kernel's end is its predecessors' too.
#include <algorithm>
#include <utility>
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace crisp {
using namespace ptx;

namespace {

constexpr int kWgRows = 8;                        // rows of a softmax warp group
constexpr uint32_t kPage = kB * kD;               // bytes of a page of one head, K or V
constexpr int kMaxTail = kMaxQLen - 1;            // keys that only some of the rows see
constexpr float kLo = 16.f;                       // the second piece's scale
constexpr int kStep = 2;                           // tiles of a step
constexpr int kMaxSlots = 6;                      // K (or V) page slots

// kWG groups: rows, CTAs per SM, and the page slots that leave room for them.
template <int kWG>
struct Cfg {
  static constexpr int rows = kWG * kWgRows;
  static constexpr int workers = kWG * 4;                   // softmax warps
  static constexpr int threads = (workers + 4) * 32;
  static constexpr int per_sm = kWG == 1 ? 2 : 1;
  static constexpr int k_slots = kWG == 1 ? 3 : 5;
  static constexpr int v_slots = kWG == 1 ? 3 : 5;
  // Where one CTA has the SM to itself, nothing else runs while it waits for a
  // step's V product: P' and O get a second buffer, and O is added a step later.
  static constexpr int bufs = kWG == 1 ? 1 : 2;
  static constexpr int N = 2 * rows;                        // columns of B
  static constexpr uint32_t op = N * 128;                   // bytes of Q' or of a tile's P'
  static constexpr uint32_t smem = 1024 + (k_slots + v_slots) * kPage + (2 + kStep * bufs) * op;
  static constexpr uint32_t o_col = 2 * kStep * N;          // S: two buffers of a step, then O
  static constexpr uint32_t tmem = 4 * kStep * N;           // (a power of two)
};

template <int kWG>
struct Shared {
  uint64_t k_full[kMaxSlots], k_empty[kMaxSlots], v_full[kMaxSlots], v_empty[kMaxSlots];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], v_start, drain;
  uint32_t tmem_base;
  int abort;
  int warp_sum[kWG * 4 + 4];
  uint32_t odd[kMaxBatch / 32];                     // sequences with an odd number of pages
  int odd_before[kMaxBatch / 32], cut[2];           // how many before these 32; the run's bounds
  alignas(16) float qs[2][kWG * kWgRows];           // q scale * scale * log2(e) per row
  alignas(16) float red[2][kWG][4][kWgRows];        // warps' row maxima
  float sum[kWG][4][kWgRows];                       // and, at an item's end, their row sums
  alignas(16) float ref[kWG * 4][kWgRows];          // per warp: the step's maximum - 8 (0 for a row without keys)
  alignas(16) float alpha[kWG * 4][kWgRows];        // what scales the accumulators to the new maximum
  alignas(16) float wl[kWG * 4][2][kWgRows];        // weight of the step's p and O at it
  float tail[2][kWG * kWgRows][kMaxTail + 1];       // p of keys that only some rows see
};

// A split item, recorded by the CTA in which it begins: under the CTA's number
// (one item at most begins in it and goes on), or, with more than eight rows and
// no more items than CTAs, under the item's: then the joining kernel has a block
// a row for every item and not for every CTA (28 rows, 4 heads: 112 and not
// 4256, 39.1 us and not 40.6; with eight rows or fewer it gains nothing).
struct Split {
  int b, gc;        // sequence (-1: no such item); kv head * chunks + row chunk
  int first, last;  // the CTAs in which it begins and ends
};

struct Args {
  int batch, hkv, group, q_len, rows, chunks, num_pages, max_pages, ctas;
  int records;                         // joining blocks a row: ctas, or the number of items
  const float *k_scale, *v_scale;
  const int32_t *table, *lens;
  const uint8_t* v;                    // for the tail keys
  int64_t page_stride, head_stride;
  const __nv_bfloat16* q;
  int64_t q_b, q_h, q_t;
  __nv_bfloat16* out;
  int64_t o_b, o_h, o_t;
  float c;                             // scale * log2(e)
  float* part;                         // [2 ctas][rows of a chunk][128]
  float2* part_ml;                     // [2 ctas][rows of a chunk]  (m, l)
  Split* split;                        // [records]
  float* lse;                          // [batch][hkv][rows]  log2 sum of 2^s, +inf for a row without keys; or null
  float* scores;                       // [batch][hkv][rows][128 max_pages] or null
  DevStatus* status;
};

__device__ __forceinline__ int clamped_len(const Args& a, int b, bool& bad) {
  const int n = a.lens[b], cap = a.max_pages * kB;
  bad = n < 0 || n > cap;
  return min(max(n, 0), cap);
}

// `runs` CTAs share `total` tiles or steps (every one of them gets one): run c
// begins at floor(total c / runs).
struct Shares {
  int total, runs, each, rest;  // each = total / runs, rest = total % runs
  __device__ __forceinline__ Shares(int total_, int ctas) {
    total = total_;
    runs = min(total, ctas);
    each = runs > 0 ? total / runs : 0;
    rest = total - each * runs;
  }
  __device__ __forceinline__ int begin(int c) const { return each * c + rest * c / runs; }  // rest, c < runs <= 304
  // The run that holds tile (or step) t.
  __device__ __forceinline__ int of(int t) const {
    int c = static_cast<int>((static_cast<float>(t) + 0.5f) * static_cast<float>(runs) / static_cast<float>(total));
    c = min(max(c, 0), runs - 1);
    while (c > 0 && begin(c) > t) --c;
    while (c + 1 < runs && begin(c + 1) <= t) ++c;
    return c;
  }
};

template <class T>
__device__ __forceinline__ T bcast(T v, int lane) {
  return __shfl_sync(0xffffffffu, v, lane);
}

__device__ __forceinline__ void fail(int* abort, DevStatus* st, uint32_t where) {
  *reinterpret_cast<volatile int*>(abort) = 1;
  report_error(st, CRISP_ERR_TIMEOUT, where);
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* abort) {
  bool ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  ok = mbar_wait(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}

// Walks the items of a run: the tile's sequence, kv head and chunk, and how
// many of the item's tiles the run still has from it on.
struct Walk {
  int b, gc, page, pages, left;
  __device__ __forceinline__ void begin(const int* pre, const Args& a, int t, int n) {
    const int hc = a.hkv * a.chunks;
    int lo = 0, hi = a.batch - 1;  // the last b with pre[b] * hc <= t that has pages: pre[b + 1] * hc > t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid + 1] * hc > t) hi = mid;
      else lo = mid + 1;
    }
    b = lo;
    pages = pre[lo + 1] - pre[lo];
    const int rem = t - pre[lo] * hc;
    gc = rem / pages;
    page = rem - gc * pages;
    left = min(pages - page, n);
  }
  // To the next item; n: tiles of the run from it on (> 0).
  __device__ __forceinline__ void next(const int* pre, const Args& a, int n) {
    page = 0;
    if (++gc == a.hkv * a.chunks) {
      gc = 0;
      do ++b;
      while (pre[b + 1] == pre[b]);
      pages = pre[b + 1] - pre[b];
    }
    left = min(pages, n);
  }
};

// The page of a tile: its id (-1 if the table names none of the pool's).
__device__ __forceinline__ int page_id(const Args& a, int b, int page) {
  const int id = a.table[static_cast<int64_t>(b) * a.max_pages + page];
  return id >= 0 && id < a.num_pages ? id : -1;
}

// Row r of the lanes' values v[r], reduced over the warp: lane L returns row
// L >> (5 - log2 kR). Halves the rows a step while it can: kR - 1 + (5 -
// log2 kR) exchanges.
template <int kR, bool kMax>
__device__ __forceinline__ float warp_rows(float (&v)[kR]) {
  const int lane = threadIdx.x & 31;
  auto op = [](float x, float y) { return kMax ? fmaxf(x, y) : x + y; };
  int off = 16;
#pragma unroll
  for (int n = kR / 2; n >= 1; n >>= 1, off >>= 1) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int k = 0; k < kR / 2; ++k) {
      if (k >= n) break;
      const float send = up ? v[k] : v[k + n], mine = up ? v[k + n] : v[k];
      v[k] = op(mine, __shfl_xor_sync(0xffffffffu, send, off));
    }
  }
  for (; off >= 1; off >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], off));
  return v[0];
}

// A group's eight rows of two accumulators (16 columns each): v[r] = hi + lo / 16.
__device__ __forceinline__ void load_rows(uint32_t ta, uint32_t tb, float (&v)[kWgRows], float (&w)[kWgRows]) {
  uint32_t x[16], y[16];
  tmem_ld16x2(ta, tb, x, y);
#pragma unroll
  for (int r = 0; r < 8; r += 2) {
    ffma2(v[r], v[r + 1], __uint_as_float(x[8 + r]), __uint_as_float(x[9 + r]), 1.f / kLo, 1.f / kLo,
          __uint_as_float(x[r]), __uint_as_float(x[r + 1]));
    ffma2(w[r], w[r + 1], __uint_as_float(y[8 + r]), __uint_as_float(y[9 + r]), 1.f / kLo, 1.f / kLo,
          __uint_as_float(y[r]), __uint_as_float(y[r + 1]));
  }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Q' of kRows rows from rb on of a chunk whose first row is r0, by one warp: four
// features a lane, first in registers. All rows are asked for before the first
// is made.
template <int kRows>
struct QRows {
  uint32_t hi[kRows], lo[kRows];
  float scale;  // lane r: of row r, with scale * log2(e)

  __device__ __forceinline__ void make(const Args& a, int b, int g, int r0, int rb) {
    const int lane = threadIdx.x & 31;
    uint2 w[kRows];
#pragma unroll
    for (int rr = 0; rr < kRows; ++rr) {
      const int row = r0 + rb + rr;
      w[rr] = make_uint2(0u, 0u);
      if (row < a.rows) {
        const int i = a.q_len == 1 ? 0 : row / a.group, h = g * a.group + row - i * a.group;
        w[rr] = *reinterpret_cast<const uint2*>(a.q + b * a.q_b + h * a.q_h + i * a.q_t + lane * 4);
      }
    }
    scale = 0.f;
#pragma unroll
    for (int rr = 0; rr < kRows; ++rr) {
      float v[4] = {__uint_as_float(w[rr].x << 16), __uint_as_float(w[rr].x & 0xffff0000u),
                    __uint_as_float(w[rr].y << 16), __uint_as_float(w[rr].y & 0xffff0000u)};
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!isfinite(v[e])) v[e] = __int_as_float(0x7fffffff);  // the row's scores become NaN
        amax = fmaxf(amax, fabsf(v[e]));                          // passes over NaN
      }
      const int e2 = scale_exponent(warp_max(amax));
      const float inv = exp2_int(-e2);
      hi[rr] = lo[rr] = 0;
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float y0 = v[e] * inv, y1 = v[e + 1] * inv;
        const uint16_t h2 = pack_e4m3x2(y0, y1);
        float h0, h1;
        unpack_e4m3x2(h2, h0, h1);
        hi[rr] |= static_cast<uint32_t>(h2) << (8 * e);
        lo[rr] |= static_cast<uint32_t>(pack_e4m3x2((y0 - h0) * kLo, (y1 - h1) * kLo)) << (8 * e);
      }
      if (lane == rr) scale = exp2_int(e2) * a.c;
    }
  }
  __device__ __forceinline__ void store(uint8_t* dst, float* qs, int rb) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int rr = 0; rr < kRows; ++rr) {
      const int r = rb + rr;
      // rows 16 (r / 8) + r % 8 and 8 further on; 16-byte chunks are swizzled by the row's low 3 bits
      const uint32_t at = (r / 8 * 16 + r % 8) * 128 + (((lane >> 2) ^ (r % 8)) << 4) + (lane & 3) * 4;
      *reinterpret_cast<uint32_t*>(dst + at) = hi[rr];
      *reinterpret_cast<uint32_t*>(dst + 8 * 128 + at) = lo[rr];
    }
    if (lane < kRows) qs[rb + lane] = scale;
  }
};

template <int kWG, bool kScores>
__global__ void __launch_bounds__(Cfg<kWG>::threads, Cfg<kWG>::per_sm)
    decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                  const __grid_constant__ Args a) {
  using C = Cfg<kWG>;
  constexpr int kR = C::rows, kKWarp = C::workers, kVWarp = C::workers + 1, kMmaWarp = C::workers + 2, kQWarp = C::workers + 3;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = base;
  uint8_t* sV = sK + C::k_slots * kPage;
  uint8_t* sQ = sV + C::v_slots * kPage;  // two buffers
  uint8_t* sP = sQ + 2 * C::op;           // C::bufs steps' tiles
  int* pre = reinterpret_cast<int*>(sP + C::bufs * kStep * C::op);
  __shared__ Shared<kWG> sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    sh.abort = 0;
    for (int s = 0; s < C::k_slots; ++s) {
      mbar_init(&sh.k_full[s], 1);
      mbar_init(&sh.k_empty[s], 1);
    }
    for (int s = 0; s < C::v_slots; ++s) {
      mbar_init(&sh.v_full[s], 1);
      mbar_init(&sh.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.q_full[s], C::workers);
      mbar_init(&sh.q_empty[s], 1 + kWG);  // the last score product of the item; the softmax groups' end of it
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.p_full[s], C::workers * 32);
      mbar_init(&sh.o_full[s], 1);
    }
    mbar_init(&sh.v_start, 1);
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem_base, C::tmem);
    tmem_relinquish();
  }
  if (lane == 0 && (warp == kKWarp || warp == kVWarp)) prefetch_tmap(warp == kKWarp ? &tk : &tv);
  // The lengths, and a line of the page table by each CTA, are asked for: what
  // of the table is used is known two reads from here.
  if (warp == 1 && lane * 32 < a.batch) prefetch_l2(a.lens + lane * 32);
  if (threadIdx.x == 0 && static_cast<int>(blockIdx.x) * 32 < a.batch * a.max_pages)
    prefetch_l2(a.table + static_cast<int>(blockIdx.x) * 32);
  // From here on what earlier kernels of the stream wrote is read, and results are written.
  grid_dep_wait();
  // Pages before each sequence (an inclusive scan over the batch, a block of sequences at a time).
  int before = 0;
  if (threadIdx.x == 0) pre[0] = 0;
  for (int b0 = 0; b0 < a.batch; b0 += C::threads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int n = 0;
    if (b < a.batch) {
      bool bad;
      n = (clamped_len(a, b, bad) + kB - 1) / kB;
      if (bad && blockIdx.x == 0) report_error(a.status, CRISP_ERR_BOUNDS, 0x601);
    }
    const int own = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += up;
    }
    if (lane == 31) sh.warp_sum[warp] = n;
    const uint32_t odd = __ballot_sync(0xffffffffu, own & 1);
    if (lane == 0 && b < a.batch) sh.odd[b / 32] = odd;
    __syncthreads();
    int add = before;
    for (int w = 0; w < warp; ++w) add += sh.warp_sum[w];
    if (b < a.batch) pre[b + 1] = n + add;
    for (int w = 0; w < C::threads / 32; ++w) before += sh.warp_sum[w];
    if (b0 + C::threads < a.batch) __syncthreads();  // warp_sum is written again
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = sh.tmem_base;
  // (the host has seen to it that the tiles a full table holds are an int's worth)
  const int hc = a.hkv * a.chunks, run = static_cast<int>(blockIdx.x);
  const bool by_item = kWG > 1 && a.records < a.ctas;
  // Many short items are shared out by steps, not by tiles: the step of an odd
  // last tile takes as long as another (1000 sequences of up to 1000 tokens, 8
  // heads: 243 us, 257 by tiles). Longer items gain nothing.
  const bool by_step = before <= 16 * a.batch && before * hc >= 4 * a.ctas;
  int odds = 0;  // sequences with an odd number of pages
  if (by_step) {
    int c = lane < (a.batch + 31) / 32 ? __popc(sh.odd[lane]) : 0;
    const int mine = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += up;
    }
    if (warp == 0) sh.odd_before[lane] = c - mine;
    odds = __shfl_sync(0xffffffffu, c, 31);
  }
  const Shares shares(by_step ? (before + odds) / 2 * hc : before * hc, a.ctas);
  int t_lo = run < shares.runs ? shares.begin(run) : 0;
  int n = run < shares.runs ? shares.begin(run + 1) - t_lo : 0;
  // steps of a head before sequence b
  auto steps_before = [&](int b) {
    return (pre[b] + sh.odd_before[b >> 5] + __popc(sh.odd[b >> 5] & ((1u << (b & 31)) - 1u))) / 2;
  };
  if (by_step) {
    __syncthreads();
    if (lane == 0 && warp < 2) {
      // the first tile of the run, and the one behind its last
      const int t = warp == 0 ? t_lo : t_lo + n;
      int lo = 0, hi = a.batch;  // the last sequence whose first step is not behind t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (steps_before(mid) * hc <= t) lo = mid;
        else hi = mid;
      }
      const int pages = pre[lo + 1] - pre[lo], each = (pages + 1) / 2;
      const int rem = t - steps_before(lo) * hc, gc = each > 0 ? rem / each : 0;  // (hc behind the last sequence)
      sh.cut[warp] = pre[lo] * hc + gc * pages + 2 * (rem - gc * each);
    }
    __syncthreads();
    t_lo = sh.cut[0];
    n = sh.cut[1] - t_lo;
  }

  if (n > 0 && (warp == kKWarp || warp == kVWarp)) {
    // The K pages, or the V pages, of the run in order: each lane looks up one of
    // 32 tiles, lane 0 issues the copies.
    const bool is_k = warp == kKWarp;
    const CUtensorMap* map = is_k ? &tk : &tv;
    uint8_t* slots = is_k ? sK : sV;
    uint64_t *full = is_k ? sh.k_full : sh.v_full, *empty = is_k ? sh.k_empty : sh.v_empty;
    const int count = is_k ? C::k_slots : C::v_slots;
    // Scores are read back by weights_kernel: the pages, which are not, leave L2 first.
    const uint64_t policy = kScores ? policy_evict_first() : 0;
    constexpr int kFirst = kWG == 1 ? kStep : 2 * kStep;  // at most a K slot each
    int slot = 0, phase = 1, issued = 0;
    bool go = true;
    for (int i0 = 0; go && i0 < n; i0 += 32) {
      int z = -1, g = 0;
      if (i0 + lane < n) {
        Walk x;
        x.begin(pre, a, t_lo + i0 + lane, n);
        z = page_id(a, x.b, x.page);
        g = a.chunks == 1 ? x.gc : x.gc / a.chunks;
        if (z < 0) report_error(a.status, CRISP_ERR_BOUNDS, 0x602);
      }
      const int m = min(32, n - i0);
      if (!is_k && i0 == 0 && !warp_wait(&sh.v_start, 0, &sh.abort)) {
        go = false;
        if (lane == 0) fail(&sh.abort, a.status, 0x615);
      }
      for (int k = 0; k < m; ++k) {
        const int zt = bcast(z, k), gt = bcast(g, k);
        if (lane == 0 && go) {
          go = mbar_wait(&empty[slot], phase, &sh.abort);
          if (!go) {
            fail(&sh.abort, a.status, 0x610);
          } else if (zt >= 0) {
            mbar_arrive_expect_tx(&full[slot], kPage);
            if (kScores) tma_load_4d_hint(slots + slot * kPage, map, &full[slot], 0, 0, gt, zt, policy);
            else tma_load_4d(slots + slot * kPage, map, &full[slot], 0, 0, gt, zt);
          } else {
            mbar_arrive(&full[slot]);  // a bad page id: nothing is copied, and the tile counts as empty
          }
          issued += go;
          // the first scores' K pages go ahead of any V page
          if (is_k && issued == min(kFirst, n)) mbar_arrive(&sh.v_start);
          if (++slot == count) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      go = bcast(static_cast<int>(go), 0) != 0;
    }
    if (lane == 0) {
      // Every copy issued has landed before the CTA ends (bounded waits that
      // ignore the abort flag).
      const int never = 0;
      for (int q = max(0, issued - count); q < issued; ++q) mbar_wait(&full[q % count], (q / count) & 1, &never);
    }
  } else if (n > 0 && warp == kMmaWarp) {
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_e4m3_f32(128, C::N, false, false);
      constexpr uint32_t idesc_pv = idesc_e4m3_f32(128, C::N, true, true);
      const uint64_t dk0 = sdesc_sw128(smem_u32(sK), 16, 1024), dv0 = sdesc_sw128(smem_u32(sV), 1024, 1024);
      const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024), dp = sdesc_mn8(smem_u32(sP), 128, kB * 16);
      bool go = true;
      Walk x;  // of the score products, up to two steps ahead of the others
      x.begin(pre, a, t_lo, n);
      int ik = 0, iv = 0, item = -1, sk = 0;  // tiles taken, items begun, steps of scores issued
      int ks = 0, kph = 0, vs = 0, vph = 0;   // page slots and their phases
      bool begins = true;
      int size[3];                            // tiles of the steps in flight, by step % 3
      auto wait = [&](uint64_t* bar, int parity) { return mbar_wait(bar, parity, &sh.abort); };
      // S of the next step, if the run has one more; false on abort
      auto issue_qk = [&]() -> bool {
        if (ik == n) return true;
        if (begins) {
          ++item;
          if (!wait(&sh.q_full[item & 1], (item >> 1) & 1)) return false;
        }
        const int m = min(kStep, x.left), buf = sk & 1;
        const uint64_t dqi = dq + (item & 1) * (C::op >> 4);
        for (int j = 0; j < m; ++j) {
          if (!wait(&sh.k_full[ks], kph)) return false;
          tc_fence_after();
          // 32 features a product
          umma_f8_x4<2, 2>(tmem + (buf * kStep + j) * C::N, dk0 + ks * (kPage >> 4), dqi, idesc_qk);
          umma_commit(&sh.k_empty[ks]);
          if (++ks == C::k_slots) {
            ks = 0;
            kph ^= 1;
          }
        }
        ik += m;
        x.left -= m;
        begins = x.left == 0;
        umma_commit(&sh.s_full[buf]);
        if (begins) {
          umma_commit(&sh.q_empty[item & 1]);
          if (ik < n) x.next(pre, a, n - ik);
        }
        if (sk % 3 == 0) size[0] = m;
        else if (sk % 3 == 1) size[1] = m;
        else size[2] = m;
        ++sk;
        return true;
      };
      go = issue_qk() && issue_qk();
      for (int st = 0; go && iv < n; ++st) {
        const int ob = st % C::bufs, m = st % 3 == 0 ? size[0] : st % 3 == 1 ? size[1] : size[2];
        if (!wait(&sh.p_full[ob], (st / C::bufs) & 1)) go = false;
        for (int j = 0; go && j < m; ++j) {
          if (!wait(&sh.v_full[vs], vph)) {
            go = false;
            break;
          }
          tc_fence_after();
          // 32 keys a product: 4096 bytes of V, 512 of P'
          umma_f8_x4<256, 32>(tmem + C::o_col + (ob * kStep + j) * C::N, dv0 + vs * (kPage >> 4),
                              dp + (ob * kStep + j) * (C::op >> 4), idesc_pv);
          umma_commit(&sh.v_empty[vs]);
          if (++vs == C::v_slots) {
            vs = 0;
            vph ^= 1;
          }
        }
        if (!go) break;
        umma_commit(&sh.o_full[ob]);
        iv += m;
        go = issue_qk();
      }
      if (!go) fail(&sh.abort, a.status, 0x611);
      // Every product has completed before TMEM is released (bounded, ignores the abort flag).
      umma_commit(&sh.drain);
      const int never = 0;
      if (!mbar_wait(&sh.drain, 0, &never)) fail(&sh.abort, a.status, 0x612);
    }
  } else if (n > 0 && warp == kQWarp) {
    // Q' of the items of the run but the first, which the softmax warps make
    // while they wait for its scores.
    Walk x;
    x.begin(pre, a, t_lo, n);
    // whether the item begins here and goes on behind the run
    auto record = [&](bool ends_run) {
      const int rest = x.pages - x.page - x.left;  // its pages behind this run
      const bool goes_on = x.page == 0 && rest > 0;
      int ends_in = run;
      if (goes_on)
        ends_in = shares.of(by_step ? steps_before(x.b) * hc + (x.gc + 1) * ((x.pages + 1) / 2) - 1 : t_lo + n - 1 + rest);
      const Split sp{goes_on ? x.b : -1, x.gc, run, ends_in};
      if (!by_item) {
        if (ends_run) a.split[run] = sp;
      } else if (x.page == 0) {
        a.split[x.b * a.hkv * a.chunks + x.gc] = sp;
      }
    };
    int t = x.left;
    bool ok = true;
    for (int item = 1; t < n; ++item) {
      if (by_item && lane == 0) record(false);
      x.next(pre, a, n - t);
      t += x.left;
      const int buf = item & 1, g = x.gc / a.chunks, r0 = (x.gc - g * a.chunks) * kR;
      // the first rows are made while their buffer is still in use
      constexpr int kAtOnce = kR < 16 ? kR : 16;
      QRows<kAtOnce> q;
      q.make(a, x.b, g, r0, 0);
      if (ok && !warp_wait(&sh.q_empty[buf], ((item >> 1) & 1) ^ 1, &sh.abort)) {
        if (lane == 0) fail(&sh.abort, a.status, 0x613);
        ok = false;
      }
      if (!ok) continue;  // every item is recorded all the same
      q.store(sQ + buf * C::op, sh.qs[buf], 0);
      for (int rb = kAtOnce; rb < kR; rb += kAtOnce) {
        q.make(a, x.b, g, r0, rb);
        q.store(sQ + buf * C::op, sh.qs[buf], rb);
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive_n(&sh.q_full[buf], C::workers);
    }
    if (lane == 0) record(true);
  } else if (n > 0 && warp < C::workers) {
    const int wg = warp >> 2, quarter = warp & 3;
    const int tid = threadIdx.x & 127;              // key of a tile, feature of the output
    const int row0 = wg * kWgRows;                  // the group's rows of the chunk
    const int bar = 1 + wg;
    const uint32_t lane_tmem = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 2 * row0;
    // P' is MN-major: key `tid`'s 16 bytes of the group's rows (hi, then lo) lie together
    uint8_t* const p_at = sP + (wg * kB + tid) * 16;
    const int my_row = lane & (kWgRows - 1);        // row of the lane-held maximum
    float acc[kWgRows], l[kWgRows];
    float m = -INFINITY;                            // running maximum of row my_row, base 2
    // A wait that gives up lets its warp go on, and so does every wait after it:
    // all warps of a group take every step of the run, so none is left behind in
    // a named barrier. What is computed then goes to the call's own buffers, and
    // the status says that it is worth nothing.
    auto await = [&](uint64_t* b, int parity) {
      bool done = mbar_try_wait(b, parity);
      if (__all_sync(0xffffffffu, done)) return;
      const volatile int* abort = &sh.abort;
      const unsigned long long t0 = globaltimer_ns();
      while (!done && !*abort && globaltimer_ns() - t0 <= kWaitLimitNs) done = mbar_try_wait(b, parity);
      if (!done) fail(&sh.abort, a.status, 0x614);
      __syncwarp();
    };
    // tiles by 32: lane L looks up tile win + L (its page, scales, and sequence's length)
    int win = 0, z = -1, ln = 0;
    float ks = 0.f, vs = 0.f;
    int id = -1, id_head = 0;  // as asked for
    auto ask = [&](int i) {
      win = i;
      id = -1;
      if (i + lane < n) {
        Walk y;
        y.begin(pre, a, t_lo + i + lane, n);
        id = a.table[static_cast<int64_t>(y.b) * a.max_pages + y.page];
        id_head = a.chunks == 1 ? y.gc : y.gc / a.chunks;
        bool bad;
        ln = clamped_len(a, y.b, bad);
      }
    };
    auto take = [&]() {
      z = id >= 0 && id < a.num_pages ? id : -1;
      ks = vs = 0.f;
      if (z >= 0) {
        const int64_t at = static_cast<int64_t>(z) * a.hkv + id_head;
        ks = a.k_scale[at];
        vs = a.v_scale[at];
      }
    };
    auto look_up = [&](int i) {
      ask(i);
      take();
    };
    ask(0);
    Walk x;
    x.begin(pre, a, t_lo, n);
    {
      // the first item's Q', two rows a warp
      const int g0 = x.gc / a.chunks;
      QRows<2> q;
      q.make(a, x.b, g0, (x.gc - g0 * a.chunks) * kR, warp * 2);
      q.store(sQ, sh.qs[0], warp * 2);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[0]);
    }
    take();
    int item = 0, i = 0, steps = 0, len = 0, g = 0, r0 = 0, toks_r0 = -1;
    uint32_t toks = 0;
    auto tok_of = [&](int r) { return static_cast<int>(toks >> (4 * r) & 15u); };
    bool begins = true;
    // An item as its end needs it (`end`: the page behind the last one taken).
    struct Item {
      int b, gc, g, r0, end, pages, len;
      uint32_t toks;
    };
    // the step whose O is still to be added
    struct {
      int tiles, page;
      float vs[kStep];
      bool tail;
    } o{};
    Item prev{};  // its item (one buffer: an item ends while the next one's first step runs)

    // A page's rows [lo, end) hold keys that only the later tokens see.
    auto tail_rows = [&](int len, int page, int& lo, int& end) {
      lo = max(len - (a.q_len - 1) - page * kB, 0);
      end = min(max(len - page * kB, 0), kB);
    };

    auto add_o = [&](int st, const Item& of) {
      const int ob = st % C::bufs;
      await(&sh.o_full[ob], (st / C::bufs) & 1);
      tc_fence_after();
      float wl[kWgRows];
      load8(sh.wl[warp][ob], wl);
      float both[kStep][kWgRows];  // of a step of one tile, the second is not used
      load_rows(lane_tmem + C::o_col + ob * kStep * C::N, lane_tmem + C::o_col + (ob * kStep + 1) * C::N, both[0], both[1]);
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        if (j >= o.tiles) break;
        float(&v)[kWgRows] = both[j];
        if (o.tail) {
          // added here, one by one, so that what those keys hold does not
          // reach the rows that do not see them
          const int page = o.page + j, id = page_id(a, of.b, page);
          int lo, end;
          tail_rows(of.len, page, lo, end);
          const int first = page * kB - (of.len - (a.q_len - 1));  // row 0's place among those keys
          const uint8_t* vp = a.v + id * a.page_stride + of.g * a.head_stride + tid;
          for (int k = lo; id >= 0 && k < end; ++k) {
            float val, none;
            unpack_e4m3x2(vp[k * kD], val, none);
#pragma unroll
            for (int r = 0; r < kWgRows; ++r) {
              const float p = sh.tail[ob][row0 + r][first + k];
              if (p >= 0.f || p != p) v[r] = fmaf(p, val, v[r]);  // -1: not seen
            }
          }
        }
#pragma unroll
        for (int r = 0; r < kWgRows; r += 2) {
          float w0, w1;
          fmul2(w0, w1, wl[r], wl[r + 1], o.vs[j], o.vs[j]);
          ffma2(acc[r], acc[r + 1], v[r], v[r + 1], w0, w1, acc[r], acc[r + 1]);
        }
      }
    };

    // The end of an item in this run; i_end: tiles of the run up to it.
    auto finish = [&](int i_end, const Item& of) {
      const float wsum = warp_rows<kWgRows, false>(l);
      if ((lane & 3) == 0) sh.sum[wg][quarter][lane >> 2] = wsum;
      named_bar_sync(bar, 128);
      const int t_item = t_lo + i_end - of.end;  // the item's first tile
      const bool whole = t_item >= t_lo && of.end == of.pages;
      const int slot = 2 * run + (t_item < t_lo ? 0 : 1);
      const int nr = min(kWgRows, a.rows - of.r0);
      // lane r holds row r's sum, its inverse, and where it goes
      const float (&sum)[4][kWgRows] = sh.sum[wg];
      const float ls = (sum[0][my_row] + sum[1][my_row]) + (sum[2][my_row] + sum[3][my_row]);
      if (whole) {
        const float inv = ls == 0.f ? 0.f : 1.f / ls;
        const int tok = static_cast<int>(of.toks >> (4 * my_row) & 15u), h = of.g * a.group + of.r0 + my_row - tok * a.group;
        const int64_t at = of.b * a.o_b + h * a.o_h + tok * a.o_t;
#pragma unroll
        for (int r = 0; r < kWgRows; ++r) {
          const float f = bcast(inv, r);
          const int64_t to = bcast(at, r);
          if (r < nr) a.out[to + tid] = __float2bfloat16_rn(acc[r] * f);
        }
        if (kScores && tid < nr)
          a.lse[(static_cast<int64_t>(of.b) * a.hkv + of.g) * a.rows + of.r0 + tid] = ls == 0.f ? INFINITY : m + log2f(ls);
      } else {
        float* to = a.part + (static_cast<int64_t>(slot) * kR + row0) * kD + tid;
#pragma unroll
        for (int r = 0; r < kWgRows; ++r)
          if (r < nr) to[r * kD] = acc[r];
        if (tid < nr) a.part_ml[slot * kR + row0 + tid] = make_float2(m, ls);
      }
    };

    for (int st = 0; i < n; ++st) {
      const int mt_tiles = min(kStep, x.left), buf = st & 1;
      if (i + kStep > win + 32) look_up(i);
      if (begins) {
        len = bcast(ln, i - win);
        g = a.chunks == 1 ? x.gc : x.gc / a.chunks;
        r0 = (x.gc - g * a.chunks) * kR + row0;
        if (r0 != toks_r0) {
          // the rows' tokens, four bits each (rows past the last count as the last token's)
          toks_r0 = r0;
          const int tok = a.q_len == 1 ? 0 : min((r0 + my_row) / a.group, kMaxQLen - 1);
          toks = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(tok) << (4 * my_row));
        }
        await(&sh.q_full[item & 1], (item >> 1) & 1);
      }
      await(&sh.s_full[buf], (st >> 1) & 1);
      tc_fence_after();
      // Row r's token sees the keys below len - (q_len - 1) + its number.
      float s[kStep][kWgRows], t[kWgRows], vst[kStep];
      bool partial[kStep], held[kStep];  // some rows do not see some keys; the page is there
      load8(&sh.qs[item & 1][row0], t);
      // of a step of one tile, the second buffer's old scores are read and not used
      load_rows(lane_tmem + buf * kStep * C::N, lane_tmem + (buf * kStep + 1) * C::N, s[0], s[1]);
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        held[j] = bcast(z, (i - win + j) & 31) >= 0;
        vst[j] = bcast(vs, (i - win + j) & 31);
        const float kst = bcast(ks, (i - win + j) & 31);
        if (j >= mt_tiles) {
          partial[j] = false;
#pragma unroll
          for (int r = 0; r < kWgRows; ++r) s[j][r] = -INFINITY;
          continue;
        }
#pragma unroll
        for (int r = 0; r < kWgRows; r += 2) {
          float c0, c1;
          fmul2(c0, c1, t[r], t[r + 1], kst, kst);
          fmul2(s[j][r], s[j][r + 1], s[j][r], s[j][r + 1], c0, c1);
        }
        const int past = (x.page + j) * kB + tid - (len - (a.q_len - 1));  // < 0: every row sees the key
        partial[j] = !held[j] || (x.page + j + 1) * kB > len - (a.q_len - 1);
        if (partial[j]) {
#pragma unroll
          for (int r = 0; r < kWgRows; ++r)
            if (!held[j] || past >= tok_of(r)) s[j][r] = -INFINITY;
        }
      }
      // The step's row maxima, over the group's four warps.
#pragma unroll
      for (int r = 0; r < kWgRows; ++r) t[r] = warp_max(fmaxf(s[0][r], s[1][r]));
      if (lane == 0) {
        float4* red = reinterpret_cast<float4*>(sh.red[buf][wg][quarter]);
        red[0] = make_float4(t[0], t[1], t[2], t[3]);
        red[1] = make_float4(t[4], t[5], t[6], t[7]);
      }
      // The step before: its product has run meanwhile.
      if (C::bufs == 1 && st > 0) add_o(st - 1, prev);
      if (begins) {
        if (C::bufs == 1 && st > 0) finish(i, prev);
#pragma unroll
        for (int r = 0; r < kWgRows; ++r) acc[r] = l[r] = 0.f;
        m = -INFINITY;
      }
      named_bar_sync(bar, 128);
      if (x.left == mt_tiles && tid == 0) mbar_arrive(&sh.q_empty[item & 1]);  // the item's last step has its q scales
      {
        const float (&red)[4][kWgRows] = sh.red[buf][wg];
        const float mt = fmaxf(fmaxf(red[0][my_row], red[1][my_row]), fmaxf(red[2][my_row], red[3][my_row]));
        const float mn = fmaxf(m, mt);
        // a row without keys so far: nothing to scale, and weight 0 (2^(-inf))
        const float base2 = mn == -INFINITY ? 0.f : mn;
        if (lane < kWgRows) {
          const float al = ex2_approx(m - base2);
          sh.ref[warp][my_row] = mt == -INFINITY ? 0.f : mt - 8.f;
          sh.alpha[warp][my_row] = al;
          sh.wl[warp][st % C::bufs][my_row] = ex2_approx(mt - base2 - 8.f);
          // the O still to be added is weighted for the maximum before
          if (C::bufs == 2 && !begins) sh.wl[warp][(st - 1) % C::bufs][my_row] *= al;
        }
        m = mn;
      }
      __syncwarp();
      float wl[kWgRows];
      load8(sh.alpha[warp], t);
      load8(sh.wl[warp][st % C::bufs], wl);
#pragma unroll
      for (int r = 0; r < kWgRows; r += 2) {
        fmul2(acc[r], acc[r + 1], acc[r], acc[r + 1], t[r], t[r + 1]);
        fmul2(l[r], l[r + 1], l[r], l[r + 1], t[r], t[r + 1]);
      }
      load8(sh.ref[warp], t);
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        if (j >= mt_tiles) break;
        float p[kWgRows];
#pragma unroll
        for (int r = 0; r < kWgRows; ++r) p[r] = ex2_approx(s[j][r] - t[r]);
#pragma unroll
        for (int r = 0; r < kWgRows; r += 2) ffma2(l[r], l[r + 1], p[r], p[r + 1], wl[r], wl[r + 1], l[r], l[r + 1]);
        if (partial[j]) {
          int lo, end;
          tail_rows(len, x.page + j, lo, end);
          if (!held[j]) lo = 0;
          if (held[j] && tid >= lo && tid < end) {
            const int past = (x.page + j) * kB + tid - (len - (a.q_len - 1));
#pragma unroll
            for (int r = 0; r < kWgRows; ++r) {
              sh.tail[st % C::bufs][row0 + r][past] = past < tok_of(r) ? p[r] : -1.f;
              p[r] = 0.f;
            }
          }
          if (wg == 0) {
            // V rows that not every row sees become zeros: p = 0 there, and what
            // the page holds (anything past the end) must not matter
            const int sl = (i + j) % C::v_slots;
            await(&sh.v_full[sl], ((i + j) / C::v_slots) & 1);
            if (tid >= lo) {
              uint4* rowp = reinterpret_cast<uint4*>(sV + sl * kPage + tid * 128);
#pragma unroll
              for (int e = 0; e < 8; ++e) rowp[e] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int r = 0; r < kWgRows; r += 2) {
          uint16_t h, l2;
          split_e4m3x2(p[r], p[r + 1], h, l2);
          hi[r / 2] = h;
          lo[r / 2] = l2;
        }
        *reinterpret_cast<uint4*>(p_at + (st % C::bufs * kStep + j) * C::op) = make_uint4(
            hi[0] | hi[1] << 16, hi[2] | hi[3] << 16, lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      }
      fence_async_shared();
      tc_fence_before();
      mbar_arrive(&sh.p_full[st % C::bufs]);
      if (kScores) {
        const int64_t cap = static_cast<int64_t>(a.max_pages) * kB;
        float* dst = a.scores + ((static_cast<int64_t>(x.b) * a.hkv + g) * a.rows + r0) * cap + x.page * kB + tid;
        const int nr = min(kWgRows, a.rows - r0);
#pragma unroll
        for (int r = 0; r < kWgRows; ++r) {
          if (r >= nr) break;
          dst[0] = s[0][r];
          if (mt_tiles > 1) dst[kB] = s[1][r];
          dst += cap;
        }
      }
      const Item now{x.b, x.gc, g, r0, x.page + mt_tiles, x.pages, len, toks};
      if (C::bufs == 2 && !begins) add_o(st - 1, now);
      o.tiles = mt_tiles;
      o.page = x.page;
      o.vs[0] = vst[0];
      o.vs[1] = vst[1];
      o.tail = a.q_len > 1 && (partial[0] || partial[1]);
      if (o.tail) named_bar_sync(bar, 128);  // every warp's tail p is written
      if (C::bufs == 1) prev = now;
      x.left -= mt_tiles;
      x.page += mt_tiles;
      i += mt_tiles;
      steps = st + 1;
      begins = x.left == 0;
      if (begins) {
        if (C::bufs == 2) {
          add_o(st, now);
          finish(i, now);
        }
        ++item;
        if (i < n) x.next(pre, a, n - i);
      }
    }
    if (C::bufs == 1) {
      add_o(steps - 1, prev);
      finish(n, prev);
    }
  }
  if (n == 0 && threadIdx.x == 0 && !by_item) a.split[run] = Split{-1, 0, 0, 0};
  // Sequences without a page have no tile: their rows of the output are zeros.
  for (int b = run; b < a.batch; b += a.ctas) {
    if (pre[b + 1] != pre[b]) continue;
    if (by_item)
      for (int e = threadIdx.x; e < a.hkv * a.chunks; e += C::threads) a.split[b * a.hkv * a.chunks + e] = Split{-1, 0, 0, 0};
    for (int e = threadIdx.x; e < a.hkv * a.rows * kD; e += C::threads) {
      const int d = e % kD, row = e / kD % a.rows, g = e / kD / a.rows;
      a.out[b * a.o_b + (g * a.group + row % a.group) * a.o_h + row / a.group * a.o_t + d] = __float2bfloat16_rn(0.f);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, C::tmem);
}

constexpr int kJoinThreads = 256;

// Joins the items that several CTAs worked on: block (j, r) takes row r of the
// item of record j. Eight warps share the CTAs of the
// item, a lane has four features; the sums run in a fixed order.
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Args a, int kr) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ float f[kMaxDecodeCtas];
  __shared__ float red_m[kWarps], red_l[kWarps];
  __shared__ float4 red[kWarps][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = blockIdx.y;
  grid_dep_launch();
  grid_dep_wait();
  const Split sp = a.split[blockIdx.x];
  const int c0 = sp.first;
  const int g = sp.gc / a.chunks, row = (sp.gc - g * a.chunks) * kr + r;
  if (sp.b < 0 || row >= a.rows) return;
  const int nc = sp.last - c0 + 1;
  auto slot_of = [&](int x) { return 2 * (c0 + x) + (x == 0 ? 1 : 0); };
  auto part_of = [&](int x) {
    return *reinterpret_cast<const float4*>(a.part + (static_cast<int64_t>(slot_of(x)) * kr + r) * kD + lane * 4);
  };
  // this warp's first accumulators are asked for together with the statistics
  constexpr int kFirst = 4;
  float4 first[kFirst];
#pragma unroll
  for (int u = 0; u < kFirst; ++u) first[u] = warp + u * kWarps < nc ? part_of(warp + u * kWarps) : make_float4(0, 0, 0, 0);
  static_assert(kMaxDecodeCtas <= 2 * kJoinThreads, "two CTAs' statistics a thread");
  float2 ml[2];
  float m = -INFINITY;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int x = tid + u * kJoinThreads;
    ml[u] = x < nc ? a.part_ml[slot_of(x) * kr + r] : make_float2(-INFINITY, 0.f);
    m = fmaxf(m, ml[u].x);
  }
  m = warp_max(m);
  if (lane == 0) red_m[warp] = m;
  __syncthreads();
  m = warp_max(red_m[lane & (kWarps - 1)]);
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int x = tid + u * kJoinThreads;
    const float fx = ex2_approx(ml[u].x - base);
    if (x < nc) f[x] = fx;
    l = fmaf(fx, ml[u].y, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) red_l[warp] = l;
  __syncthreads();
  l = 0.f;
  for (int w = 0; w < kWarps; ++w) l += red_l[w];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float fx, const float4& v) {
    acc.x = fmaf(fx, v.x, acc.x);
    acc.y = fmaf(fx, v.y, acc.y);
    acc.z = fmaf(fx, v.z, acc.z);
    acc.w = fmaf(fx, v.w, acc.w);
  };
#pragma unroll
  for (int u = 0; u < kFirst; ++u)
    if (warp + u * kWarps < nc) add(f[warp + u * kWarps], first[u]);
#pragma unroll 4
  for (int x = warp + kFirst * kWarps; x < nc; x += kWarps) add(f[x], part_of(x));
  red[warp][lane] = acc;
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < kWarps; ++w) {
      const float4 v = red[w][lane];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16* dst = a.out + sp.b * a.o_b + (g * a.group + row % a.group) * a.o_h + row / a.group * a.o_t;
    *reinterpret_cast<uint2*>(dst + lane * 4) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0 && a.lse != nullptr)
      a.lse[(static_cast<int64_t>(sp.b) * a.hkv + g) * a.rows + row] = l == 0.f ? INFINITY : m + log2f(l);
  }
}

// weights_out = weights_in + the sum over the rows of 2^(s - lse): kWeightKeys
// keys of one sequence and kv head a block, four a thread at a time.
constexpr int kWeightThreads = 256;
constexpr int kWeightKeys = 4 * kWeightThreads;
__global__ void __launch_bounds__(kWeightThreads)
    weights_kernel(const __grid_constant__ Args a, const float* w_in, float* w_out) {
  __shared__ float lse[kMaxGroupRows];
  const int g = blockIdx.y, b = blockIdx.z;
  grid_dep_launch();
  const int key = blockIdx.x * kWeightKeys + threadIdx.x * 4;
  const int64_t cap = static_cast<int64_t>(a.max_pages) * kB, bg = static_cast<int64_t>(b) * a.hkv + g;
  const int64_t at = bg * cap + key;
  float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
  // Rows of weights and scores end at a multiple of 128: whole groups of four are
  // there. What came before this call has ended when its first kernel lets the
  // next ones start, so w_in is read at once (from L2).
  if (w_in != nullptr && key < cap) w = __ldcg(reinterpret_cast<const float4*>(w_in + at));
  // before any return: this kernel may not end before the ones it depends on
  grid_dep_wait();
  bool bad;
  const int len = clamped_len(a, b, bad);
  if (static_cast<int>(blockIdx.x) * kWeightKeys >= len) return;
  for (int r = threadIdx.x; r < a.rows; r += kWeightThreads) lse[r] = a.lse[bg * a.rows + r];
  __syncthreads();
  if (key >= len) return;
  const float* sc = a.scores + bg * a.rows * cap + key;
  float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int r = 0; r < a.rows; ++r) {
    const float4 s = __ldcs(reinterpret_cast<const float4*>(sc + r * cap));
    const float e = lse[r];
    // a key that the row does not see (-inf) has no weight from it, even where the row's sum is NaN
    auto weight = [&](float x) { return x == -INFINITY ? 0.f : ex2_approx(x - e); };
    p.x += weight(s.x);
    p.y += weight(s.y);
    p.z += weight(s.z);
    p.w += weight(s.w);
  }
  w.x += p.x;
  w.y += p.y;
  w.z += p.z;
  w.w += p.w;
  if (key + 4 <= len) {
    *reinterpret_cast<float4*>(w_out + at) = w;
  } else {
    const float v[3] = {w.x, w.y, w.z};
    for (int e = 0; key + e < len; ++e) w_out[at + e] = v[e];
  }
}

int groups_of(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

template <int kWG, bool kScores>
cudaError_t launch_groups(const KvMaps& maps, const Args& a, cudaStream_t st) {
  using C = Cfg<kWG>;
  // The limit belongs to the kernel, not to the call: every call sets the same
  // one, so that host threads with other batches do not lower it in between.
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<kWG, kScores>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::smem + (kMaxBatch + 1) * 4);
  if (e != cudaSuccess) return e;
  return launch_dependent(decode_kernel<kWG, kScores>, dim3(static_cast<unsigned>(a.ctas)), C::threads,
                          C::smem + (a.batch + 1) * 4, st, maps.k, maps.v, a);
}
template <int kWG>
cudaError_t launch_groups(const KvMaps& maps, const Args& a, cudaStream_t st) {
  return a.scores != nullptr ? launch_groups<kWG, true>(maps, a, st) : launch_groups<kWG, false>(maps, a, st);
}

}  // namespace

int decode_row_chunks(int rows) {
  const int kr = groups_of(rows) * kWgRows;
  return (rows + kr - 1) / kr;
}

DecodeLayout decode_layout(const crisp_kv_cache& c, int hq, int q_len, bool with_weights) {
  const size_t rows = static_cast<size_t>(hq / c.hkv) * q_len, kr = groups_of(static_cast<int>(rows)) * kWgRows;
  DecodeLayout L{};
  size_t o = align_up(sizeof(DevStatus));
  L.part = o;    o = align_up(o + size_t(2) * kMaxDecodeCtas * kr * kD * 4);
  L.part_ml = o; o = align_up(o + size_t(2) * kMaxDecodeCtas * kr * 8);
  L.split = o;   o = align_up(o + size_t(kMaxDecodeCtas) * sizeof(Split));
  L.lse = o;
  if (with_weights) o = align_up(o + c.batch * c.hkv * rows * 4);
  L.scores = o;
  if (with_weights) o = align_up(o + c.batch * c.hkv * rows * c.max_pages * kB * 4);
  L.total = o;
  return L;
}

cudaError_t launch_decode(const crisp_kv_cache& c, const KvMaps& maps, int hq, int q_len, float scale,
                          const crisp_tokens& q, const crisp_tokens& out, const float* weights_in, float* weights_out,
                          char* ws, int sms, cudaStream_t st) {
  const DecodeLayout L = decode_layout(c, hq, q_len, weights_out != nullptr);
  Args a{};
  a.batch = c.batch;
  a.hkv = c.hkv;
  a.group = hq / c.hkv;
  a.q_len = q_len;
  a.rows = a.group * q_len;
  const int wg = groups_of(a.rows), kr = wg * kWgRows;
  a.chunks = decode_row_chunks(a.rows);
  a.num_pages = c.num_pages;
  a.max_pages = c.max_pages;
  // what the chip holds at once, and no more than the table can hold tiles
  const long long most = static_cast<long long>(c.batch) * c.max_pages * c.hkv * a.chunks;
  a.ctas = static_cast<int>(std::min<long long>(std::min((wg >= 2 ? 1 : 2) * sms, kMaxDecodeCtas), most));
  a.records = wg > 1 ? static_cast<int>(std::min<long long>(a.ctas, most / c.max_pages)) : a.ctas;
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.table = c.table;
  a.lens = c.lens;
  a.v = static_cast<const uint8_t*>(c.v);
  a.page_stride = c.page_stride;
  a.head_stride = c.head_stride;
  a.q = static_cast<const __nv_bfloat16*>(q.data);
  a.q_b = q.batch_stride;
  a.q_h = q.head_stride;
  a.q_t = q.tok_stride;
  a.out = static_cast<__nv_bfloat16*>(const_cast<void*>(out.data));
  a.o_b = out.batch_stride;
  a.o_h = out.head_stride;
  a.o_t = out.tok_stride;
  a.c = scale * 1.4426950408889634f;
  a.part = reinterpret_cast<float*>(ws + L.part);
  a.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  a.split = reinterpret_cast<Split*>(ws + L.split);
  a.lse = weights_out ? reinterpret_cast<float*>(ws + L.lse) : nullptr;
  a.scores = weights_out ? reinterpret_cast<float*>(ws + L.scores) : nullptr;
  a.status = reinterpret_cast<DevStatus*>(ws);
  cudaError_t e = wg == 1 ? launch_groups<1>(maps, a, st) : wg == 2 ? launch_groups<2>(maps, a, st)
                                                                    : launch_groups<4>(maps, a, st);
  if (e != cudaSuccess) return e;
  const unsigned rows = static_cast<unsigned>(std::min(kr, a.rows));
  e = launch_dependent(join_kernel, dim3(static_cast<unsigned>(a.records), rows), kJoinThreads, 0, st, a, kr);
  if (e != cudaSuccess || weights_out == nullptr) return e;
  const unsigned blocks = static_cast<unsigned>((c.max_pages * kB + kWeightKeys - 1) / kWeightKeys);
  return launch_dependent(weights_kernel, dim3(blocks, static_cast<unsigned>(c.hkv), static_cast<unsigned>(c.batch)),
                          kWeightThreads, 0, st, a, weights_in, weights_out);
}

}  // namespace crisp
