// Attention of a few new tokens over the paged 8-bit cache.
//
// Per kv head the rows are the G query heads times the q_len tokens, kR of
// them at a time. One page (128 keys) is one tile; codes kc, vc in e4m3 with
// the page's scales ks, vs:
//   S^T = Kc Q'^T        tcgen05.mma kind::f8f6f4: A = the K page (M = 128 keys, K-major), B = Q' (N = 2 kR)
//   p   = 2^(s - m_t)    softmax warps, m_t = the row's largest s of the tile
//   O^T = Vc^T P'^T      A = the V page (M = 128 features, MN-major), B = P' (N = 2 kR, 128 keys)
//   acc = acc 2^(m - m') + O^T vs 2^(m_t - m')      fp32 registers, m' = max(m, m_t)
// K and V go from HBM by TMA to shared memory and into the tensor cores as
// they are: nothing dequantises them. The other operand is made of two e4m3
// pieces, x = hi + lo / 16 (rows r and kR + r of B): a bf16 q at a power-of-two
// row scale is exactly that sum down to 2^-14 of the row's largest element;
// p (scaled to 256 at the tile's maximum) is off by at most 2^-8 of itself, as
// a bf16 p would be. O^T is read back every tile, so that page scales and the
// running maximum act in fp32 and a tile of small p is as exact as any other.
//
// The work is the list of all tiles of the batch, item (sequence, kv head, row
// chunk) by item; every CTA takes an equal run of it, so ragged batches stay
// balanced and one long sequence spreads over the chip. An item inside one
// CTA's run is finished there; the others leave (m, l, acc) per CTA and
// join_kernel adds them in CTA order: results do not depend on timing.
//
// Warps: 0-3 softmax and accumulation (thread t: key t of a tile, feature t
// of the output), 4 TMA, 5 MMA issue (and TMEM), 6 the Q' operand.
#include <algorithm>
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace crisp {
using namespace ptx;

namespace {

constexpr int kWorkers = 4;                       // softmax warps
constexpr int kTmaWarp = 4, kMmaWarp = 5, kQWarp = 6;
constexpr int kThreads = 7 * 32;
constexpr uint32_t kPage = kB * kD;               // bytes of a page of one head, K or V
constexpr int kMaxTail = kMaxQLen - 1;            // keys that only some of the rows see
constexpr float kLo = 16.f;                       // the second piece's scale

// Rows a CTA takes at once and the page slots that leave two CTAs per SM.
template <int kR>
struct Cfg {
  static constexpr int slots = kR == 8 ? 6 : kR == 16 ? 5 : 4;
  static constexpr int N = 2 * kR;                          // columns of B
  static constexpr uint32_t op = N * 128;                   // bytes of Q' or P'
  static constexpr uint32_t smem = 1024 + slots * kPage + 4 * op;
  static constexpr uint32_t tmem = 4 * N;                   // S and O, two buffers each
};

template <int kR>
struct Shared {
  uint64_t full[6], empty[6];          // page slots
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], drain;
  uint32_t tmem_base;
  int abort;
  int warp_sum[8];
  float qs[2][kR];                     // q scale * scale * log2(e) per row
  float red[2][kWorkers][kR];          // warps' row maxima (sums at an item's end)
  float ref[kWorkers][kR];             // m_t - 8 (0 for a row without keys), per warp
  float alpha[kWorkers][2][kR], wl[kWorkers][2][kR];
  float tail[2][kR][kMaxTail + 1];     // p of keys that only some rows see
};

struct Args {
  int batch, hkv, group, q_len, rows, chunks, num_pages, max_pages, ctas;
  const float *k_scale, *v_scale;
  const int32_t *table, *lens;
  const uint8_t* v;                    // for the tail keys
  int64_t page_stride, head_stride;
  const __nv_bfloat16* q;
  int64_t q_b, q_h, q_t;
  __nv_bfloat16* out;
  int64_t o_b, o_h, o_t;
  float c;                             // scale * log2(e)
  float* part;                         // [2 ctas][kR][128]
  float2* part_ml;                     // [2 ctas][kR]  (m, l)
  float* lse;                          // [items][kR]   log2 sum of 2^s, +inf for a row without keys
  float* scores;                       // [batch][hkv][rows][128 max_pages] or null
  DevStatus* status;
};

__device__ __forceinline__ int clamped_len(const Args& a, int b, bool& bad) {
  const int n = a.lens[b], cap = a.max_pages * kB;
  bad = n < 0 || n > cap;
  return min(max(n, 0), cap);
}

// The CTAs that share `total` tiles: every one of them gets a tile.
__device__ __forceinline__ int sharing(long long total, int ctas) {
  return static_cast<int>(total < ctas ? total : ctas);
}
// First tile of run c of `runs`, and the run that holds tile t.
__device__ __forceinline__ long long run_begin(long long total, int c, int runs) { return total * c / runs; }
__device__ __forceinline__ int run_of(long long total, long long t, int runs) {
  return static_cast<int>(((t + 1) * runs - 1) / total);
}

// One tile of the list.
struct Tile {
  int b, gc;       // sequence; kv head * chunks + row chunk
  int page;        // page of the sequence
  int pages;       // pages of the sequence
  int len;         // tokens of the sequence
};

// pre[b]: pages of the sequences before b.
__device__ __forceinline__ Tile find_tile(const int* pre, const Args& a, long long t) {
  const int hc = a.hkv * a.chunks;
  int lo = 0, hi = a.batch - 1;  // the last b with pre[b] * hc <= t that has pages: pre[b + 1] * hc > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<long long>(pre[mid + 1]) * hc > t) hi = mid;
    else lo = mid + 1;
  }
  Tile x;
  x.b = lo;
  x.pages = pre[lo + 1] - pre[lo];
  const int rem = static_cast<int>(t - static_cast<long long>(pre[lo]) * hc);
  x.gc = rem / x.pages;
  x.page = rem - x.gc * x.pages;
  bool bad;
  x.len = clamped_len(a, lo, bad);
  return x;
}

// The page id of a tile, -1 if the table holds none of the pool's.
__device__ __forceinline__ int page_id(const Args& a, const Tile& x) {
  const int id = a.table[static_cast<int64_t>(x.b) * a.max_pages + x.page];
  return id >= 0 && id < a.num_pages ? id : -1;
}

template <class T>
__device__ __forceinline__ T bcast(T v, int lane) {
  return __shfl_sync(0xffffffffu, v, lane);
}

__device__ __forceinline__ void fail(int* abort, DevStatus* st, uint32_t where) {
  *reinterpret_cast<volatile int*>(abort) = 1;
  report_error(st, CRISP_ERR_TIMEOUT, where);
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* abort) {
  const bool ok = mbar_wait(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}

// Slot positions in the order the products need them: K0 K1 V0 K2 V1 .. K(n-1) V(n-2) V(n-1).
__device__ __forceinline__ int k_pos(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int v_pos(int i, int n) { return i < n - 1 ? 2 * i + 2 : 2 * n - 1; }

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

// 2 kR accumulator columns: v[r] = hi + lo / 16.
template <int kR>
__device__ __forceinline__ void load_rows(uint32_t taddr, float (&v)[kR]) {
  if constexpr (kR == 8) {
    uint32_t x[16];
    tmem_ld16(taddr, x);
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = fmaf(__uint_as_float(x[8 + r]), 1.f / kLo, __uint_as_float(x[r]));
  } else if constexpr (kR == 16) {
    uint32_t x[32];
    tmem_ld32(taddr, x);
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r] = fmaf(__uint_as_float(x[16 + r]), 1.f / kLo, __uint_as_float(x[r]));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t x[16], y[16];
      tmem_ld16(taddr + 16 * h, x);
      tmem_ld16(taddr + 32 + 16 * h, y);
#pragma unroll
      for (int r = 0; r < 16; ++r)
        v[16 * h + r] = fmaf(__uint_as_float(y[r]), 1.f / kLo, __uint_as_float(x[r]));
    }
  }
}

template <int kR>
__global__ void __launch_bounds__(kThreads, 2)
    decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                  const __grid_constant__ Args a) {
  using C = Cfg<kR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* slots = base;
  uint8_t* sQ = base + C::slots * kPage;  // two buffers
  uint8_t* sP = sQ + 2 * C::op;           // two buffers
  int* pre = reinterpret_cast<int*>(sP + 2 * C::op);
  __shared__ Shared<kR> sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    sh.abort = 0;
    for (int s = 0; s < C::slots; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.q_full[s], 1);
      mbar_init(&sh.q_empty[s], 2);  // the last score product of the item; the softmax warps' end of it
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.p_full[s], kWorkers * 32);
      mbar_init(&sh.o_full[s], 1);
    }
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem_base, C::tmem);
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  // Pages before each sequence (an inclusive scan over the batch, a block of sequences at a time).
  int before = 0;
  if (threadIdx.x == 0) pre[0] = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int n = 0;
    if (b < a.batch) {
      bool bad;
      n = (clamped_len(a, b, bad) + kB - 1) / kB;
      if (bad && blockIdx.x == 0) report_error(a.status, CRISP_ERR_BOUNDS, 0x601);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += up;
    }
    if (lane == 31) sh.warp_sum[warp] = n;
    __syncthreads();
    int add = before;
    for (int w = 0; w < warp; ++w) add += sh.warp_sum[w];
    if (b < a.batch) pre[b + 1] = n + add;
    for (int w = 0; w < kThreads / 32; ++w) before += sh.warp_sum[w];
    __syncthreads();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = sh.tmem_base;
  const long long total = static_cast<long long>(before) * a.hkv * a.chunks;
  const int runs = sharing(total, a.ctas), run = static_cast<int>(blockIdx.x);
  const long long t_lo = run < runs ? run_begin(total, run, runs) : 0;
  const int n = run < runs ? static_cast<int>(run_begin(total, run + 1, runs) - t_lo) : 0;

  if (n > 0 && warp == kTmaWarp) {
    // Tiles by 32: each lane looks up one tile's page, lane 0 issues the copies.
    bool go = true;
    int pos = 0;
    int zk = 0, gk = 0, zv = 0, gv = 0;  // the tile being loaded (K), and the one before (V)
    auto load = [&](const CUtensorMap* map, int z, int g) {
      const int s = pos % C::slots;
      if (!mbar_wait(&sh.empty[s], ((pos / C::slots) & 1) ^ 1, &sh.abort)) {
        fail(&sh.abort, a.status, 0x610);
        go = false;
        return;
      }
      ++pos;
      if (z >= 0) {
        mbar_arrive_expect_tx(&sh.full[s], kPage);
        tma_load_4d(slots + s * kPage, map, &sh.full[s], 0, 0, g, z);
      } else {
        mbar_arrive(&sh.full[s]);  // a bad page id: nothing is copied, and the tile counts as empty
      }
    };
    for (int i0 = 0; i0 < n; i0 += 32) {
      int z = -1, g = 0;
      if (i0 + lane < n) {
        const Tile x = find_tile(pre, a, t_lo + i0 + lane);
        z = page_id(a, x);
        g = x.gc / a.chunks;
        if (z < 0) report_error(a.status, CRISP_ERR_BOUNDS, 0x602);
      }
      for (int k = 0; k < 32 && i0 + k < n; ++k) {
        zv = zk;
        gv = gk;
        zk = bcast(z, k);
        gk = bcast(g, k);
        if (lane == 0 && go) load(&tk, zk, gk);
        if (lane == 0 && go && i0 + k > 0) load(&tv, zv, gv);
      }
    }
    if (lane == 0) {
      if (go) load(&tv, zk, gk);
      // Every copy issued has landed before the CTA ends (a bounded wait that
      // ignores the abort flag).
      const int never = 0;
      for (int q = max(0, pos - C::slots); q < pos; ++q)
        mbar_wait(&sh.full[q % C::slots], (q / C::slots) & 1, &never);
    }
  } else if (n > 0 && warp == kMmaWarp) {
    constexpr uint32_t idesc_qk = idesc_e4m3_f32(128, C::N, false, false);
    constexpr uint32_t idesc_pv = idesc_e4m3_f32(128, C::N, true, false);
    const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024), dp = sdesc_sw128(smem_u32(sP), 16, 1024);
    bool go = true;
    int item = -1;  // items begun
    // first/last tile of an item in this run: bits of the 32 tiles looked up by the lanes
    uint32_t first = 0, last = 0;
    int held = -1;
    auto flags = [&](int i) {
      if (i / 32 == held) return;
      held = i / 32;
      bool f = false, l = false;
      const int t = held * 32 + lane;
      if (t < n) {
        const Tile x = find_tile(pre, a, t_lo + t);
        f = t == 0 || x.page == 0;
        l = t == n - 1 || x.page == x.pages - 1;
      }
      first = __ballot_sync(0xffffffffu, f);
      last = __ballot_sync(0xffffffffu, l);
    };
    auto issue_qk = [&](int i) {
      flags(i);
      if (first >> (i & 31) & 1u) {
        ++item;
        if (!mbar_wait(&sh.q_full[item & 1], (item >> 1) & 1, &sh.abort)) go = false;
      }
      const int pos = k_pos(i), s = pos % C::slots;
      if (go && !mbar_wait(&sh.full[s], (pos / C::slots) & 1, &sh.abort)) go = false;
      go = __all_sync(0xffffffffu, go);
      if (!go) return;
      tc_fence_after();
      if (lane == 0) {
        const uint64_t dk = sdesc_sw128(smem_u32(slots + s * kPage), 16, 1024);
        const uint64_t dqi = dq + (item & 1) * (C::op >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)  // 32 features a step
          umma_f8_ss(tmem + (i & 1) * C::N, dk + 2 * kk, dqi + 2 * kk, idesc_qk, kk > 0);
        umma_commit(&sh.s_full[i & 1]);
        umma_commit(&sh.empty[s]);
        if (last >> (i & 31) & 1u) umma_commit(&sh.q_empty[item & 1]);
      }
      __syncwarp();
    };
    issue_qk(0);
    if (go && n > 1) issue_qk(1);
    for (int i = 0; go && i < n; ++i) {
      const int pos = v_pos(i, n), s = pos % C::slots;
      if (!mbar_wait(&sh.p_full[i & 1], (i >> 1) & 1, &sh.abort)) go = false;
      if (go && !mbar_wait(&sh.full[s], (pos / C::slots) & 1, &sh.abort)) go = false;
      go = __all_sync(0xffffffffu, go);
      if (!go) break;
      tc_fence_after();
      if (lane == 0) {
        const uint64_t dv = sdesc_sw128(smem_u32(slots + s * kPage), 1024, 1024);
        const uint64_t dpi = dp + (i & 1) * (C::op >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)  // 32 keys a step: 4096 bytes of V, 32 of P'
          umma_f8_ss(tmem + 2 * C::N + (i & 1) * C::N, dv + 256 * kk, dpi + 2 * kk, idesc_pv, kk > 0);
        umma_commit(&sh.o_full[i & 1]);
        umma_commit(&sh.empty[s]);
      }
      __syncwarp();
      if (i + 2 < n) issue_qk(i + 2);
    }
    if (lane == 0) {
      if (!go) fail(&sh.abort, a.status, 0x611);
      // Every product has completed before TMEM is released (bounded, ignores the abort flag).
      umma_commit(&sh.drain);
      const int never = 0;
      if (!mbar_wait(&sh.drain, 0, &never)) fail(&sh.abort, a.status, 0x612);
    }
  } else if (n > 0 && warp == kQWarp) {
    // Q' of each item of the run: one row at a time, four features a lane.
    int item = 0;
    for (int t = 0; t < n; ++item) {
      const Tile x = find_tile(pre, a, t_lo + t);
      const int buf = item & 1, g = x.gc / a.chunks, r0 = (x.gc % a.chunks) * kR;
      if (!warp_wait(&sh.q_empty[buf], ((item >> 1) & 1) ^ 1, &sh.abort)) {
        if (lane == 0) fail(&sh.abort, a.status, 0x613);
        break;
      }
      uint8_t* dst = sQ + buf * C::op;
#pragma unroll 4
      for (int r = 0; r < kR; ++r) {
        const int row = r0 + r;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (row < a.rows) {
          const int i = row / a.group, h = g * a.group + row % a.group;
          const uint2 w = *reinterpret_cast<const uint2*>(a.q + x.b * a.q_b + h * a.q_h + i * a.q_t + lane * 4);
          v[0] = __uint_as_float(w.x << 16);
          v[1] = __uint_as_float(w.x & 0xffff0000u);
          v[2] = __uint_as_float(w.y << 16);
          v[3] = __uint_as_float(w.y & 0xffff0000u);
        }
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!isfinite(v[e])) v[e] = __int_as_float(0x7fffffff);  // the row's scores become NaN
          amax = fmaxf(amax, fabsf(v[e]));                          // ignores NaN
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int e2 = scale_exponent(amax);
        const float inv = exp2_int(-e2);
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float y0 = v[e] * inv, y1 = v[e + 1] * inv;
          const uint16_t h2 = pack_e4m3x2(y0, y1);
          float h0, h1;
          unpack_e4m3x2(h2, h0, h1);
          hi |= static_cast<uint32_t>(h2) << (8 * e);
          lo |= static_cast<uint32_t>(pack_e4m3x2((y0 - h0) * kLo, (y1 - h1) * kLo)) << (8 * e);
        }
        const uint32_t at = (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;  // kR is a multiple of 8
        *reinterpret_cast<uint32_t*>(dst + r * 128 + at) = hi;
        *reinterpret_cast<uint32_t*>(dst + (kR + r) * 128 + at) = lo;
        if (lane == 0) sh.qs[buf][r] = exp2_int(e2) * a.c;
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[buf]);
      t += x.pages - x.page;
    }
  } else if (n > 0 && warp < kWorkers) {
    const int tid = threadIdx.x;
    const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
    const int my_row = lane & (kR - 1);            // row of the lane-held statistics
    constexpr int kShift = kR == 8 ? 2 : kR == 16 ? 1 : 0;  // warp_rows: lane L holds row L >> kShift
    float acc[kR], l[kR];
    float m = -INFINITY;                            // running maximum of row my_row, base 2
    int item = -1;
    bool ok = true;
    // tiles by 32: each lane looks up one
    Tile mine{};
    int z = -1;
    float ks = 0.f, vs = 0.f;
    // of the tile whose O is still to be added
    float o_vs = 0.f;
    int o_tail0 = 0, o_ntail = 0, o_g = 0, o_z = -1, o_row0 = 0;

    auto add_o = [&](int i) -> bool {
      if (!warp_wait(&sh.o_full[i & 1], (i >> 1) & 1, &sh.abort)) return false;
      tc_fence_after();
      float o[kR];
      load_rows<kR>(tmem + lane_addr + 2 * C::N + (i & 1) * C::N, o);
      if (o_ntail > 0) {
        // keys that only the later tokens see: added here, one by one, so
        // that what they hold does not reach the rows that do not see them
        const uint8_t* vp = a.v + o_z * a.page_stride + o_g * a.head_stride + tid;
        for (int k = 0; k < o_ntail; ++k) {
          float val, none;
          unpack_e4m3x2(vp[(o_row0 + k) * kD], val, none);
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            const float p = sh.tail[i & 1][r][o_tail0 + k];
            if (p >= 0.f || p != p) o[r] = fmaf(p, val, o[r]);  // -1: not seen
          }
        }
      }
      const float* al = sh.alpha[warp][i & 1];
      const float* wl = sh.wl[warp][i & 1];
#pragma unroll
      for (int r = 0; r < kR; ++r) acc[r] = fmaf(o[r], wl[r] * o_vs, acc[r] * al[r]);
      return true;
    };

    for (int i = 0; ok && i < n; ++i) {
      const int k32 = i & 31, buf = i & 1;
      if (k32 == 0) {
        z = -1;
        ks = vs = 0.f;
        if (i + lane < n) {
          mine = find_tile(pre, a, t_lo + i + lane);
          z = page_id(a, mine);
          if (z >= 0) {
            const int64_t at = static_cast<int64_t>(z) * a.hkv + mine.gc / a.chunks;
            ks = a.k_scale[at];
            vs = a.v_scale[at];
          }
        }
      }
      const int b = bcast(mine.b, k32), gc = bcast(mine.gc, k32), page = bcast(mine.page, k32);
      const int pages = bcast(mine.pages, k32), len = bcast(mine.len, k32), zt = bcast(z, k32);
      const float kst = bcast(ks, k32), vst = bcast(vs, k32);
      const int g = gc / a.chunks, r0 = (gc - g * a.chunks) * kR;
      if (i == 0 || page == 0) {
        ++item;
        m = -INFINITY;
#pragma unroll
        for (int r = 0; r < kR; ++r) acc[r] = l[r] = 0.f;
      }
      if (!warp_wait(&sh.s_full[buf], (i >> 1) & 1, &sh.abort) ||
          !warp_wait(&sh.q_full[item & 1], (item >> 1) & 1, &sh.abort)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float s[kR];
      load_rows<kR>(tmem + lane_addr + buf * C::N, s);
      const float* qs = sh.qs[item & 1];
#pragma unroll
      for (int r = 0; r < kR; ++r) s[r] *= qs[r] * kst;
      // Row r belongs to token (r0 + r) / group, which sees keys below all_see + that.
      const int key0 = page * kB, all_see = zt < 0 ? -1 : len - (a.q_len - 1);
      const bool partial = key0 + kB > all_see;
      if (partial) {
        const int past = zt < 0 ? kB : key0 + tid - all_see;  // < 0: every row sees the key
#pragma unroll
        for (int r = 0; r < kR; ++r)
          if (past >= 0 && (zt < 0 || past >= (r0 + r) / a.group)) s[r] = -INFINITY;
      }
      if (a.scores != nullptr) {
        float* dst = a.scores + ((static_cast<int64_t>(b) * a.hkv + g) * a.rows + r0) *
                                    (static_cast<int64_t>(a.max_pages) * kB) + key0 + tid;
#pragma unroll
        for (int r = 0; r < kR; ++r)
          if (r0 + r < a.rows) dst[static_cast<int64_t>(r) * a.max_pages * kB] = s[r];
      }
      // The tile's row maxima, over the four warps.
      {
        float t[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) t[r] = s[r];
        const float wm = warp_rows<kR, true>(t);
        if ((lane & ((1 << kShift) - 1)) == 0) sh.red[buf][warp][lane >> kShift] = wm;
      }
      named_bar_sync(1, kWorkers * 32);
      {
        const float mt = fmaxf(fmaxf(sh.red[buf][0][my_row], sh.red[buf][1][my_row]),
                               fmaxf(sh.red[buf][2][my_row], sh.red[buf][3][my_row]));
        const float mn = fmaxf(m, mt);
        // a row without keys so far: nothing to scale, and weight 0 (2^(-inf))
        const float base2 = mn == -INFINITY ? 0.f : mn;
        if (lane < kR) {
          sh.ref[warp][my_row] = mt == -INFINITY ? 0.f : mt - 8.f;
          sh.alpha[warp][buf][my_row] = ex2_approx(m - base2);
          sh.wl[warp][buf][my_row] = ex2_approx(mt - base2 - 8.f);
        }
        m = mn;
      }
      __syncwarp();
      uint8_t* dst = sP + buf * C::op;
      const int ntail_lo = max(all_see - key0, 0);           // first row of the page some rows do not see
      const int row_end = min(max(len - key0, 0), kB);       // tokens held in the page
      const bool is_tail = partial && zt >= 0 && tid >= ntail_lo && tid < row_end;
      const uint32_t col = ((tid >> 4) << 4), in16 = tid & 15;
#pragma unroll
      for (int r = 0; r < kR; r += 2) {
        float p0 = ex2_approx(s[r] - sh.ref[warp][r]), p1 = ex2_approx(s[r + 1] - sh.ref[warp][r + 1]);
        l[r] = fmaf(p0, sh.wl[warp][buf][r], l[r] * sh.alpha[warp][buf][r]);
        l[r + 1] = fmaf(p1, sh.wl[warp][buf][r + 1], l[r + 1] * sh.alpha[warp][buf][r + 1]);
        if (is_tail) {
          const int past = key0 + tid - all_see;
          sh.tail[buf][r][past] = past < (r0 + r) / a.group ? p0 : -1.f;
          sh.tail[buf][r + 1][past] = past < (r0 + r + 1) / a.group ? p1 : -1.f;
          p0 = p1 = 0.f;
        }
        const uint16_t hi = pack_e4m3x2(p0, p1);
        float h0, h1;
        unpack_e4m3x2(hi, h0, h1);
        const uint16_t lo = pack_e4m3x2((p0 - h0) * kLo, (p1 - h1) * kLo);
        const uint32_t c0 = (col ^ ((r & 7) << 4)) + in16, c1 = (col ^ (((r + 1) & 7) << 4)) + in16;
        dst[r * 128 + c0] = static_cast<uint8_t>(hi);
        dst[(r + 1) * 128 + c1] = static_cast<uint8_t>(hi >> 8);
        dst[(kR + r) * 128 + c0] = static_cast<uint8_t>(lo);
        dst[(kR + r + 1) * 128 + c1] = static_cast<uint8_t>(lo >> 8);
      }
      if (partial) {
        // V rows that not every row sees become zeros: p = 0 there, and what
        // the page holds (anything past the end) must not matter
        const int pos = v_pos(i, n), sl = pos % C::slots;
        if (!warp_wait(&sh.full[sl], (pos / C::slots) & 1, &sh.abort)) {
          ok = false;
          break;
        }
        if (tid >= ntail_lo) {
          uint4* rowp = reinterpret_cast<uint4*>(slots + sl * kPage + tid * 128);
#pragma unroll
          for (int e = 0; e < 8; ++e) rowp[e] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_async_shared();
      tc_fence_before();
      mbar_arrive(&sh.p_full[buf]);
      // The tile before: its product has run meanwhile.
      if (i > 0 && page != 0 && !add_o(i - 1)) {
        ok = false;
        break;
      }
      o_vs = vst;
      o_z = zt;
      o_g = g;
      o_row0 = ntail_lo;
      o_tail0 = key0 + ntail_lo - all_see;
      o_ntail = partial && zt >= 0 ? max(row_end - ntail_lo, 0) : 0;
      if (o_ntail > 0) named_bar_sync(2, kWorkers * 32);  // every warp's tail p is written
      if (i == n - 1 || page == pages - 1) {
        // End of the item in this run.
        if (!add_o(i)) {
          ok = false;
          break;
        }
        const float wsum = warp_rows<kR, false>(l);
        named_bar_sync(1, kWorkers * 32);  // red's readers of this tile are done
        if ((lane & ((1 << kShift) - 1)) == 0) sh.red[buf][warp][lane >> kShift] = wsum;
        if (lane < kR) sh.ref[warp][my_row] = m;
        named_bar_sync(1, kWorkers * 32);
        if (tid == 0) mbar_arrive(&sh.q_empty[item & 1]);
        const long long t_item = t_lo + i - page;  // the item's first tile
        const bool whole = t_item >= t_lo && page == pages - 1;
        const int slot = 2 * blockIdx.x + (t_item < t_lo ? 0 : 1);
        const int nr = min(kR, a.rows - r0);
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          if (r >= nr) break;
          const float ls = (sh.red[buf][0][r] + sh.red[buf][1][r]) + (sh.red[buf][2][r] + sh.red[buf][3][r]);
          if (whole) {
            const int tok = (r0 + r) / a.group, h = g * a.group + (r0 + r) % a.group;
            const float v = ls == 0.f ? 0.f : acc[r] / ls;
            a.out[b * a.o_b + h * a.o_h + tok * a.o_t + tid] = __float2bfloat16_rn(v);
          } else {
            a.part[(static_cast<int64_t>(slot) * kR + r) * kD + tid] = acc[r];
          }
        }
        if (tid < nr) {
          const float ls = (sh.red[buf][0][tid] + sh.red[buf][1][tid]) + (sh.red[buf][2][tid] + sh.red[buf][3][tid]);
          const float mr = sh.ref[warp][tid];
          if (whole)
            a.lse[(static_cast<int64_t>(b) * a.hkv * a.chunks + gc) * kR + tid] =
                ls == 0.f ? INFINITY : mr + log2f(ls);
          else
            a.part_ml[slot * kR + tid] = make_float2(mr, ls);
        }
        named_bar_sync(1, kWorkers * 32);  // red and ref are free again
      }
    }
    if (!ok && lane == 0) fail(&sh.abort, a.status, 0x614);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, C::tmem);
}

constexpr int kJoinThreads = 512;
constexpr int kWeightKeys = 2 * kJoinThreads;  // keys a block of the weights part takes

// Joins the items that several CTAs worked on, and adds the weights. Blocks
// [0, batch * hkv * rows): one row of the output. The rest: kWeightKeys keys of
// one sequence and kv head.
__global__ void __launch_bounds__(kJoinThreads)
    join_kernel(const __grid_constant__ Args a, int kr, const float* w_in, float* w_out, int key_blocks) {
  __shared__ float f[kMaxDecodeCtas];
  __shared__ float red[kJoinThreads];
  __shared__ int pages_before[kJoinThreads / 32], pages_all[kJoinThreads / 32];
  __shared__ float lse[kMaxGroupRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows_total = a.batch * a.hkv * a.rows;
  const bool is_row = static_cast<int>(blockIdx.x) < rows_total;
  int b, g, row = 0, kb = 0;
  if (is_row) {
    row = blockIdx.x % a.rows;
    const int bg = blockIdx.x / a.rows;
    b = bg / a.hkv;
    g = bg % a.hkv;
  } else {
    const int x = blockIdx.x - rows_total;
    kb = x % key_blocks;
    b = x / key_blocks / a.hkv;
    g = x / key_blocks % a.hkv;
  }
  bool bad;
  const int len = clamped_len(a, b, bad), pages = (len + kB - 1) / kB;
  if (!is_row && kb * kWeightKeys >= len) return;
  // pages of the sequences before b, and of all
  int mine = 0, all = 0;
  for (int x = tid; x < a.batch; x += kJoinThreads) {
    bool bx;
    const int p = (clamped_len(a, x, bx) + kB - 1) / kB;
    all += p;
    if (x < b) mine += p;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mine += __shfl_xor_sync(0xffffffffu, mine, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  if (lane == 0) {
    pages_before[warp] = mine;
    pages_all[warp] = all;
  }
  __syncthreads();
  mine = all = 0;
  for (int w = 0; w < kJoinThreads / 32; ++w) {
    mine += pages_before[w];
    all += pages_all[w];
  }
  const int hc = a.hkv * a.chunks;
  const long long total = static_cast<long long>(all) * hc;
  grid_dep_wait();

  // The CTAs of row chunk c of this (sequence, kv head): c0 .. c1.
  auto span = [&](int c, int& c0, int& c1) {
    const long long s0 = static_cast<long long>(mine) * hc + static_cast<long long>(g * a.chunks + c) * pages;
    c0 = run_of(total, s0, sharing(total, a.ctas));
    c1 = run_of(total, s0 + pages - 1, sharing(total, a.ctas));
  };
  auto slot_of = [](int c, int c0) { return 2 * c + (c == c0 ? 1 : 0); };

  if (is_row) {
    const int tok = row / a.group, h = g * a.group + row % a.group;
    __nv_bfloat16* dst = a.out + b * a.o_b + h * a.o_h + tok * a.o_t;
    if (pages == 0) {
      if (tid < kD) dst[tid] = __float2bfloat16_rn(0.f);
      return;
    }
    const int chunk = row / kr, r = row - chunk * kr;
    int c0, c1;
    span(chunk, c0, c1);
    if (c0 == c1) return;  // finished by its CTA
    const int nc = c1 - c0 + 1;
    // factors 2^(m_c - M), in CTA order; nc <= kMaxDecodeCtas <= kJoinThreads
    float mc = -INFINITY, lc = 0.f;
    if (tid < nc) {
      const float2 ml = a.part_ml[slot_of(c0 + tid, c0) * kr + r];
      mc = ml.x;
      lc = ml.y;
    }
    red[tid] = mc;
    __syncthreads();
    float M = -INFINITY;
    for (int x = lane; x < nc; x += 32) M = fmaxf(M, red[x]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    __syncthreads();
    if (tid < nc) {
      const float fc = ex2_approx(mc - (M == -INFINITY ? 0.f : M));
      f[tid] = fc;
      red[tid] = fc * lc;
    }
    __syncthreads();
    float L = 0.f;
    for (int x = lane; x < nc; x += 32) L += red[x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    __syncthreads();
    const int d = tid & (kD - 1), part = tid / kD;
    float acc = 0.f;
#pragma unroll 4
    for (int x = part; x < nc; x += kJoinThreads / kD)
      acc = fmaf(f[x], a.part[(static_cast<int64_t>(slot_of(c0 + x, c0)) * kr + r) * kD + d], acc);
    red[tid] = acc;
    __syncthreads();
    if (tid < kD) {
      float v = 0.f;
      for (int x = 0; x < kJoinThreads / kD; ++x) v += red[tid + x * kD];
      dst[tid] = __float2bfloat16_rn(L == 0.f ? 0.f : v / L);
    }
    return;
  }

  // weights_out = weights_in + sum over the rows of 2^(s - lse)
  for (int row2 = warp; row2 < a.rows; row2 += kJoinThreads / 32) {
    const int chunk = row2 / kr, r = row2 - chunk * kr;
    int c0, c1;
    span(chunk, c0, c1);
    float v;
    if (c0 == c1) {
      v = a.lse[(static_cast<int64_t>(b) * hc + g * a.chunks + chunk) * kr + r];
    } else {
      float M = -INFINITY;
      for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, a.part_ml[slot_of(c, c0) * kr + r].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      float L = 0.f;
      for (int c = c0 + lane; c <= c1; c += 32) {
        const float2 ml = a.part_ml[slot_of(c, c0) * kr + r];
        L = fmaf(ex2_approx(ml.x - (M == -INFINITY ? 0.f : M)), ml.y, L);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      v = L == 0.f ? INFINITY : M + log2f(L);
    }
    if (lane == 0) lse[row2] = v;
  }
  __syncthreads();
  const int64_t cap = static_cast<int64_t>(a.max_pages) * kB, bg = static_cast<int64_t>(b) * a.hkv + g;
  const int key = kb * kWeightKeys + tid * 2;
  if (key >= len) return;
  const float* sc = a.scores + bg * a.rows * cap + key;
  float w0 = 0.f, w1 = 0.f;
#pragma unroll 4
  for (int r = 0; r < a.rows; ++r) {
    const float2 s = *reinterpret_cast<const float2*>(sc + r * cap);
    w0 += ex2_approx(s.x - lse[r]);
    w1 += ex2_approx(s.y - lse[r]);
  }
  const int64_t at = bg * cap + key;
  if (w_in != nullptr) {
    w0 += w_in[at];
    if (key + 1 < len) w1 += w_in[at + 1];
  }
  if (key + 1 < len)
    *reinterpret_cast<float2*>(w_out + at) = make_float2(w0, w1);
  else
    w_out[at] = w0;
}

int rows_per_cta(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

template <int kR>
cudaError_t launch_rows(const KvMaps& maps, const Args& a, cudaStream_t st) {
  using C = Cfg<kR>;
  const uint32_t smem = C::smem + (a.batch + 1) * 4;
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<kR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  decode_kernel<kR><<<a.ctas, kThreads, smem, st>>>(maps.k, maps.v, a);
  return cudaGetLastError();
}

}  // namespace

int decode_row_chunks(int rows) { return (rows + rows_per_cta(rows) - 1) / rows_per_cta(rows); }

DecodeLayout decode_layout(const crisp_kv_cache& c, int hq, int q_len, bool with_weights) {
  const int rows = hq / c.hkv * q_len, kr = rows_per_cta(rows), chunks = (rows + kr - 1) / kr;
  DecodeLayout L{};
  size_t o = align_up(sizeof(DevStatus));
  L.part = o;    o = align_up(o + size_t(2) * kMaxDecodeCtas * kr * kD * 4);
  L.part_ml = o; o = align_up(o + size_t(2) * kMaxDecodeCtas * kr * 8);
  L.lse = o;     o = align_up(o + size_t(c.batch) * c.hkv * chunks * kr * 4);
  L.scores = o;
  if (with_weights) o = align_up(o + size_t(c.batch) * c.hkv * rows * c.max_pages * kB * 4);
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
  const int kr = rows_per_cta(a.rows);
  a.chunks = (a.rows + kr - 1) / kr;
  a.num_pages = c.num_pages;
  a.max_pages = c.max_pages;
  // two CTAs per SM, and no more than the table can hold tiles
  const long long most = static_cast<long long>(c.batch) * c.max_pages * c.hkv * a.chunks;
  a.ctas = static_cast<int>(std::min<long long>(std::min(2 * sms, kMaxDecodeCtas), most));
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
  a.lse = reinterpret_cast<float*>(ws + L.lse);
  a.scores = weights_out ? reinterpret_cast<float*>(ws + L.scores) : nullptr;
  a.status = reinterpret_cast<DevStatus*>(ws);
  cudaError_t e = kr == 8 ? launch_rows<8>(maps, a, st) : kr == 16 ? launch_rows<16>(maps, a, st)
                                                                   : launch_rows<32>(maps, a, st);
  if (e != cudaSuccess) return e;
  const int key_blocks = weights_out ? (c.max_pages * kB + kWeightKeys - 1) / kWeightKeys : 0;
  const long long blocks = static_cast<long long>(c.batch) * c.hkv * (a.rows + key_blocks);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel, a, kr, weights_in, weights_out, key_blocks);
}

}  // namespace crisp
