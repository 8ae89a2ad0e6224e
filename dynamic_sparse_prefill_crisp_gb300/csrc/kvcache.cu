// The paged 8-bit cache: writing tokens into it, and cutting it down by
// accumulated attention weight.
//
// A page of a head is 128 tokens x 128 e4m3 codes with one power-of-two scale
// (csrc/common.cuh, scale_exponent). Both kernels that write pages take one
// page of one head per CTA: 8 threads hold a row (16 codes each), 32 rows at a
// time, the whole page in registers between its maximum and its codes, so
// every value is read once. They are bound by HBM.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace crisp {
using namespace ptx;
namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 256;
constexpr int kRowThreads = 8;                    // threads of a row, 16 codes each
constexpr int kRowsAtOnce = kThreads / kRowThreads;
constexpr int kPasses = kB / kRowsAtOnce;         // 4

__device__ __forceinline__ float block_max(float v, float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_max(v);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return warp_max(red[lane & (kThreads / 32 - 1)]);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// |x| of a finite x, 0 for the others.
__device__ __forceinline__ float finite_abs(float x) {
  const float y = fabsf(x);
  return y <= 3.402823466e38f ? y : 0.f;
}
// The code of x at inv = 1 / scale; a non-finite x becomes NaN.
__device__ __forceinline__ float scaled(float x, float inv) {
  return fabsf(x) <= 3.402823466e38f ? x * inv : __int_as_float(0x7fffffff);
}
// The larger magnitudes of two bf16 pairs (as 16-bit integers they order the
// same way; infinities and NaN are 0x7f80 and above).
constexpr uint32_t kBf16Inf = 0x7f80u;
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
// Eight bf16 values as codes at inv = 1 / scale, a power of two (so the product
// is exact, or far below half the smallest code).
template <bool kFinite>
__device__ __forceinline__ uint2 codes8(const uint4& x, float inv) {
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = (&x.x)[e];
    float a, b;
    if (kFinite) {
      fmul2(a, b, bf16_lo(w), bf16_hi(w), inv, inv);
    } else {
      a = scaled(bf16_lo(w), inv);
      b = scaled(bf16_hi(w), inv);
    }
    c[e] = pack_e4m3x2(a, b);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Two codes rounded again at `ratio` times their values, for a power of two
// 2^-24 <= ratio <= 2^15: e4m3 values and their products with it are fp16
// values (down to 2^-24, far below what a code can hold), so there is one rounding.
__device__ __forceinline__ uint32_t rescale2(uint32_t c, uint32_t ratio2) {
  uint16_t d;
  asm("{\n\t.reg .b32 h;\n\t"
      "cvt.rn.f16x2.e4m3x2 h, %1;\n\t"
      "mul.f16x2 h, h, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 %0, h;\n\t}"
      : "=h"(d)
      : "h"(static_cast<uint16_t>(c)), "r"(ratio2));
  return d;
}
__device__ __forceinline__ uint32_t rescale4_any(uint32_t c, float ratio) {
  float a0, a1, a2, a3;
  unpack_e4m3x2(static_cast<uint16_t>(c), a0, a1);
  unpack_e4m3x2(static_cast<uint16_t>(c >> 16), a2, a3);
  return static_cast<uint32_t>(pack_e4m3x2(a0 * ratio, a1 * ratio)) |
         static_cast<uint32_t>(pack_e4m3x2(a2 * ratio, a3 * ratio)) << 16;
}
// 16 codes rounded again at `ratio` times their values.
__device__ __forceinline__ uint4 rescale16(uint4 c, float ratio) {
  if (ratio == 1.f) return c;
  if ((__float_as_uint(ratio) & 0x7FFFFFu) == 0u && ratio >= 0x1p-24f && ratio <= 0x1p15f) {
    uint32_t r2;
    asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(r2) : "f"(ratio));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = (&c.x)[e];
      (&c.x)[e] = rescale2(w, r2) | rescale2(w >> 16, r2) << 16;
    }
    return c;
  }
  // tiny codes scaled up a long way, or a scale that is no power of two
  return make_uint4(rescale4_any(c.x, ratio), rescale4_any(c.y, ratio), rescale4_any(c.z, ratio),
                    rescale4_any(c.w, ratio));
}
// The largest magnitude of 16 codes (NaN is passed over).
__device__ __forceinline__ float max16(const uint4& c) {
  uint32_t m = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = (&c.x)[e];
    asm("{\n\t.reg .b32 a, b;\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 a, l;\n\tcvt.rn.f16x2.e4m3x2 b, h;\n\t"
        "and.b32 a, a, 0x7fff7fff;\n\tand.b32 b, b, 0x7fff7fff;\n\t"
        "max.f16x2 a, a, b;\n\tmax.f16x2 %0, %0, a;\n\t}"
        : "+r"(m)
        : "r"(w));
  }
  float x, y;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(x), "=f"(y)
      : "r"(m));
  return fmaxf(x, y);
}

struct Pool {
  uint8_t* codes;
  float* scale;
};

// New tokens of one page of one head, K or V: the page's new scale from the
// new values (and its old scale, where it held tokens before them), the new
// tokens' codes, and the old tokens' codes again if the scale grew.
__global__ void __launch_bounds__(kThreads, 4)
    append_kernel(Pool pk, Pool pv, int64_t page_stride, int64_t head_stride, int hkv, int num_pages, int max_pages,
                  const int32_t* table, const int32_t* lens, const int32_t* new_lens, int n_new, crisp_tokens kt,
                  crisp_tokens vt, DevStatus* status) {
  __shared__ float red[kThreads / 32];
  const int g = blockIdx.y >> 1, b = blockIdx.z;
  const bool is_v = blockIdx.y & 1;
  const int cap = max_pages * kB;
  grid_dep_launch();
  grid_dep_wait();
  int len = lens[b], cnt = new_lens != nullptr ? new_lens[b] : n_new;
  const bool bad = len < 0 || len > cap || cnt < 0 || cnt > min(n_new, len);
  if (bad && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) report_error(status, CRISP_ERR_BOUNDS, 0x701);
  len = min(max(len, 0), cap);
  cnt = min(max(cnt, 0), min(n_new, len));
  const int start = len - cnt;
  const int page = start / kB + static_cast<int>(blockIdx.x);
  const int lo = page * kB;  // position of the page's row 0
  if (cnt == 0 || lo >= len) return;
  const int32_t* entry = table + static_cast<int64_t>(b) * max_pages + page;
  const crisp_tokens t = is_v ? vt : kt;
  const auto* src = static_cast<const __nv_bfloat16*>(t.data) + b * t.batch_stride + g * t.head_stride;
  const int col = (threadIdx.x & (kRowThreads - 1)) * 16, row0 = threadIdx.x / kRowThreads;
  const int first = max(start - lo, 0), end = min(len - lo, kB);  // rows [first, end) are new, [0, first) old
  // the new values are asked for before the page is looked up
  uint4 x[kPasses][2];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int row = row0 + p * kRowsAtOnce;
    x[p][0] = x[p][1] = make_uint4(0u, 0u, 0u, 0u);
    if (row >= first && row < end) {
      const auto* s = reinterpret_cast<const uint4*>(src + (lo + row - start) * t.tok_stride + col);
      x[p][0] = __ldcs(s);
      x[p][1] = __ldcs(s + 1);
    }
  }
  const int id = *entry;
  if (id < 0 || id >= num_pages) {
    if (blockIdx.y == 0 && threadIdx.x == 0) report_error(status, CRISP_ERR_BOUNDS, 0x702);
    return;
  }
  const Pool pool = is_v ? pv : pk;
  uint8_t* codes = pool.codes + id * page_stride + g * head_stride;
  float* scale = pool.scale + static_cast<int64_t>(id) * hkv + g;
  const bool held = first > 0;
  const float s_old = held ? *scale : 0.f;
  uint32_t top = 0u;
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max_abs2(top, (&x[p][h].x)[e]);
  top = max(top & 0xffffu, top >> 16);
  const bool finite = top < kBf16Inf;  // this thread's values
  float amax = bf16_lo(top);
  if (!finite) {
    amax = 0.f;
    for (int p = 0; p < kPasses; ++p)
      for (int h = 0; h < 2; ++h)
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = (&x[p][h].x)[e];
          amax = fmaxf(amax, fmaxf(finite_abs(bf16_lo(w)), finite_abs(bf16_hi(w))));
        }
  }
  amax = block_max(amax, red);
  float s = exp2_int(scale_exponent(amax));
  if (held) s = fmaxf(s, s_old);
  const float inv = 1.f / s;  // exact for the powers of two that the library writes
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int row = row0 + p * kRowsAtOnce;
    if (row >= first && row < end) {
      const uint2 lo8 = finite ? codes8<true>(x[p][0], inv) : codes8<false>(x[p][0], inv);
      const uint2 hi8 = finite ? codes8<true>(x[p][1], inv) : codes8<false>(x[p][1], inv);
      *reinterpret_cast<uint4*>(codes + row * kD + col) = make_uint4(lo8.x, lo8.y, hi8.x, hi8.y);
    } else if (row < first && s != s_old) {
      uint4* at = reinterpret_cast<uint4*>(codes + row * kD + col);
      *at = rescale16(*at, s_old * inv);
    }
  }
  if (threadIdx.x == 0 && (!held || s != s_old)) *scale = s;
}

// ------------------------------------------------------------------ eviction
// Which tokens stay: the `keep` largest of n keys, equal keys by lowest
// position. Keys order as the weights do (32-bit integers; NaN above every
// number), tokens that always stay above all. The keep-th largest key is found
// digit by digit from the top (11 + 11 + 10 bits): a histogram of the keys that
// match the digits found so far, then the digit in which the keep-th falls. A
// last pass writes the kept positions in order. The keys are read four times,
// from L2 after the first; a long sequence takes a cluster of 16 CTAs with a
// contiguous part each, which read each other's histograms through
// distributed shared memory (512k tokens: one CTA would read 2 MB a pass).
constexpr int kSelThreads = 512;
constexpr int kBins = 2048;
constexpr int kClusterLen = 16384;  // capacities from which a cluster is used
constexpr int kCluster = 16;
constexpr int kAhead = 4;           // loads of four keys a thread has in flight

__device__ __forceinline__ uint32_t weight_key(float w) {
  // + 0 makes one zero of both and one NaN of all (0x7fffffff)
  const int u = __float_as_int(w + 0.f);
  return min(static_cast<uint32_t>(u ^ (u >> 31 | INT32_MIN)), 0xfffffffeu);
}
// Keys of the four weights from position i on; those at or past n do not count
// (0, which is no weight's key).
__device__ __forceinline__ void weight_keys(const float4& w, int i, int sink, int tail, int n, uint32_t (&key)[4]) {
  key[0] = weight_key(w.x);
  key[1] = weight_key(w.y);
  key[2] = weight_key(w.z);
  key[3] = weight_key(w.w);
  if (i < sink || i + 4 > tail) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i + e < sink || i + e >= tail) key[e] = 0xffffffffu;
      if (i + e >= n) key[e] = 0u;
    }
  }
}

// Inclusive scan over the block of one value a thread; returns it and the total.
__device__ __forceinline__ int block_scan(int v, int* warp_tot, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_tot[warp] = v;
  __syncthreads();
  int w = lane < kSelThreads / 32 ? warp_tot[lane] : 0;
  int before = lane < warp ? w : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    w += __shfl_xor_sync(0xffffffffu, w, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  total = w;
  __syncthreads();
  return v + before;
}

template <int kC>
__global__ void __launch_bounds__(kSelThreads, 2)
    select_kernel(const float* weights, const int32_t* lens, int32_t* new_lens, int hkv, int cap, int keep, int sink,
                  int recent, const int32_t* table, int num_pages, float* new_weights, int64_t new_cap, int32_t* kept,
                  int64_t kept_stride, int32_t* list, int64_t list_stride, DevStatus* status) {
  __shared__ alignas(8) int hist[2][kBins];
  __shared__ int bin_total[2][kC > 1 ? kBins / kC : 1];
  __shared__ int warp_tot[kSelThreads / 32];
  __shared__ int digit, above_digit;
  __shared__ alignas(8) int tot[2][kAhead * kSelThreads / 32];
  __shared__ int own[2];  // this CTA's keys above the threshold, and equal to it
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x;
  const int part = kC > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int bg = blockIdx.x / kC, b = bg / hkv;
  int n = lens[b];
  if (bg % hkv == 0 && part == 0 && tid == 0) {
    if (n < 0 || n > cap) report_error(status, CRISP_ERR_BOUNDS, 0x711);
    new_lens[b] = min(min(max(n, 0), cap), keep);
  }
  n = min(max(n, 0), cap);
  const float* w = weights + static_cast<int64_t>(bg) * cap;
  int32_t* dst = list + bg * list_stride;
  float* dst_w = new_weights != nullptr ? new_weights + bg * new_cap : nullptr;
  int32_t* dst_pos = kept != nullptr ? kept + bg * kept_stride : nullptr;
  const int32_t* pages = table + static_cast<int64_t>(b) * (cap / kB);
  // Position i is kept in place `at`: where its codes are (-1: on no page), and what it carries along.
  auto emit = [&](int at, int i, int id, float weight) {
    dst[at] = id >= 0 && id < num_pages ? id * kB + i % kB : -1;
    if (dst_pos) dst_pos[at] = i;
    if (dst_w) dst_w[at] = weight;
  };
  // this CTA's part of the positions, whole groups of four
  const int quads = (n + 3) / 4;
  const int lo = static_cast<int>(static_cast<int64_t>(quads) * part / kC) * 4;
  const int hi = min(static_cast<int>(static_cast<int64_t>(quads) * (part + 1) / kC) * 4, n);
  if (n <= keep) {  // uniform over the cluster
    for (int i = lo + tid; i < hi; i += kSelThreads) emit(i, i, pages[i / kB], w[i]);
    return;
  }
  const int tail = n - recent;
  // rows are 512-byte aligned and cap is a multiple of 128: whole groups of four are there
  auto load4 = [&](int i) { return *reinterpret_cast<const float4*>(w + i); };

  constexpr int kTurn = kSelThreads * 4;  // positions the block takes with one load a thread
  float4 v[kAhead];                       // a part of one turn is read once
  auto load_first = [&]() {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (lo + u * kTurn + tid * 4 < hi) v[u] = load4(lo + u * kTurn + tid * 4);
  };

  uint32_t found = 0;   // the digits found, in place
  int want = keep;      // the threshold is the want-th largest of the keys that match them
  int above_own = 0;    // this CTA's keys above (this thread's part)
  constexpr int kShift[3] = {21, 10, 0};
  constexpr uint32_t kMask[3] = {2047u, 2047u, 1023u};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    int* h = hist[pass & 1];
    for (int x = tid; x < kBins; x += kSelThreads) h[x] = 0;
    __syncthreads();
    const uint32_t fixed = pass == 0 ? 0u : ~0u << kShift[pass - 1];
    if (pass == 0 || hi - lo > kTurn * kAhead) load_first();
    for (int i0 = lo + tid * 4; i0 < hi; i0 += kTurn * kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kTurn;
        if (i >= hi) break;
        uint32_t key[4];
        weight_keys(v[u], i, sink, tail, n, key);
        if (i + kTurn * kAhead < hi) v[u] = load4(i + kTurn * kAhead);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // a key of 0 counts only in the first pass, in bin 0, where no weight's key falls (-inf is in bin 3)
          if (pass == 0 || ((key[e] ^ found) & fixed) == 0u)
            atomicAdd(&h[pass == 0 ? key[e] >> kShift[0] : (key[e] >> kShift[pass]) & kMask[pass]], 1);
        }
      }
    }
    if (kC > 1) cg::this_cluster().sync();
    else __syncthreads();
    // thread t takes kPer bins of the whole sequence, the largest first
    constexpr int kPer = kBins / kSelThreads;
    const int top = kBins - 1 - kPer * tid;
    int c[kPer], sum = 0;
    if constexpr (kC > 1) {
      // CTA r adds up bins r * kOwn .. of all CTAs; everyone then reads the sums
      // from their owners (reading every CTA's whole histogram instead made
      // all CTAs queue at one after the other: 40 us a pass against 3)
      constexpr int kOwn = kBins / kC, kSplit = kSelThreads / kOwn;
      int* total = bin_total[pass & 1];
      if (tid < kOwn) total[tid] = 0;
      __syncthreads();
      int part_sum = 0;
#pragma unroll
      for (int u = 0; u < kC / kSplit; ++u)
        part_sum += cg::this_cluster().map_shared_rank(h, tid / kOwn * (kC / kSplit) + u)[part * kOwn + tid % kOwn];
      if (part_sum) atomicAdd(&total[tid % kOwn], part_sum);
      cg::this_cluster().sync();
#pragma unroll
      for (int u = 0; u < kPer; ++u)
        c[u] = cg::this_cluster().map_shared_rank(total, (top - u) / kOwn)[(top - u) % kOwn];
    } else {
#pragma unroll
      for (int u = 0; u < kPer; ++u) c[u] = h[top - u];
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) sum += c[u];
    int all;
    const int incl = block_scan(sum, warp_tot, all);
    int before = incl - sum;
    if (before < want && want <= incl) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        if (before < want && want <= before + c[u]) {
          digit = top - u;
          above_digit = before;
        }
        before += c[u];
      }
    }
    __syncthreads();
    const int d = digit;
    want -= above_digit;
    found |= static_cast<uint32_t>(d) << kShift[pass];
    // this CTA's own keys above the digit
    int mine = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) mine += top - u > d ? h[top - u] : 0;
    above_own += mine;
    if (kC > 1 && pass == 2) {
      int own_above;
      block_scan(above_own, warp_tot, own_above);
      if (tid == 0) {
        own[0] = own_above;
        own[1] = h[d];
      }
    }
  }
  // Kept before this CTA's part: all keys above the threshold `found`, and the
  // first `want` equal to it.
  int gt = 0, eq = 0;
  if (kC > 1) {
    cg::this_cluster().sync();
    if ((tid & 31) < part) {
      const int* o = cg::this_cluster().map_shared_rank(own, tid & 31);
      gt = o[0];
      eq = o[1];
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    cg::this_cluster().sync();  // nobody's shared memory goes away while it is read
  }
  // A turn's kept positions are first put in order in shared memory (where the
  // histograms were), then written out by neighbouring threads.
  constexpr int kWarps = kSelThreads / 32;
  const int warp = tid >> 5, lane = tid & 31;
  static_assert(sizeof(hist) >= 2 * kTurn * kAhead, "a turn's offsets fit the histograms");
  uint16_t* order = reinterpret_cast<uint16_t*>(hist);
  if (hi - lo > kTurn * kAhead) load_first();
  for (int i0 = lo, turn = 0; i0 < hi; i0 += kTurn * kAhead, ++turn) {
    // counts before this thread: keys above in the high half, equal in the low
    // (at most 8192 of either in a turn)
    int before[kAhead];
    uint32_t above = 0, tie = 0;  // one bit a key
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * kTurn + tid * 4;
      int mine = 0;
      if (i < hi) {
        uint32_t key[4];
        weight_keys(v[u], i, sink, tail, n, key);
        if (i + kTurn * kAhead < hi) v[u] = load4(i + kTurn * kAhead);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          above |= (key[e] > found ? 1u : 0u) << (4 * u + e);
          tie |= (key[e] == found ? 1u : 0u) << (4 * u + e);
        }
        mine = __popc(above >> (4 * u) & 15u) << 16 | __popc(tie >> (4 * u) & 15u);
      }
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      before[u] = incl - mine;
      if (lane == 31) tot[turn & 1][u * kWarps + warp] = incl;
    }
    __syncthreads();
    // the kAhead * kWarps totals in order, two a lane
    static_assert(kAhead * kWarps == 64, "two totals a lane");
    const int2 pair = *reinterpret_cast<const int2*>(&tot[turn & 1][2 * lane]);
    int incl = pair.x + pair.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const int all = __shfl_sync(0xffffffffu, incl, 31), excl = incl - pair.x - pair.y;
    const int begin = gt + min(eq, want);  // the turn's first place
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int place = u * kWarps + warp;  // of this warp's total
      const int at2 = __shfl_sync(0xffffffffu, excl, place / 2), first = __shfl_sync(0xffffffffu, pair.x, place / 2);
      const int base = before[u] + at2 + (place & 1 ? first : 0);
      int g1 = gt + (base >> 16) - begin, e1 = eq + (base & 0xffff);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool a = above >> (4 * u + e) & 1u, t = tie >> (4 * u + e) & 1u;
        if (a || (t && e1 < want)) order[g1 + min(e1, want)] = static_cast<uint16_t>(u * kTurn + tid * 4 + e);
        g1 += a;
        e1 += t;
      }
    }
    gt += all >> 16;
    eq += all & 0xffff;
    const int count = gt + min(eq, want) - begin;
    __syncthreads();
    for (int j0 = tid; j0 < count; j0 += kSelThreads * 4) {
      int i[4], id[4];
      float f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        i[u] = j0 + u * kSelThreads < count ? i0 + order[j0 + u * kSelThreads] : i0;
        id[u] = pages[i[u] / kB];
        f[u] = dst_w ? w[i[u]] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j0 + u * kSelThreads < count) emit(begin + j0 + u * kSelThreads, i[u], id[u], f[u]);
    }
  }
}

// Asynchronous copies of 16 or 4 bytes to shared memory; nothing is read and
// zeros are written where `there` is false.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// New pages: their kept tokens' codes gathered from the old pages (a row is
// 128 contiguous bytes), the scale their values need, and the codes at it. A
// CTA takes every gridDim.x-th page of one head, K and V together. A row is
// found through the list, so a page is three dependent reads and a write: the
// copies of the next two pages are under way while one is packed (each thread
// copies what it packs itself, so nothing but the maximum is shared). Without
// that, with four such CTAs on an SM, 512k -> 128k tokens took 105 us against
// 79 at the copy rate.
constexpr int kStages = 3;
struct PackStage {
  uint4 codes[2][kPasses][kThreads];
  float scale[2][kPasses][kRowsAtOnce];  // copied and read by a row's first thread
};
constexpr size_t kPackSmem = kStages * sizeof(PackStage);

__global__ void __launch_bounds__(kThreads, 2)
    pack_kernel(Pool sk, Pool sv, int64_t s_page, int64_t s_head, int s_max, Pool dk, Pool dv, int64_t d_page,
                int64_t d_head, const int32_t* d_table, int d_num, int d_max, int hkv, const int32_t* lens, int keep,
                int new_pages, int items, const int32_t* list, int64_t list_stride, DevStatus* status) {
  grid_dep_launch();
  extern __shared__ uint8_t smem_raw[];
  PackStage* stages = reinterpret_cast<PackStage*>(smem_raw);
  __shared__ float red[2][2][kThreads / 32];
  const int tid = threadIdx.x;
  const int col = (tid & (kRowThreads - 1)) * 16, row0 = tid / kRowThreads;
  grid_dep_wait();

  // The next item of this CTA that has rows: its head, rows, and page (-1: none left).
  struct Item {
    int g, rows, id;
  };
  int at = static_cast<int>(blockIdx.x);
  auto start = [&](PackStage& st) -> Item {
    Item it{0, 0, -1};
    for (; at < items; at += static_cast<int>(gridDim.x)) {
      const int page = at % new_pages, bg = at / new_pages, b = bg / hkv;
      const int n = min(min(max(lens[b], 0), s_max * kB), keep);
      if (n <= page * kB) continue;
      it.g = bg - b * hkv;
      it.rows = min(n - page * kB, kB);
      it.id = d_table[static_cast<int64_t>(b) * d_max + page];
      if (it.id < 0 || it.id >= d_num) {
        if (tid == 0) report_error(status, CRISP_ERR_BOUNDS, 0x712);
        it.id = -1;
        continue;
      }
      const int32_t* where = list + bg * list_stride + page * kB;
      int src[kPasses];
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int row = row0 + p * kRowsAtOnce;
        src[p] = row < it.rows ? where[row] : 0;
      }
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const bool there = row0 + p * kRowsAtOnce < it.rows && src[p] >= 0;
        if (src[p] < 0) {
          report_error(status, CRISP_ERR_BOUNDS, 0x713);
          src[p] = 0;
        }
        const int64_t from = src[p] / kB * s_page + it.g * s_head + (src[p] % kB) * kD + col;
        const int64_t sat = static_cast<int64_t>(src[p] / kB) * hkv + it.g;
        copy16(&st.codes[0][p][tid], sk.codes + from, there);
        copy16(&st.codes[1][p][tid], sv.codes + from, there);
        if (col == 0) {
          copy4(&st.scale[0][p][row0], sk.scale + sat, there);
          copy4(&st.scale[1][p][row0], sv.scale + sat, there);
        }
      }
      at += static_cast<int>(gridDim.x);
      break;
    }
    copies_commit();
    return it;
  };

  Item now = start(stages[0]), next = start(stages[1]);
  for (int k = 0; now.id >= 0; ++k) {
    const Item after = start(stages[(k + 2) % kStages]);
    copies_wait<2>();
    const PackStage& st = stages[k % kStages];
    float amax[2] = {0.f, 0.f}, s[2][kPasses];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        s[x][p] = __shfl_sync(0xffffffffu, col == 0 ? st.scale[x][p][row0] : 0.f, tid & 31 & ~(kRowThreads - 1));
        amax[x] = fmaxf(amax[x], max16(st.codes[x][p][tid]) * s[x][p]);
      }
    // both maxima over the block
    float(&rd)[2][kThreads / 32] = red[k & 1];
    amax[0] = warp_max(amax[0]);
    amax[1] = warp_max(amax[1]);
    if ((tid & 31) == 0) {
      rd[0][tid >> 5] = amax[0];
      rd[1][tid >> 5] = amax[1];
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float sn = exp2_int(scale_exponent(warp_max(rd[x][tid & (kThreads / 32 - 1)]))), inv = 1.f / sn;
      uint8_t* codes = (x ? dv : dk).codes + now.id * d_page + now.g * d_head;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int row = row0 + p * kRowsAtOnce;
        if (row >= now.rows) continue;
        *reinterpret_cast<uint4*>(codes + row * kD + col) = rescale16(st.codes[x][p][tid], s[x][p] * inv);
      }
      if (tid == 0) (x ? dv : dk).scale[static_cast<int64_t>(now.id) * hkv + now.g] = sn;
    }
    now = next;
    next = after;
  }
  copies_wait<0>();
}

Pool k_pool(const crisp_kv_cache& c) { return {static_cast<uint8_t*>(c.k), c.k_scale}; }
Pool v_pool(const crisp_kv_cache& c) { return {static_cast<uint8_t*>(c.v), c.v_scale}; }

}  // namespace

cudaError_t launch_kv_append(const crisp_kv_cache& c, const crisp_tokens& k_new, const crisp_tokens& v_new, int n_new,
                             const int32_t* new_lens, DevStatus* status, cudaStream_t st) {
  const unsigned reach = static_cast<unsigned>((n_new + kB - 2) / kB + 1);  // pages n_new tokens can touch
  return launch_dependent(append_kernel, dim3(reach, static_cast<unsigned>(2 * c.hkv), static_cast<unsigned>(c.batch)),
                          kThreads, 0, st, k_pool(c), v_pool(c), c.page_stride, c.head_stride, c.hkv, c.num_pages,
                          c.max_pages, c.table, static_cast<const int32_t*>(c.lens), new_lens, n_new, k_new, v_new,
                          status);
}

cudaError_t launch_kv_evict(const crisp_kv_cache& src, const crisp_kv_cache& dst, const float* weights, int keep,
                            int sink, int recent, float* new_weights, int32_t* kept, int32_t* list,
                            int64_t list_stride, DevStatus* status, int sms, cudaStream_t st) {
  const int cap = src.max_pages * kB;
  const int64_t new_cap = static_cast<int64_t>(dst.max_pages) * kB;
  const bool wide = cap >= kClusterLen;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attrs[2] = {};
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kSelThreads);
  cfg.gridDim = dim3(static_cast<unsigned>(src.batch * src.hkv * (wide ? kCluster : 1)));
  cudaError_t e;
  if (wide) {
    e = cudaFuncSetAttribute(select_kernel<kCluster>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = kCluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  e = cudaLaunchKernelEx(&cfg, wide ? select_kernel<kCluster> : select_kernel<1>, weights,
                         static_cast<const int32_t*>(src.lens), dst.lens, src.hkv, cap, keep, sink, recent, src.table,
                         src.num_pages, new_weights, new_cap, kept, new_cap, list, list_stride, status);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(pack_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kPackSmem));
  if (e != cudaSuccess) return e;
  const int new_pages = (min(keep, cap) + kB - 1) / kB;
  const int items = src.batch * src.hkv * new_pages;
  return launch_dependent(pack_kernel, dim3(static_cast<unsigned>(min(items, 2 * sms))), kThreads, kPackSmem, st,
                          k_pool(src), v_pool(src), src.page_stride, src.head_stride, src.max_pages, k_pool(dst),
                          v_pool(dst), dst.page_stride, dst.head_stride, dst.table, dst.num_pages, dst.max_pages,
                          src.hkv, static_cast<const int32_t*>(src.lens), keep, new_pages, items,
                          static_cast<const int32_t*>(list), list_stride, status);
}

}  // namespace crisp
