// The paged 8-bit cache: writing tokens into it, and cutting it down by
// accumulated attention weight.
//
// A page of a head is 128 tokens x 128 e4m3 codes with one power-of-two scale
// (csrc/common.cuh, scale_exponent). In the kernels that write pages 8 threads
// hold a row (16 codes each), 32 rows at a time, and every value is read once:
// an append CTA has a page of one head, K or V, in registers between its
// maximum and its codes; a packing CTA takes page after page of a head, K and V
// together, and has them in shared memory, copied there ahead. They are bound
// by HBM.
#include <cuda_bf16.h>
#include <type_traits>

#include "common.cuh"
#include "ptx.cuh"

namespace crisp {
using namespace ptx;

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
// tokens' codes, and the old tokens' codes again if the scale grew. Bound by
// HBM from a few thousand tokens on (32k tokens of 8 heads: 33 us, 6.2 TB/s);
// before bf16 values were handled in pairs it was bound by instructions (39
// us). A token for each of 64 sequences takes 4.7 us, a chain of four reads.
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
// digit by digit from the top (10 + 11 + 11 bits): a histogram of the keys that
// match the digits found so far, then the digit in which the keep-th falls. A
// last pass writes the kept positions in order.
//
// A cache of up to kChunk positions takes one CTA per sequence and kv head and
// one launch (2175 tokens: 5.7 us, of it 3 in barriers and scans; the keys stay
// in registers up to 8192). A longer one is cut into chunks of kChunk, a CTA
// each and a launch per pass, so that a few long rows fill the chip. The chunks'
// first histograms go to the workspace and every CTA of the next pass adds up
// its row's; the later ones, mostly zeros, are added to the row's totals, which
// the first pass clears. The last pass needs to know what stands in the chunks
// before its own: each leaves, for every last digit, how many of its keys are at
// or above it. 8 rows of 512k tokens take 29 us this way (one token kept, and
// packed), 39 when every pass adds up all histograms, 48 with a cluster of 16
// CTAs per row (8 such clusters fill half the SMs).
constexpr int kSelThreads = 512;
constexpr int kBins = 2048;
constexpr int kPer = kBins / kSelThreads;  // bins of a thread
constexpr int kAhead = 4;                  // loads of four keys a thread has in flight
constexpr int kTurn = kSelThreads * 4;     // positions the block takes with one load a thread
constexpr int kChunk = 2 * kAhead * kTurn;
constexpr int kFirstBins = 1024;           // of the first digit
__host__ __device__ constexpr int digit_shift(int pass) { return pass == 0 ? 22 : pass == 1 ? 11 : 0; }
__host__ __device__ constexpr uint32_t digit_mask(int pass) { return pass == 0 ? kFirstBins - 1u : kBins - 1u; }

// What a chunk's CTA knows: the digits found, how many of the keys that match
// them are still wanted, and how many of the chunk's keys are above them.
struct SelState {
  uint32_t found;
  int want, above, pad;
};

struct SelArgs {
  const float* weights;
  const int32_t* lens;
  int32_t* new_lens;
  const int32_t* table;
  float* new_weights;   // or null
  int32_t* kept;        // or null
  int32_t* list;
  int64_t new_cap, list_stride;
  int hkv, cap, keep, sink, recent, num_pages;
  uint16_t* hist;       // [batch hkv][chunks][kFirstBins]  (long caches)
  uint16_t* from;       // [batch hkv][chunks][kBins]  keys whose last digit is that or above
  int* total;           // [2][batch hkv][kBins]  the rows' second and third histograms
  SelState* state;      // [batch hkv][chunks]
  int chunks, rows;     // rows: batch hkv
  DevStatus* status;
};

__device__ __forceinline__ uint32_t weight_key(float w) {
  // + 0 makes one zero of both and one NaN of all (0x7fffffff)
  const int u = __float_as_int(w + 0.f);
  return min(static_cast<uint32_t>(u ^ (u >> 31 | INT32_MIN)), 0xfffffffeu);
}

// One sequence and kv head.
struct SelRow {
  int n, sink, tail;
  const float* w;
  const int32_t* pages;
  __device__ __forceinline__ SelRow(const SelArgs& a, int b, int bg) {
    n = min(max(a.lens[b], 0), a.cap);
    sink = a.sink;
    tail = n - a.recent;
    w = a.weights + static_cast<int64_t>(bg) * a.cap;
    pages = a.table + static_cast<int64_t>(b) * (a.cap / kB);
  }
  // rows are 512-byte aligned and cap is a multiple of 128: whole groups of four are there
  __device__ __forceinline__ float4 load4(int i) const { return *reinterpret_cast<const float4*>(w + i); }
  // Keys of the four weights from position i on; those at or past n do not
  // count (0, which is no weight's key).
  __device__ __forceinline__ void keys(const float4& x, int i, uint32_t (&key)[4]) const {
    key[0] = weight_key(x.x);
    key[1] = weight_key(x.y);
    key[2] = weight_key(x.z);
    key[3] = weight_key(x.w);
    if (i < sink || i + 4 > tail) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (i + e < sink || i + e >= tail) key[e] = 0xffffffffu;
        if (i + e >= n) key[e] = 0u;
      }
    }
  }
};

// Position i is kept in place `at`: where its codes are (-1: on no page), and what it carries along.
__device__ __forceinline__ void emit(const SelArgs& a, int bg, int at, int i, int id, float weight) {
  a.list[bg * a.list_stride + at] = id >= 0 && id < a.num_pages ? id * kB + i % kB : -1;
  if (a.kept != nullptr) a.kept[bg * a.new_cap + at] = i;
  if (a.new_weights != nullptr) a.new_weights[bg * a.new_cap + at] = weight;
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

struct SelShared {
  alignas(8) int hist[2][kBins];  // (and, in the last pass, a turn's kept positions)
  alignas(8) int tot[2][kAhead * kSelThreads / 32];
  int warp_tot[kSelThreads / 32];
  int digit, above;
};

// The first turn's keys of [lo, hi).
__device__ __forceinline__ void load_first(const SelRow& r, int lo, int hi, float4 (&v)[kAhead]) {
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int i = lo + u * kTurn + static_cast<int>(threadIdx.x) * 4;
    if (i < hi) v[u] = r.load4(i);
  }
}

// Adds the keys of [lo, hi) that match `found` above digit `pass` to the
// histogram h of that digit; v: the first turn's. Ends with a barrier. Returns,
// in the last pass, how many of this thread's keys are above those that match.
template <int pass>
__device__ __forceinline__ int count(const SelRow& r, int lo, int hi, uint32_t found, int* h, float4 (&v)[kAhead]) {
  for (int x = threadIdx.x; x < kBins; x += kSelThreads) h[x] = 0;
  __syncthreads();
  constexpr uint32_t fixed = pass == 0 ? 0u : ~0u << digit_shift(pass - 1);
  int above = 0;
  for (int i0 = lo + static_cast<int>(threadIdx.x) * 4; i0 < hi; i0 += kTurn * kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * kTurn;
      if (i >= hi) break;
      uint32_t key[4];
      r.keys(v[u], i, key);
      if (i + kTurn * kAhead < hi) v[u] = r.load4(i + kTurn * kAhead);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // a key of 0 counts only in the first pass, in bin 0, where no weight's key falls (-inf is in bin 1)
        if (pass == 0 || ((key[e] ^ found) & fixed) == 0u)
          atomicAdd(&h[(key[e] >> digit_shift(pass)) & digit_mask(pass)], 1);
        if (pass == 2) above += key[e] > (found | ~fixed);
      }
    }
  }
  __syncthreads();
  return above;
}

// The digit in which the want-th largest key falls; c: this thread's kPer bins
// of the row's histogram, the largest (kBins - 1 - kPer * thread) first.
__device__ __forceinline__ void pick(SelShared& sh, const int (&c)[kPer], int pass, uint32_t& found, int& want) {
  const int top = kBins - 1 - kPer * static_cast<int>(threadIdx.x);
  int sum = 0;
#pragma unroll
  for (int u = 0; u < kPer; ++u) sum += c[u];
  int all;
  const int incl = block_scan(sum, sh.warp_tot, all);
  int before = incl - sum;
  if (before < want && want <= incl) {
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if (before < want && want <= before + c[u]) {
        sh.digit = top - u;
        sh.above = before;
      }
      before += c[u];
    }
  }
  __syncthreads();
  want -= sh.above;
  found |= static_cast<uint32_t>(sh.digit) << digit_shift(pass);
}

// Writes the kept positions of [lo, hi): keys above `found`, and those equal to
// it while fewer than `want` of them came before; gt, eq: the row's keys above
// and equal before lo; v: the first turn's keys. A turn's kept positions are
// first put in order in shared memory (where the histograms were), then
// written out by neighbouring threads.
__device__ __forceinline__ void write_kept(const SelArgs& a, const SelRow& r, SelShared& sh, int bg, int lo, int hi,
                                           uint32_t found, int want, int gt, int eq, float4 (&v)[kAhead]) {
  constexpr int kWarps = kSelThreads / 32;
  static_assert(sizeof(sh.hist) >= 2 * kTurn * kAhead, "a turn's offsets fit the histograms");
  static_assert(kAhead * kWarps == 64, "two totals a lane");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint16_t* order = reinterpret_cast<uint16_t*>(sh.hist);
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
        r.keys(v[u], i, key);
        if (i + kTurn * kAhead < hi) v[u] = r.load4(i + kTurn * kAhead);
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
      if (lane == 31) sh.tot[turn & 1][u * kWarps + warp] = incl;
    }
    __syncthreads();
    // the kAhead * kWarps totals in order, two a lane
    const int2 pair = *reinterpret_cast<const int2*>(&sh.tot[turn & 1][2 * lane]);
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
        const bool is_above = above >> (4 * u + e) & 1u, is_tie = tie >> (4 * u + e) & 1u;
        if (is_above || (is_tie && e1 < want))
          order[g1 + min(e1, want)] = static_cast<uint16_t>(u * kTurn + tid * 4 + e);
        g1 += is_above;
        e1 += is_tie;
      }
    }
    gt += all >> 16;
    eq += all & 0xffff;
    const int total = gt + min(eq, want) - begin;
    __syncthreads();
    for (int j0 = tid; j0 < total; j0 += kSelThreads * 4) {
      int i[4], id[4];
      float f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        i[u] = j0 + u * kSelThreads < total ? i0 + order[j0 + u * kSelThreads] : i0;
        id[u] = r.pages[i[u] / kB];
        f[u] = a.new_weights != nullptr ? r.w[i[u]] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j0 + u * kSelThreads < total) emit(a, bg, begin + j0 + u * kSelThreads, i[u], id[u], f[u]);
    }
  }
}

__device__ __forceinline__ void write_len(const SelArgs& a, int b) {
  const int n = a.lens[b];
  if (n < 0 || n > a.cap) report_error(a.status, CRISP_ERR_BOUNDS, 0x711);
  a.new_lens[b] = min(min(max(n, 0), a.cap), a.keep);
}

// All passes of a row in one CTA.
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const __grid_constant__ SelArgs a) {
  __shared__ SelShared sh;
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x, bg = blockIdx.x, b = bg / a.hkv;
  if (bg % a.hkv == 0 && tid == 0) write_len(a, b);
  const SelRow r(a, b, bg);
  if (r.n <= a.keep) {
    for (int i = tid; i < r.n; i += kSelThreads) emit(a, bg, i, i, r.pages[i / kB], r.w[i]);
    return;
  }
  float4 v[kAhead];
  const bool once = r.n <= kTurn * kAhead;  // one turn: its keys stay in registers
  uint32_t found = 0;
  int want = a.keep;
  const int top = kBins - 1 - kPer * tid;
  int c[kPer];
  auto pass = [&](auto which) {
    constexpr int p = decltype(which)::value;
    if (p == 0 || !once) load_first(r, 0, r.n, v);
    count<p>(r, 0, r.n, found, sh.hist[p & 1], v);
#pragma unroll
    for (int u = 0; u < kPer; ++u) c[u] = sh.hist[p & 1][top - u];
    pick(sh, c, p, found, want);
  };
  pass(std::integral_constant<int, 0>());
  pass(std::integral_constant<int, 1>());
  pass(std::integral_constant<int, 2>());
  if (!once) load_first(r, 0, r.n, v);
  write_kept(a, r, sh, bg, 0, r.n, found, want, 0, 0, v);
}

// The first digit, from the histograms of all chunks of a row; two halves of
// the block take every second chunk.
__device__ __forceinline__ void digest_first(const SelArgs& a, SelShared& sh, int bg, int n, SelState& st) {
  constexpr int kHalf = kSelThreads / 2;
  static_assert(kFirstBins == kPer * kHalf && 2 * kFirstBins == kBins, "a half's threads have the bins among them");
  const int tid = threadIdx.x, half = tid / kHalf, bin = kPer * (tid % kHalf), chunks = (n + kChunk - 1) / kChunk;
  const uint16_t* h = a.hist + static_cast<int64_t>(bg) * a.chunks * kFirstBins + bin;
  int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll 8
  for (int x = half; x < chunks; x += 2) {
    const uint2 q = *reinterpret_cast<const uint2*>(h + static_cast<int64_t>(x) * kFirstBins);
    sum.x += q.x & 0xffffu;
    sum.y += q.x >> 16;
    sum.z += q.y & 0xffffu;
    sum.w += q.y >> 16;
  }
  *reinterpret_cast<int4*>(&sh.hist[1][half * kFirstBins + bin]) = sum;
  __syncthreads();
  const int top = kBins - 1 - kPer * tid;
  int c[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u)
    c[u] = top < kFirstBins ? sh.hist[1][top - u] + sh.hist[1][kFirstBins + top - u] : 0;
  pick(sh, c, 0, st.found, st.want);
}

// The second or third digit, from the row's totals.
__device__ __forceinline__ void digest_total(const SelArgs& a, SelShared& sh, int bg, int pass, SelState& st) {
  const int top = kBins - 1 - kPer * static_cast<int>(threadIdx.x);
  const int4 q = *reinterpret_cast<const int4*>(a.total + (static_cast<int64_t>(pass - 1) * a.rows + bg) * kBins +
                                                top - (kPer - 1));
  const int c[kPer] = {q.w, q.z, q.y, q.x};
  pick(sh, c, pass, st.found, st.want);
}

// Digit `pass` of one chunk.
template <int pass>
__global__ void __launch_bounds__(kSelThreads, 2) chunk_kernel(const __grid_constant__ SelArgs a) {
  __shared__ SelShared sh;
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x, chunk = blockIdx.x, b = blockIdx.z, bg = b * a.hkv + blockIdx.y;
  const SelRow r(a, b, bg);
  const int lo = chunk * kChunk, hi = min(lo + kChunk, r.n);
  if (r.n <= a.keep || lo >= r.n) return;
  float4 v[kAhead];
  load_first(r, lo, hi, v);
  const int64_t at = static_cast<int64_t>(bg) * a.chunks + chunk;
  SelState st{0u, a.keep, 0, 0};
  if (pass == 0 && chunk == 0) {  // every row that goes on has a first chunk
#pragma unroll
    for (int p = 0; p < 2; ++p)
      *reinterpret_cast<int4*>(a.total + (static_cast<int64_t>(p) * a.rows + bg) * kBins + kPer * tid) =
          make_int4(0, 0, 0, 0);
  }
  if (pass == 1) digest_first(a, sh, bg, r.n, st);
  if (pass == 2) {
    st = a.state[at];
    digest_total(a, sh, bg, 1, st);
  }
  const int above = count<pass>(r, lo, hi, st.found, sh.hist[0], v);
  const int4 x = *reinterpret_cast<const int4*>(&sh.hist[0][kPer * tid]);
  if (pass == 0) {
    if (tid < kFirstBins / kPer)
      *reinterpret_cast<uint2*>(a.hist + at * kFirstBins + kPer * tid) =
          make_uint2(static_cast<uint32_t>(x.x) | static_cast<uint32_t>(x.y) << 16,
                     static_cast<uint32_t>(x.z) | static_cast<uint32_t>(x.w) << 16);
    return;
  }
  int* total = a.total + (static_cast<int64_t>(pass - 1) * a.rows + bg) * kBins + kPer * tid;
  if (x.x != 0) atomicAdd(total, x.x);
  if (x.y != 0) atomicAdd(total + 1, x.y);
  if (x.z != 0) atomicAdd(total + 2, x.z);
  if (x.w != 0) atomicAdd(total + 3, x.w);
  if (pass == 2) {
    const int sum = x.x + x.y + x.z + x.w;
    int all;
    const int from = sum - block_scan(sum, sh.warp_tot, all);  // minus what stands in the bins below
    const int f0 = from + all, f1 = f0 - x.x, f2 = f1 - x.y, f3 = f2 - x.z;
    *reinterpret_cast<uint2*>(a.from + at * kBins + kPer * tid) =
        make_uint2(static_cast<uint32_t>(f0) | static_cast<uint32_t>(f1) << 16,
                   static_cast<uint32_t>(f2) | static_cast<uint32_t>(f3) << 16);
    block_scan(above, sh.warp_tot, st.above);
  }
  if (tid == 0) a.state[at] = st;
}

// The kept positions of one chunk.
__global__ void __launch_bounds__(kSelThreads, 2) chunk_kept_kernel(const __grid_constant__ SelArgs a) {
  __shared__ SelShared sh;
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x, chunk = blockIdx.x, b = blockIdx.z, bg = b * a.hkv + blockIdx.y;
  if (chunk == 0 && blockIdx.y == 0 && tid == 0) write_len(a, b);
  const SelRow r(a, b, bg);
  const int lo = chunk * kChunk, hi = min(lo + kChunk, r.n);
  if (r.n <= a.keep) {
    for (int i = lo + tid; i < hi; i += kSelThreads) emit(a, bg, i, i, r.pages[i / kB], r.w[i]);
    return;
  }
  if (lo >= r.n) return;
  float4 v[kAhead];
  load_first(r, lo, hi, v);
  const int64_t row = static_cast<int64_t>(bg) * a.chunks;
  SelState st = a.state[row + chunk];
  digest_total(a, sh, bg, 2, st);
  // keys above, and equal, in the chunks before: a thread each (64 at most)
  static_assert(kMaxSeq / kChunk <= kSelThreads, "a thread for every chunk");
  int gt = 0, eq = 0;
  if (tid < chunk) {
    const uint16_t* from = a.from + (row + tid) * kBins + sh.digit;
    const int next = sh.digit + 1 < kBins ? from[1] : 0;
    gt = a.state[row + tid].above + next;
    eq = from[0] - next;
  }
  int all_gt, all_eq;
  block_scan(gt, sh.warp_tot, all_gt);
  block_scan(eq, sh.warp_tot, all_eq);
  write_kept(a, r, sh, bg, lo, hi, st.found, st.want, all_gt, all_eq, v);
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
// copies what it packs itself, so nothing but the maximum is shared). 512k ->
// 128k tokens of 8 heads: 91 us, 79 at the copy rate (a kept row is 128 bytes
// somewhere in its page); with four plain CTAs on an SM 105 us, and 120 us with
// the codes scaled in fp32.
constexpr int kStages = 3;
struct PackStage {
  uint4 codes[2][kPasses][kThreads];
  float scale[2][kPasses][kRowsAtOnce];  // copied and read by a row's first thread
};
constexpr size_t kPackSmem = kStages * sizeof(PackStage);

__global__ void __launch_bounds__(kThreads, 2)
    pack_kernel(Pool sk, Pool sv, int64_t s_page, int64_t s_head, int s_max, Pool dk, Pool dv, int64_t d_page,
                int64_t d_head, const int32_t* d_table, int d_num, int d_max, int batch, int hkv, const int32_t* lens,
                int keep, int new_pages, int items, const int32_t* list, int64_t list_stride, DevStatus* status) {
  grid_dep_launch();
  extern __shared__ uint8_t smem_raw[];
  PackStage* stages = reinterpret_cast<PackStage*>(smem_raw);
  __shared__ float red[2][2][kThreads / 32];
  __shared__ int held[kMaxBatch];  // what each sequence keeps
  const int tid = threadIdx.x;
  const int col = (tid & (kRowThreads - 1)) * 16, row0 = tid / kRowThreads;
  grid_dep_wait();
  for (int b = tid; b < batch; b += kThreads) held[b] = min(min(max(lens[b], 0), s_max * kB), keep);
  __syncthreads();

  // An item of this CTA (a page that gets rows): its head and rows (0: there are
  // no more), its page, and where the rows of this thread come from.
  struct Look {
    int g, rows, id, src[kPasses];
  };
  int at = static_cast<int>(blockIdx.x);
  // The lookups of the next item; what they read is not needed before copy().
  auto look = [&]() -> Look {
    Look l{};
    for (; at < items && l.rows <= 0; at += static_cast<int>(gridDim.x)) {
      const int page = at % new_pages, bg = at / new_pages, b = bg / hkv;
      l.rows = min(held[b] - page * kB, kB);
      if (l.rows <= 0) continue;
      l.g = bg - b * hkv;
      l.id = d_table[static_cast<int64_t>(b) * d_max + page];
      const int32_t* where = list + bg * list_stride + page * kB;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int row = row0 + p * kRowsAtOnce;
        l.src[p] = row < l.rows ? where[row] : 0;
      }
    }
    l.rows = max(l.rows, 0);
    return l;
  };
  // Starts the copies of an item.
  auto copy = [&](const Look& l, PackStage& st) {
    if (l.rows > 0) {
      if ((l.id < 0 || l.id >= d_num) && tid == 0) report_error(status, CRISP_ERR_BOUNDS, 0x712);
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        if (l.src[p] < 0) report_error(status, CRISP_ERR_BOUNDS, 0x713);
        const int src = max(l.src[p], 0);
        const bool there = row0 + p * kRowsAtOnce < l.rows && l.src[p] >= 0;
        const int64_t from = src / kB * s_page + l.g * s_head + (src % kB) * kD + col;
        const int64_t sat = static_cast<int64_t>(src / kB) * hkv + l.g;
        copy16(&st.codes[0][p][tid], sk.codes + from, there);
        copy16(&st.codes[1][p][tid], sv.codes + from, there);
        if (col == 0) {
          copy4(&st.scale[0][p][row0], sk.scale + sat, there);
          copy4(&st.scale[1][p][row0], sv.scale + sat, there);
        }
      }
    }
    copies_commit();
  };

  Look now = look();
  copy(now, stages[0]);
  Look next = look();
  copy(next, stages[1]);
  Look after = look();
  for (int k = 0; now.rows > 0; ++k) {
    copy(after, stages[(k + 2) % kStages]);
    const Look later = look();
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
    if (now.id >= 0 && now.id < d_num) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float sn = exp2_int(scale_exponent(warp_max(rd[x][tid & (kThreads / 32 - 1)]))), inv = 1.f / sn;
        uint8_t* codes = (x ? dv : dk).codes + now.id * d_page + now.g * d_head;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
          const int row = row0 + p * kRowsAtOnce;
          if (row >= now.rows) continue;
          // A row of zeros does not raise the page's scale: old over new may pass the largest float, and
          // zeros have to stay zeros (a code of another value needs 2^18 at most: the page holds it).
          const float up = s[x][p] * inv, ratio = up > 0x1p127f ? 0x1p127f : up;
          *reinterpret_cast<uint4*>(codes + row * kD + col) = rescale16(st.codes[x][p][tid], ratio);
        }
        if (tid == 0) (x ? dv : dk).scale[static_cast<int64_t>(now.id) * hkv + now.g] = sn;
      }
    }
    now = next;
    next = after;
    after = later;
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

EvictLayout evict_layout(const crisp_kv_cache& src, int keep) {
  const size_t rows = static_cast<size_t>(src.batch) * src.hkv;
  const size_t chunks = src.max_pages * kB > kChunk ? (src.max_pages * kB + kChunk - 1) / kChunk : 0;
  EvictLayout L{};
  size_t o = align_up(sizeof(DevStatus));
  L.list_stride = align_up(static_cast<size_t>(keep) * 4) / 4;
  L.list = o;  o = align_up(o + rows * L.list_stride * 4);
  L.hist = o;  o = align_up(o + rows * chunks * kFirstBins * sizeof(uint16_t));
  L.from = o;  o = align_up(o + rows * chunks * kBins * sizeof(uint16_t));
  L.total_bins = o; o = align_up(o + (chunks > 0 ? 2 * rows * kBins * sizeof(int) : 0));
  L.state = o; o = align_up(o + rows * chunks * sizeof(SelState));
  L.total = o;
  return L;
}

cudaError_t launch_kv_evict(const crisp_kv_cache& src, const crisp_kv_cache& dst, const float* weights, int keep,
                            int sink, int recent, float* new_weights, int32_t* kept, char* ws, int sms,
                            cudaStream_t st) {
  const EvictLayout L = evict_layout(src, keep);
  SelArgs a{};
  a.weights = weights;
  a.lens = src.lens;
  a.new_lens = dst.lens;
  a.table = src.table;
  a.new_weights = new_weights;
  a.kept = kept;
  a.list = reinterpret_cast<int32_t*>(ws + L.list);
  a.new_cap = static_cast<int64_t>(dst.max_pages) * kB;
  a.list_stride = static_cast<int64_t>(L.list_stride);
  a.hkv = src.hkv;
  a.cap = src.max_pages * kB;
  a.keep = keep;
  a.sink = sink;
  a.recent = recent;
  a.num_pages = src.num_pages;
  a.hist = reinterpret_cast<uint16_t*>(ws + L.hist);
  a.from = reinterpret_cast<uint16_t*>(ws + L.from);
  a.total = reinterpret_cast<int*>(ws + L.total_bins);
  a.state = reinterpret_cast<SelState*>(ws + L.state);
  a.chunks = (a.cap + kChunk - 1) / kChunk;
  a.rows = src.batch * src.hkv;
  a.status = reinterpret_cast<DevStatus*>(ws);
  cudaError_t e;
  if (a.chunks == 1) {
    e = launch_dependent(select_kernel, dim3(static_cast<unsigned>(a.rows)), kSelThreads, 0, st, a);
  } else {
    const dim3 grid(static_cast<unsigned>(a.chunks), static_cast<unsigned>(a.hkv), static_cast<unsigned>(src.batch));
    e = launch_dependent(chunk_kernel<0>, grid, kSelThreads, 0, st, a);
    if (e == cudaSuccess) e = launch_dependent(chunk_kernel<1>, grid, kSelThreads, 0, st, a);
    if (e == cudaSuccess) e = launch_dependent(chunk_kernel<2>, grid, kSelThreads, 0, st, a);
    if (e == cudaSuccess) e = launch_dependent(chunk_kept_kernel, grid, kSelThreads, 0, st, a);
  }
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(pack_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kPackSmem));
  if (e != cudaSuccess) return e;
  const int new_pages = (min(keep, a.cap) + kB - 1) / kB;
  const int items = a.rows * new_pages;
  return launch_dependent(pack_kernel, dim3(static_cast<unsigned>(min(items, 2 * sms))), kThreads, kPackSmem, st,
                          k_pool(src), v_pool(src), src.page_stride, src.head_stride, src.max_pages, k_pool(dst),
                          v_pool(dst), dst.page_stride, dst.head_stride, dst.table, dst.num_pages, dst.max_pages,
                          src.batch, src.hkv, static_cast<const int32_t*>(src.lens), keep, new_pages, items,
                          static_cast<const int32_t*>(a.list), a.list_stride, a.status);
}

}  // namespace crisp
