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
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = red[lane & (kThreads / 32 - 1)];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
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

// Four codes rounded again at `ratio` times their values.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float ratio) {
  float a0, a1, a2, a3;
  unpack_e4m3x2(static_cast<uint16_t>(c), a0, a1);
  unpack_e4m3x2(static_cast<uint16_t>(c >> 16), a2, a3);
  return static_cast<uint32_t>(pack_e4m3x2(a0 * ratio, a1 * ratio)) |
         static_cast<uint32_t>(pack_e4m3x2(a2 * ratio, a3 * ratio)) << 16;
}
__device__ __forceinline__ uint4 rescale16(uint4 c, float ratio) {
  return make_uint4(rescale4(c.x, ratio), rescale4(c.y, ratio), rescale4(c.z, ratio), rescale4(c.w, ratio));
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
  float amax = 0.f;
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
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = (&x[p][h].x)[e];
        amax = fmaxf(amax, fmaxf(finite_abs(bf16_lo(w)), finite_abs(bf16_hi(w))));
      }
  amax = block_max(amax, red);
  float s = exp2_int(scale_exponent(amax));
  if (held) s = fmaxf(s, s_old);
  const float inv = 1.f / s;  // exact for the powers of two that the library writes
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int row = row0 + p * kRowsAtOnce;
    if (row >= first && row < end) {
      uint4 c;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w0 = (&x[p][e >> 1].x)[(e & 1) * 2], w1 = (&x[p][e >> 1].x)[(e & 1) * 2 + 1];
        (&c.x)[e] = static_cast<uint32_t>(pack_e4m3x2(scaled(bf16_lo(w0), inv), scaled(bf16_hi(w0), inv))) |
                    static_cast<uint32_t>(pack_e4m3x2(scaled(bf16_lo(w1), inv), scaled(bf16_hi(w1), inv))) << 16;
      }
      *reinterpret_cast<uint4*>(codes + row * kD + col) = c;
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
constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;
constexpr int kClusterLen = 16384;  // capacities from which a cluster is used
constexpr int kCluster = 16;
constexpr int kAhead = 4;           // loads of four keys a thread has in flight

__device__ __forceinline__ uint32_t weight_key(float w, int pos, int sink, int tail) {
  if (pos < sink || pos >= tail) return 0xffffffffu;
  if (w != w) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 as 0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
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
  int w = warp_tot[lane];  // kSelThreads / 32 = 32 warps
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
__global__ void __launch_bounds__(kSelThreads, 1)
    select_kernel(const float* weights, const int32_t* lens, int32_t* new_lens, int hkv, int cap, int keep, int sink,
                  int recent, float* new_weights, int64_t new_cap, int32_t* list, int64_t list_stride,
                  DevStatus* status) {
  __shared__ int hist[2][kBins];
  __shared__ int bin_total[2][kC > 1 ? kBins / kC : 1];
  __shared__ int warp_tot[kSelThreads / 32];
  __shared__ int digit, above_digit;
  __shared__ int own[2];  // this CTA's keys above the threshold, and equal to it
  grid_dep_launch();
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
  // this CTA's part of the positions, whole groups of four
  const int quads = (n + 3) / 4;
  const int lo = static_cast<int>(static_cast<int64_t>(quads) * part / kC) * 4;
  const int hi = min(static_cast<int>(static_cast<int64_t>(quads) * (part + 1) / kC) * 4, n);
  if (n <= keep) {  // uniform over the cluster
    for (int i = lo + tid; i < hi; i += kSelThreads) {
      dst[i] = i;
      if (dst_w) dst_w[i] = w[i];
    }
    return;
  }
  const int tail = n - recent;
  auto load4 = [&](int i, float (&v)[4]) {
    // rows are 512-byte aligned and cap is a multiple of 128
    const float4 q = *reinterpret_cast<const float4*>(w + i);
    v[0] = q.x;
    v[1] = q.y;
    v[2] = q.z;
    v[3] = q.w;
  };

  uint32_t found = 0;   // the digits found, in place
  int want = keep;      // the threshold is the want-th largest of the keys that match them
  int above_own = 0;    // this CTA's keys above
  constexpr int kShift[3] = {21, 10, 0};
  constexpr uint32_t kMask[3] = {2047u, 2047u, 1023u};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    int* h = hist[pass & 1];
    h[tid] = h[tid + kSelThreads] = 0;
    __syncthreads();
    const uint32_t fixed = pass == 0 ? 0u : ~0u << kShift[pass - 1];
    for (int i0 = lo + tid * 4; i0 < hi; i0 += kSelThreads * 4 * kAhead) {
      float v[kAhead][4];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i0 + u * kSelThreads * 4 < hi) load4(i0 + u * kSelThreads * 4, v[u]);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = i0 + u * kSelThreads * 4 + e;
          if (i >= hi) continue;
          const uint32_t key = weight_key(v[u][e], i, sink, tail);
          if ((key & fixed) == found) atomicAdd(&h[(key >> kShift[pass]) & kMask[pass]], 1);
        }
    }
    if (kC > 1) cg::this_cluster().sync();
    else __syncthreads();
    // thread t takes bins (largest first) 2t and 2t + 1 of the whole sequence
    const int b0 = kBins - 1 - 2 * tid, b1 = b0 - 1;
    int c0, c1;
    if constexpr (kC > 1) {
      // CTA r adds up bins r * kOwn .. of all CTAs; everyone then reads the sums
      // from their owners (reading every CTA's whole histogram instead made
      // all CTAs queue at one after the other: 40 us a pass against 3)
      constexpr int kOwn = kBins / kC, kSplit = kSelThreads / kOwn;
      int* total = bin_total[pass & 1];
      if (tid < kOwn) total[tid] = 0;
      __syncthreads();
      int sum = 0;
#pragma unroll
      for (int u = 0; u < kC / kSplit; ++u)
        sum += cg::this_cluster().map_shared_rank(h, tid / kOwn * (kC / kSplit) + u)[part * kOwn + tid % kOwn];
      if (sum) atomicAdd(&total[tid % kOwn], sum);
      cg::this_cluster().sync();
      c0 = cg::this_cluster().map_shared_rank(total, b0 / kOwn)[b0 % kOwn];
      c1 = cg::this_cluster().map_shared_rank(total, b1 / kOwn)[b1 % kOwn];
    } else {
      c0 = h[b0];
      c1 = h[b1];
    }
    int all;
    const int incl = block_scan(c0 + c1, warp_tot, all);
    const int before = incl - c0 - c1;
    if (before < want && want <= incl) {
      const bool second = want > before + c0;
      digit = second ? b1 : b0;
      above_digit = before + (second ? c0 : 0);
    }
    __syncthreads();
    const int d = digit;
    want -= above_digit;
    found |= static_cast<uint32_t>(d) << kShift[pass];
    // this CTA's own keys above the digit
    int mine = (b0 > d ? h[b0] : 0) + (b1 > d ? h[b1] : 0);
    int own_above;
    block_scan(mine, warp_tot, own_above);
    above_own += own_above;
    if (pass == 2 && tid == 0) {
      own[0] = above_own;
      own[1] = h[d];
    }
    __syncthreads();
  }
  // Kept before this CTA's part: all keys above the threshold `found`, and the
  // first `want` equal to it.
  int gt = 0, eq = 0;
  if (kC > 1) {
    cg::this_cluster().sync();
    for (int r = 0; r < part; ++r) {
      const int* o = cg::this_cluster().map_shared_rank(own, r);
      gt += o[0];
      eq += o[1];
    }
    cg::this_cluster().sync();  // nobody's shared memory goes away while it is read
  }
  float next[4] = {0.f, 0.f, 0.f, 0.f};
  if (lo + tid * 4 < hi) load4(lo + tid * 4, next);
  for (int i0 = lo; i0 < hi; i0 += kSelThreads * 4) {
    const int i = i0 + tid * 4;
    const float v[4] = {next[0], next[1], next[2], next[3]};
    if (i + kSelThreads * 4 < hi) load4(i + kSelThreads * 4, next);
    uint32_t key[4];
    int packed = 0;  // counts of this thread: above in the high half, equal in the low
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      key[e] = i + e < hi ? weight_key(v[e], i + e, sink, tail) : 0u;
      if (i + e < hi) packed += key[e] > found ? 1 << 16 : key[e] == found ? 1 : 0;
    }
    int all;
    const int incl = block_scan(packed, warp_tot, all) - packed;  // at most 4096 of either before
    int g1 = gt + (incl >> 16), e1 = eq + (incl & 0xffff);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i + e >= hi) break;
      const bool above = key[e] > found, tie = key[e] == found;
      if (above || (tie && e1 < want)) {
        const int at = g1 + min(e1, want);
        dst[at] = i + e;
        if (dst_w) dst_w[at] = v[e];
      }
      g1 += above;
      e1 += tie;
    }
    gt += all >> 16;
    eq += all & 0xffff;
  }
}

// One new page of one head, K and V: their kept tokens' codes gathered from the
// old pages (a row is 128 contiguous bytes), the scale their values need, and
// the codes at it. K and V together, so that the two lookups before a row
// (its position, its page) are made once and eight row pieces a thread are in
// flight.
__global__ void __launch_bounds__(kThreads)
    pack_kernel(Pool sk, Pool sv, int64_t s_page, int64_t s_head, const int32_t* s_table, int s_num, int s_max,
                Pool dk, Pool dv, int64_t d_page, int64_t d_head, const int32_t* d_table, int d_num, int d_max, int hkv,
                const int32_t* lens, int keep, const int32_t* list, int64_t list_stride, DevStatus* status) {
  __shared__ float red[2][kThreads / 32];
  const int g = blockIdx.y, b = blockIdx.z, page = blockIdx.x;
  const int n = min(min(max(lens[b], 0), s_max * kB), keep);
  const int rows = min(n - page * kB, kB);
  if (rows <= 0) return;
  const int id = d_table[static_cast<int64_t>(b) * d_max + page];
  if (id < 0 || id >= d_num) {
    if (g == 0 && threadIdx.x == 0) report_error(status, CRISP_ERR_BOUNDS, 0x712);
    return;
  }
  grid_dep_wait();
  const int col = (threadIdx.x & (kRowThreads - 1)) * 16, row0 = threadIdx.x / kRowThreads;
  const int32_t* pos = list + (static_cast<int64_t>(b) * hkv + g) * list_stride + page * kB;
  const int32_t* tab = s_table + static_cast<int64_t>(b) * s_max;
  int src[kPasses], old[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int row = row0 + p * kRowsAtOnce;
    old[p] = row < rows ? pos[row] : -1;
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) src[p] = old[p] >= 0 ? tab[old[p] / kB] : -1;
  uint4 c[2][kPasses];
  float s[2][kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    c[0][p] = c[1][p] = make_uint4(0u, 0u, 0u, 0u);
    s[0][p] = s[1][p] = 0.f;
    if (old[p] < 0) continue;
    if (src[p] < 0 || src[p] >= s_num) {
      report_error(status, CRISP_ERR_BOUNDS, 0x713);
      continue;
    }
    const int64_t at = src[p] * s_page + g * s_head + (old[p] % kB) * kD + col;
    const int64_t sat = static_cast<int64_t>(src[p]) * hkv + g;
    c[0][p] = __ldcs(reinterpret_cast<const uint4*>(sk.codes + at));
    c[1][p] = __ldcs(reinterpret_cast<const uint4*>(sv.codes + at));
    s[0][p] = sk.scale[sat];
    s[1][p] = sv.scale[sat];
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    float amax = 0.f;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      // the largest magnitude: codes without their sign order as the values do, 0x7f is NaN
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t m = (&c[x][p].x)[e] & 0x7f7f7f7fu;
        top = __vmaxu4(top, m & ~__vcmpeq4(m, 0x7f7f7f7fu));
      }
      top = __vmaxu4(top, top >> 16);
      top = __vmaxu4(top, top >> 8) & 0xffu;
      float v, none;
      unpack_e4m3x2(static_cast<uint16_t>(top), v, none);
      amax = fmaxf(amax, v * s[x][p]);
    }
    amax = block_max(amax, red[x]);
    const float sn = exp2_int(scale_exponent(amax)), inv = 1.f / sn;
    uint8_t* codes = (x ? dv : dk).codes + id * d_page + g * d_head;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int row = row0 + p * kRowsAtOnce;
      if (row >= rows) continue;
      const float ratio = s[x][p] * inv;
      *reinterpret_cast<uint4*>(codes + row * kD + col) = ratio == 1.f ? c[x][p] : rescale16(c[x][p], ratio);
    }
    if (threadIdx.x == 0) (x ? dv : dk).scale[static_cast<int64_t>(id) * hkv + g] = sn;
  }
}

Pool k_pool(const crisp_kv_cache& c) { return {static_cast<uint8_t*>(c.k), c.k_scale}; }
Pool v_pool(const crisp_kv_cache& c) { return {static_cast<uint8_t*>(c.v), c.v_scale}; }

}  // namespace

cudaError_t launch_kv_append(const crisp_kv_cache& c, const crisp_tokens& k_new, const crisp_tokens& v_new, int n_new,
                             const int32_t* new_lens, DevStatus* status, cudaStream_t st) {
  const unsigned reach = static_cast<unsigned>((n_new + kB - 2) / kB + 1);  // pages n_new tokens can touch
  append_kernel<<<dim3(reach, 2 * c.hkv, c.batch), kThreads, 0, st>>>(
      k_pool(c), v_pool(c), c.page_stride, c.head_stride, c.hkv, c.num_pages, c.max_pages, c.table, c.lens, new_lens,
      n_new, k_new, v_new, status);
  return cudaGetLastError();
}

cudaError_t launch_kv_evict(const crisp_kv_cache& src, const crisp_kv_cache& dst, const float* weights, int keep,
                            int sink, int recent, float* new_weights, int32_t* list, int64_t list_stride,
                            DevStatus* status, cudaStream_t st) {
  const int cap = src.max_pages * kB;
  const bool wide = cap >= kClusterLen;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.blockDim = dim3(kSelThreads);
  cfg.gridDim = dim3(static_cast<unsigned>(src.batch * src.hkv * (wide ? kCluster : 1)));
  cudaError_t e;
  if (wide) {
    e = cudaFuncSetAttribute(select_kernel<kCluster>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kCluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, select_kernel<kCluster>, weights, static_cast<const int32_t*>(src.lens), dst.lens,
                           src.hkv, cap, keep, sink, recent, new_weights, static_cast<int64_t>(dst.max_pages) * kB,
                           list, list_stride, status);
  } else {
    e = cudaLaunchKernelEx(&cfg, select_kernel<1>, weights, static_cast<const int32_t*>(src.lens), dst.lens, src.hkv,
                           cap, keep, sink, recent, new_weights, static_cast<int64_t>(dst.max_pages) * kB, list,
                           list_stride, status);
  }
  if (e != cudaSuccess) return e;
  attr = cudaLaunchAttribute{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.gridDim = dim3(static_cast<unsigned>((min(keep, cap) + kB - 1) / kB), src.hkv, src.batch);
  return cudaLaunchKernelEx(&cfg, pack_kernel, k_pool(src), v_pool(src), src.page_stride, src.head_stride, src.table,
                            src.num_pages, src.max_pages, k_pool(dst), v_pool(dst), dst.page_stride, dst.head_stride,
                            dst.table, dst.num_pages, dst.max_pages, src.hkv, static_cast<const int32_t*>(src.lens),
                            keep, static_cast<const int32_t*>(list), list_stride, status);
}

}  // namespace crisp
