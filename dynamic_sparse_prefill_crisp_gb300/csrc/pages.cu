// The pages of a batch: handing them out from request lengths, and reading rows
// by slot.
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace crisp {
using namespace ptx;

namespace {

// ------------------------------------------------------------------- reserve
// One CTA, a thread per sequence: what each sequence keeps, gives back and
// takes, as running sums over the batch, then its pages moved and its runs of new
// tokens written. Nothing is written before all of it is known to fit. Integers
// only; the order of pages on the stack depends on the arguments alone. Latency
// bounds it: three chains of reads, the scans between them, and code that is run
// once and fetched as it is run (64 sequences, a token each: 3.8 us; 4.7 with a
// thread's 16 pages in line instead of twice 8).
//
// Up to kFewTokens slots are written by the same CTA; more, by a second launch
// of a thread for every four, which spreads over the GPU (512 requests, a third
// replaced, 570k slots: 11.2 us together; 13 with every page looked up in the sums).
constexpr int kPlanThreads = 1024;
constexpr int kSums = 5;
constexpr int kOwn = 16;    // pages of its sequence that a thread moves itself,
constexpr int kAtOnce = 8;  // so many at a time
constexpr int kFewTokens = 4096;
constexpr int kMapThreads = 256;
constexpr int kMapTokens = 4 * kMapThreads;

struct ReserveArgs {
  int32_t *table, *lens, *free_pages, *num_free;
  const int32_t *keep, *new_lens;
  int batch, num_pages, max_pages;
  crisp_kv_step step;
  int runs;        // room for runs
  int write_maps;  // slots are this launch's work
  DevStatus* status;
};

// Running sums before each sequence, and over all.
struct Sums {
  int cu_new[kMaxBatch + 1], cu_all[kMaxBatch + 1], freed[kMaxBatch + 1], taken[kMaxBatch + 1], runs[kMaxBatch + 1];
};

// The last sequence whose sum before it is at most i (sums[n] > i): the one that holds i.
__device__ __forceinline__ int holder(const int* sums, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int slot_of(int id, int pos, int num_pages) {
  return id >= 0 && id < num_pages ? id * kB + pos % kB : -1;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const __grid_constant__ ReserveArgs a) {
  __shared__ Sums sums;
  __shared__ int keeps[kMaxBatch], warp_sums[kSums][32];
  __shared__ int problem;
  const int b = threadIdx.x, warp = b >> 5, lane = b & 31;
  if (b == 0) problem = 0;
  grid_dep_launch();
  grid_dep_wait();
  const int cap = a.max_pages * kB;
  const int had_free = *a.num_free;
  int len = 0, keep = 0, fresh = 0;
  bool bad = had_free < 0 || had_free > a.num_pages;
  if (b < a.batch) {
    len = a.lens[b];
    keep = a.keep != nullptr ? a.keep[b] : len;
    fresh = a.new_lens != nullptr ? a.new_lens[b] : 0;
    bad = bad || len < 0 || len > cap || keep < 0 || fresh < 0 || fresh > cap;
    keep = min(keep, len);
    bad = bad || keep + fresh > cap;
    if (bad) len = keep = fresh = 0;
  }
  const int kept_pages = (keep + kB - 1) / kB;
  int v[kSums];
  v[0] = fresh;
  v[1] = keep + fresh;
  v[2] = (len + kB - 1) / kB - kept_pages;
  v[3] = (keep + fresh + kB - 1) / kB - kept_pages;
  v[4] = fresh > 0 ? (keep + fresh - 1) / kB - keep / kB + 1 : 0;
  int own[kSums];
#pragma unroll
  for (int s = 0; s < kSums; ++s) {
    own[s] = v[s];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v[s], o);
      if (lane >= o) v[s] += u;
    }
    if (lane == 31) warp_sums[s][warp] = v[s];
  }
  __syncthreads();
  if (bad) problem = CRISP_ERR_BOUNDS;
#pragma unroll
  for (int s = 0; s < kSums; ++s) {
    const int before = warp_sums[s][lane];
    v[s] += __reduce_add_sync(0xffffffffu, lane < warp ? before : 0);
    int* to = s == 0 ? sums.cu_new : s == 1 ? sums.cu_all : s == 2 ? sums.freed : s == 3 ? sums.taken : sums.runs;
    if (b <= a.batch && b < kMaxBatch) to[b] = v[s] - own[s];
    if (b == kMaxBatch - 1 && a.batch == kMaxBatch) to[kMaxBatch] = v[s];
  }
  if (b < a.batch) keeps[b] = keep;
  __syncthreads();
  const int n = a.batch;
  const int total_new = sums.cu_new[n], total_all = sums.cu_all[n], freed = sums.freed[n], taken = sums.taken[n],
            runs = sums.runs[n];
  const int top = had_free + freed;
  // A thread moves the first kOwn pages of its own sequence; where sequences have
  // more, those are moved by all threads, which look the sequence up in the sums.
  int32_t* row = a.table + static_cast<int64_t>(b) * a.max_pages + kept_pages;
  const int back = own[2], want = own[3], my_runs = own[4];                     // 0 past the batch
  const int back0 = v[2] - back, want0 = v[3] - want, runs0 = v[4] - my_runs;  // of the sequences before
  auto others = [&](const int* before, int total, auto&& page) {
    for (int k = b; k < total; k += kPlanThreads) {
      const int q = holder(before, n, k), i = k - before[q];
      if (i >= kOwn) page(k, q, i, a.table + static_cast<int64_t>(q) * a.max_pages + (keeps[q] + kB - 1) / kB + i);
    }
  };
  const bool fits = problem == 0 && top <= a.num_pages && total_new <= a.step.max_new &&
                    (a.step.max_all == 0 || total_all <= a.step.max_all);
  const bool many = __syncthreads_or(back > kOwn || want > kOwn || my_runs > kOwn) != 0;
  bool no_page = false;  // what is given back has to be a page
  if (fits) {
#pragma unroll 1
    for (int e0 = 0; e0 < min(back, kOwn); e0 += kAtOnce) {
      int id[kAtOnce];
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) id[e] = e0 + e < back ? row[e0 + e] : 0;
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) no_page = no_page || id[e] < 0 || id[e] >= a.num_pages;
    }
    if (many)
      others(sums.freed, freed, [&](int, int, int, const int32_t* at) { no_page = no_page || *at < 0 || *at >= a.num_pages; });
  }
  if (__syncthreads_or(!fits || no_page || taken > top)) {
    const bool bounds = __syncthreads_or(!fits || no_page) != 0;
    if (b == 0) report_error(a.status, bounds ? CRISP_ERR_BOUNDS : CRISP_ERR_PAGES, 0x901);
    for (int i = b; i <= n; i += kPlanThreads) a.step.cu_new[i] = a.step.cu_all[i] = 0;
    for (int i = b; i <= a.runs; i += kPlanThreads) a.step.runs[i] = 0;
    return;
  }
  // Pages go back in the order in which taking them again gives each its old place.
#pragma unroll 1
  for (int e0 = 0; e0 < min(back, kOwn); e0 += kAtOnce) {
    int id[kAtOnce];
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) id[e] = e0 + e < back ? row[e0 + e] : 0;
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e)
      if (e0 + e < back) {
        a.free_pages[top - 1 - back0 - e0 - e] = id[e];
        row[e0 + e] = -1;
      }
  }
  if (many)
    others(sums.freed, freed, [&](int k, int, int, int32_t* at) {
      a.free_pages[top - 1 - k] = *at;
      *at = -1;
    });
  if (b == 0) *a.num_free = top - taken;
  __syncthreads();
#pragma unroll 1
  for (int e0 = 0; e0 < min(want, kOwn); e0 += kAtOnce) {
    int id[kAtOnce];
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) id[e] = e0 + e < want ? a.free_pages[top - 1 - want0 - e0 - e] : 0;
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e)
      if (e0 + e < want) row[e0 + e] = id[e];
  }
  if (many) others(sums.taken, taken, [&](int k, int, int, int32_t* at) { *at = a.free_pages[top - 1 - k]; });
  // Page i of those that the new tokens of sequence q touch: its first one.
  auto run_at = [&](int q, int i) { return max((keeps[q] / kB + i) * kB, keeps[q]) - keeps[q] + sums.cu_new[q]; };
  for (int e = 0; e < min(my_runs, kOwn); ++e) a.step.runs[runs0 + e] = run_at(b, e);
  if (many) others(sums.runs, runs, [&](int k, int q, int i, const int32_t*) { a.step.runs[k] = run_at(q, i); });
  for (int j = runs + b; j <= a.runs; j += kPlanThreads) a.step.runs[j] = total_new;
  for (int i = b; i <= n; i += kPlanThreads) {
    a.step.cu_new[i] = sums.cu_new[i];
    a.step.cu_all[i] = sums.cu_all[i];
    if (i < n) a.lens[i] = sums.cu_all[i + 1] - sums.cu_all[i];
  }
  if (a.write_maps == 0) return;
  __syncthreads();  // the table is written
  for (int i = b; i < total_new; i += kPlanThreads) {
    const int q = holder(sums.cu_new, n, i), pos = keeps[q] + i - sums.cu_new[q];
    a.step.slots[i] = slot_of(a.table[static_cast<int64_t>(q) * a.max_pages + pos / kB], pos, a.num_pages);
    a.step.positions[i] = pos;
  }
  if (a.step.max_all > 0)
    for (int i = b; i < total_all; i += kPlanThreads) {
      const int q = holder(sums.cu_all, n, i), pos = i - sums.cu_all[q];
      a.step.all_slots[i] = slot_of(a.table[static_cast<int64_t>(q) * a.max_pages + pos / kB], pos, a.num_pages);
    }
}

// Slots (and positions) of many tokens, four a thread: the first new_blocks
// blocks the new tokens', the others all tokens'.
__global__ void __launch_bounds__(kMapThreads) maps_kernel(const __grid_constant__ ReserveArgs a, int new_blocks) {
  grid_dep_launch();
  grid_dep_wait();
  __shared__ int cu[kMaxBatch + 1];
  const bool all = static_cast<int>(blockIdx.x) >= new_blocks;
  for (int q = threadIdx.x; q <= a.batch; q += kMapThreads) cu[q] = (all ? a.step.cu_all : a.step.cu_new)[q];
  __syncthreads();
  const int total = cu[a.batch];
  const int i0 = (static_cast<int>(blockIdx.x) - (all ? new_blocks : 0)) * kMapTokens + static_cast<int>(threadIdx.x) * 4;
  if (i0 >= total) return;
  int q = holder(cu, a.batch, i0);
  int end = cu[q + 1], first = cu[q] - (all ? 0 : a.lens[q] - (end - cu[q]));  // the packed place of position 0
  int slot[4], where[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = min(i0 + e, total - 1);
    while (i >= end) {  // (sequences of no token are passed over)
      ++q;
      const int start = end;
      end = cu[q + 1];
      first = start - (all ? 0 : a.lens[q] - (end - start));
    }
    const int pos = i - first;
    where[e] = pos;
    slot[e] = slot_of(a.table[static_cast<int64_t>(q) * a.max_pages + pos / kB], pos, a.num_pages);
  }
  int32_t* to = (all ? a.step.all_slots : a.step.slots) + i0;
  const bool whole = i0 + 4 <= total;
  if (whole && (reinterpret_cast<uintptr_t>(to) & 15u) == 0)
    *reinterpret_cast<int4*>(to) = make_int4(slot[0], slot[1], slot[2], slot[3]);
  else
    for (int e = 0; e < 4 && i0 + e < total; ++e) to[e] = slot[e];
  if (all) return;
  to = a.step.positions + i0;
  if (whole && (reinterpret_cast<uintptr_t>(to) & 15u) == 0)
    *reinterpret_cast<int4*>(to) = make_int4(where[0], where[1], where[2], where[3]);
  else
    for (int e = 0; e < 4 && i0 + e < total; ++e) to[e] = where[e];
}

// -------------------------------------------------------------------- gather
// Rows of the cache by slot, as bf16: code * scale, exact (an e4m3 value has
// four significant bits and the scale is a power of two). Eight threads a row of
// a head, 16 codes each; a CTA takes 32 slots of K or V through the heads, so
// that a run of slots is read in pieces of 4 KB and written in whole rows. Bound
// by HBM (16 contexts of up to 16k tokens, 8 heads, 300 MB read and 601 written:
// 153 us, 5.9 TB/s; 174 with 16-byte stores and one head's codes in flight).
constexpr int kGatherThreads = 256;
constexpr int kGatherRows = kGatherThreads / 8;
constexpr int kGatherHeads = 4;  // heads whose codes a thread has in flight

struct GatherArgs {
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  int64_t page_stride, head_stride;
  int hkv, num_pages;
  const int32_t *slots, *count;
  int n;
  crisp_tokens k_out, v_out;
  bool k_wide, v_wide;  // every row of a head starts at a multiple of 32 bytes
  DevStatus* status;
};

__device__ __forceinline__ uint32_t scaled_pair(uint32_t codes, float s) {
  float a, b;
  unpack_e4m3x2(static_cast<uint16_t>(codes), a, b);
  return pack_bf16x2(a * s, b * s);
}

__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const __grid_constant__ GatherArgs a) {
  const bool is_v = blockIdx.x & 1;
  const int i = static_cast<int>(blockIdx.x >> 1) * kGatherRows + static_cast<int>(threadIdx.x >> 3), col = (threadIdx.x & 7) * 16;
  grid_dep_launch();
  grid_dep_wait();
  const int n = a.count != nullptr ? min(*a.count, a.n) : a.n;
  if (i >= n) return;
  const int slot = a.slots[i];
  if (slot < 0) return;  // a row to leave alone
  const int id = slot / kB;
  if (id >= a.num_pages) {
    if ((threadIdx.x & 7) == 0 && !is_v) report_error(a.status, CRISP_ERR_BOUNDS, 0x902);
    return;
  }
  const uint8_t* codes = (is_v ? a.v : a.k) + id * a.page_stride + (slot % kB) * kD + col;
  const float* scale = (is_v ? a.v_scale : a.k_scale) + static_cast<int64_t>(id) * a.hkv;
  const crisp_tokens& t = is_v ? a.v_out : a.k_out;
  auto* out = static_cast<__nv_bfloat16*>(const_cast<void*>(t.data)) + i * t.tok_stride + col;
  const bool wide = is_v ? a.v_wide : a.k_wide;
  for (int g0 = 0; g0 < a.hkv; g0 += kGatherHeads) {
    uint4 c[kGatherHeads];
    float s[kGatherHeads];
#pragma unroll
    for (int u = 0; u < kGatherHeads; ++u)
      if (g0 + u < a.hkv) {
        c[u] = __ldcs(reinterpret_cast<const uint4*>(codes + (g0 + u) * a.head_stride));
        s[u] = scale[g0 + u];
      }
#pragma unroll
    for (int u = 0; u < kGatherHeads; ++u)
      if (g0 + u < a.hkv) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[2 * e] = scaled_pair((&c[u].x)[e], s[u]);
          w[2 * e + 1] = scaled_pair((&c[u].x)[e] >> 16, s[u]);
        }
        store32(out + (g0 + u) * t.head_stride, w, wide);
      }
  }
}

}  // namespace

cudaError_t launch_kv_reserve(const crisp_kv_cache& c, int32_t* table, int32_t* free_pages, int32_t* num_free,
                              const int32_t* keep, const int32_t* new_lens, const crisp_kv_step& step,
                              DevStatus* status, cudaStream_t st) {
  ReserveArgs a{};
  a.table = table;
  a.lens = c.lens;
  a.free_pages = free_pages;
  a.num_free = num_free;
  a.keep = keep;
  a.new_lens = new_lens;
  a.batch = c.batch;
  a.num_pages = c.num_pages;
  a.max_pages = c.max_pages;
  a.step = step;
  a.runs = static_cast<int>(max_runs(c.batch, step.max_new));
  a.status = status;
  const int64_t tokens = static_cast<int64_t>(step.max_new) + step.max_all;
  a.write_maps = tokens <= kFewTokens;
  cudaError_t e = launch_dependent(reserve_kernel, dim3(1), kPlanThreads, 0, st, a);
  if (e != cudaSuccess || a.write_maps) return e;
  const int new_blocks = (step.max_new + kMapTokens - 1) / kMapTokens;
  const int all_blocks = (step.max_all + kMapTokens - 1) / kMapTokens;
  return launch_dependent(maps_kernel, dim3(static_cast<unsigned>(new_blocks + all_blocks)), kMapThreads, 0, st, a,
                          new_blocks);
}

cudaError_t launch_kv_gather(const crisp_kv_cache& c, const int32_t* slots, int n, const int32_t* count,
                             const crisp_tokens& k_out, const crisp_tokens& v_out, DevStatus* status, cudaStream_t st) {
  GatherArgs a{};
  a.k = static_cast<const uint8_t*>(c.k);
  a.v = static_cast<const uint8_t*>(c.v);
  a.k_scale = c.k_scale;
  a.v_scale = c.v_scale;
  a.page_stride = c.page_stride;
  a.head_stride = c.head_stride;
  a.hkv = c.hkv;
  a.num_pages = c.num_pages;
  a.slots = slots;
  a.count = count;
  a.n = n;
  a.k_out = k_out;
  a.v_out = v_out;
  auto wide = [&](const crisp_tokens& t) {
    return reinterpret_cast<uintptr_t>(t.data) % 32 == 0 && (c.hkv == 1 || t.head_stride % 16 == 0) &&
           (n == 1 || t.tok_stride % 16 == 0);
  };
  a.k_wide = wide(k_out);
  a.v_wide = wide(v_out);
  a.status = status;
  return launch_dependent(gather_kernel, dim3(2 * static_cast<unsigned>((n + kGatherRows - 1) / kGatherRows)),
                          kGatherThreads, 0, st, a);
}

}  // namespace crisp
