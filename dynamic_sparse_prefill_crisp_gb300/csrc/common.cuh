// Internal declarations shared by the CRISP CUDA translation units.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/crisp.h"

namespace crisp {

constexpr int kB = 128;  // block size (tokens), "block size B=128"
constexpr int kD = 128;  // head dimension
constexpr int kMaxSeq = 1 << 20;
constexpr int kMaxBlocks = kMaxSeq / kB;  // 8192
constexpr int kProxyChunk = 16;           // key blocks per proxy CTA

// Device status word at offset 0 of every workspace: first error wins.
struct DevStatus {
  uint32_t code;
  uint32_t detail;
};

__device__ __forceinline__ void report_error(DevStatus* st, uint32_t code, uint32_t detail) {
  if (atomicCAS(&st->code, 0u, code) == 0u) atomicExch(&st->detail, detail);
}

// Bounds checks of the checking build (compiled with -DCRISP_DEBUG): a
// global index or TMA coordinate outside its buffer records CRISP_ERR_BOUNDS
// with the site code in the status word (first error wins), and the caller
// skips the access; nothing traps. Each extent is derived from the shape the
// kernel was launched with, independently of the index it guards. The
// release build compiles every check to `true`.
#ifdef CRISP_DEBUG
__device__ __forceinline__ bool in_bounds(bool ok, DevStatus* st, uint32_t site) {
  if (!ok && st != nullptr) report_error(st, CRISP_ERR_BOUNDS, site);
  return ok;
}
#define CRISP_CHECK(cond, st, site) ::crisp::in_bounds((cond), (st), (site))
#else
#define CRISP_CHECK(cond, st, site) true
#endif

// Q32 quantum of a probability: round-half-even(p * 2^32); p * 2^32 is exact
// in fp32. No float->64-bit conversion instruction is used (on this GPU those
// run on the FP64 pipe): below 2^23, adding 2^23 in fp32 rounds the value to
// the nearest even integer, whose bits minus those of 2^23 are the result;
// from 2^23 up the product is already an integer, rebuilt from its exponent
// and mantissa.
constexpr float kTwo23 = 8388608.0f;
__device__ __forceinline__ uint32_t q32_small(float x) {  // x = p * 2^32 < 2^23
  return __float_as_uint(x + kTwo23) - 0x4B000000u;
}
__device__ __forceinline__ uint64_t q32_large(float x) {  // x = p * 2^32 >= 2^23
  const uint32_t b = __float_as_uint(x);
  const uint32_t sh = min((b >> 23) - 150u, 40u);
  return static_cast<uint64_t>((b & 0x7FFFFFu) | 0x800000u) << sh;
}
__device__ __forceinline__ uint64_t q32(float p) {
  const float x = p * 4294967296.0f;
  return x < kTwo23 ? static_cast<uint64_t>(q32_small(x)) : q32_large(x);
}

// Scale of a set of values held in e4m3: the smallest e >= kMinScaleExp with
// amax <= 448 * 2^e (448 = 1.75 * 2^8 is e4m3's largest value).
constexpr int kMinScaleExp = -100;
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
  return e < kMinScaleExp ? kMinScaleExp : e;
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// Blocks are aligned at token 0; when 128 does not divide n the last block
// is short: it holds tail_len(n) in [1, 128] tokens.
inline int num_blocks(int n) { return (n + kB - 1) / kB; }
inline int tail_len(int n) { return n - (num_blocks(n) - 1) * kB; }
// Row stride (floats) of the proxy map: whole 128-column tiles.
inline int64_t map_ld(int n) { return static_cast<int64_t>(num_blocks(n)) * kB; }
inline int bit_words(int nb) { return (nb + 31) / 32; }
inline int proxy_chunks(int nb) { return (nb + kProxyChunk - 1) / kProxyChunk; }

// Scratch part of every workspace (offsets in bytes, each 256-aligned).
struct ScratchLayout {
  size_t status;       // DevStatus
  size_t proxy_part;   // float2 [hq][128][chunks]  per-chunk (max, sum) in log2 units
  size_t proxy_stats;  // float2 [hq][128]          (row max, 1/row sum)
  size_t mass_lower;   // uint64 [hq][nb]  tile c's entries with slash block nb-1-c
  size_t mass_upper;   // uint64 [hq][nb]  tile c's entries with slash block nb-2-c
  size_t mass_upper2;  // uint64 [hq][nb]  tile c's entries with slash block nb-3-c (short last block only)
  size_t mass_rec;     // uint64 [hq]      recency columns [n-128, n) that lie in tile nb-2
  size_t qbar;         // bf16 [hq][nb][128] hi, then the same for lo (block means as hi + lo)
  size_t kbar;         // bf16 [hkv][nb][128] hi, then lo
  size_t srev;         // uint32 [hq][W + 2]  slash bits reversed
  size_t rmass;        // uint64 [hq]      recency masses of crisp_select_vs (from the map)
  size_t rowbits;      // uint32 [hq][nb][W]  block mask built by crisp_sparse_prefill
  size_t counts;       // int32  [hq][nb]      blocks per row
  size_t order;        // int32  [hq*nb]       attention schedule
  size_t total;
};

// Intermediates of crisp_prefill_layer, placed after the scratch.
struct LayerLayout {
  size_t vmass, smass, rmass, cstruct, total_mass, route, vbits, sbits, pbar, pebits, rowbits, counts, order;
  size_t total;
};

ScratchLayout scratch_layout(const crisp_shape& s);
LayerLayout layer_layout(const crisp_shape& s);

bool encode_bf16_rows(CUtensorMap* m, const void* ptr, int heads, int rows);

struct TmaMaps {
  CUtensorMap q, k, v, k64;  // k: 128-token boxes (proxy); k64, v: 64-token boxes (attention)
};

// The 8-bit cache.
constexpr int kMaxBatch = 1024;
constexpr int kMaxQLen = 16;
constexpr int kMaxDecodeCtas = 304;   // 152 SMs x 2
constexpr int kMaxGroupRows = 1024;   // query heads per kv head x q_len

struct KvMaps {
  CUtensorMap k, v;  // whole pages of one head: 128 tokens x 128 codes
};

// Attention over packed sequences.
constexpr int kPackedCtas = 304;      // 152 SMs x 2
constexpr int kMaxPacked = 1 << 24;   // rows of a packed tensor

inline size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// Workspace of crisp_decode_attention (the status word comes first).
struct DecodeLayout {
  size_t part;     // fp32 [2 CTAs][rows of a chunk][128]  unfinished accumulators
  size_t part_ml;  // float2 [2 CTAs][rows of a chunk]     their running maximum and sum
  size_t split;    // [CTAs] items that go on from one CTA to another
  size_t lse;      // fp32 [batch][hkv][rows]              log2 of the sums (weights only)
  size_t scores;   // fp32 [batch][hkv][rows][128 max_pages]  scores in base 2 (weights only)
  size_t total;
};
// Workspace of crisp_kv_evict (the status word comes first).
struct EvictLayout {
  size_t list;         // int32 [batch][hkv][list_stride]  where the kept tokens' codes are (page * 128 + row)
  size_t list_stride;  // entries
  size_t hist, from, total_bins, state;  // long caches: the chunks' and rows' histograms, and what the CTAs know
  size_t total;
};
EvictLayout evict_layout(const crisp_kv_cache& src, int keep);

DecodeLayout decode_layout(const crisp_kv_cache& c, int hq, int q_len, bool with_weights);
int decode_row_chunks(int rows);  // row chunks of a (sequence, kv head)

// How the work of crisp_packed_prefill is cut.
struct PackedPlan {
  int hp, chunks, tokens;  // query heads of a tile, tiles of a group's heads, queries of a tile
  int bound;               // no batch of these sizes has more (sequence, queries) tiles
  int heads_log2;          // kv heads (times chunks) that run side by side
  int splits, split_subs;  // parts of a tile, sub-blocks of a part
};
PackedPlan packed_plan(const crisp_packed& p);

// Workspace of crisp_packed_prefill (the status word comes first).
struct PackedLayout {
  size_t part;     // fp32 [splits][total_q][hq][128]    unfinished rows
  size_t part_ml;  // float2 [splits][total_q][hq]       their references and sums
  size_t total;
};
PackedLayout packed_layout(const crisp_packed& p, const PackedPlan& plan);

// Pages that max_new new tokens of a batch can touch (runs of crisp_kv_step).
inline int64_t max_runs(int batch, int max_new) {
  const int64_t pages = max_new / kB + int64_t(2) * batch;
  return pages < max_new ? pages : max_new;
}

// A launch that may be scheduled while the kernel before it in the stream still
// ends: the kernel calls ptx::grid_dep_wait before it reads or writes what
// others do.
template <class... P, class... Q>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                             const Q&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// ---- launchers (one per translation unit); return cudaSuccess or the launch error
cudaError_t launch_proxy(const crisp_shape& s, const TmaMaps& maps, float* pmap, char* ws, cudaStream_t st);
cudaError_t launch_proxy_masses(const crisp_shape& s, const TmaMaps& maps, uint64_t* vmass, uint64_t* smass,
                                uint64_t* rmass, char* ws, cudaStream_t st);
cudaError_t launch_assemble_slash(const crisp_shape& s, const uint64_t* vmass, char* ws, uint64_t* smass,
                                  uint64_t* rmass, cudaStream_t st);
cudaError_t launch_block_masses(const crisp_shape& s, const float* pmap, uint64_t* vmass, uint64_t* smass,
                                uint64_t* rmass, char* ws, cudaStream_t st);
cudaError_t launch_route(const crisp_shape& s, const crisp_params& p, const uint64_t* vmass, const uint64_t* rmass,
                         uint64_t* cstruct, uint64_t* total, uint8_t* route, DevStatus* status, cudaStream_t st);
cudaError_t launch_route_map(const crisp_shape& s, const crisp_params& p, const float* pmap, uint64_t* cstruct,
                             uint64_t* total, uint8_t* route, DevStatus* status, cudaStream_t st);
cudaError_t launch_route_jsd(const crisp_shape& s, const crisp_params& p, const uint64_t* vmass, const float* pbar,
                             double* jsd, uint8_t* route, DevStatus* status, cudaStream_t st);
cudaError_t launch_select_vs(const crisp_shape& s, const crisp_params& p, const uint64_t* vmass,
                             const uint64_t* smass, const uint8_t* route, uint32_t* vbits, uint32_t* sbits,
                             DevStatus* status, cudaStream_t st);
cudaError_t launch_pe_map(const crisp_shape& s, const void* q, const void* k, const uint8_t* route, float* pbar,
                          char* ws, cudaStream_t st);
cudaError_t launch_select_pe(const crisp_shape& s, const crisp_params& p, const float* pbar, const uint8_t* route,
                             uint32_t* pebits, DevStatus* status, cudaStream_t st);
cudaError_t launch_build_mask(const crisp_shape& s, const uint8_t* route, const uint32_t* vbits,
                              const uint32_t* sbits, const uint32_t* pebits, uint32_t* rowbits, int32_t* counts,
                              int32_t* order, char* ws, cudaStream_t st);
cudaError_t launch_attention(const crisp_shape& s, const TmaMaps& maps, const uint32_t* rowbits,
                             const int32_t* order, void* out, char* ws, bool dense, cudaStream_t st);
cudaError_t launch_decode(const crisp_kv_cache& c, const KvMaps& maps, int hq, int q_len, float scale,
                          const crisp_tokens& q, const crisp_tokens& out, const float* weights_in, float* weights_out,
                          char* ws, int sms, cudaStream_t st);
cudaError_t launch_kv_append(const crisp_kv_cache& c, const crisp_tokens& k_new, const crisp_tokens& v_new, int n_new,
                             const int32_t* new_lens, DevStatus* status, cudaStream_t st);
cudaError_t launch_kv_append_packed(const crisp_kv_cache& c, const crisp_kv_step& step, const crisp_tokens& k_new,
                                    const crisp_tokens& v_new, DevStatus* status, cudaStream_t st);
cudaError_t launch_kv_reserve(const crisp_kv_cache& c, int32_t* table, int32_t* free_pages, int32_t* num_free,
                              const int32_t* keep, const int32_t* new_lens, const crisp_kv_step& step,
                              DevStatus* status, cudaStream_t st);
cudaError_t launch_kv_gather(const crisp_kv_cache& c, const int32_t* slots, int n, const int32_t* count,
                             const crisp_tokens& k_out, const crisp_tokens& v_out, DevStatus* status, cudaStream_t st);
cudaError_t launch_packed(const crisp_packed& p, const PackedPlan& plan, const TmaMaps& maps, float scale, const crisp_tokens& v,
                          const crisp_tokens& out, char* ws, cudaStream_t st);
cudaError_t launch_kv_evict(const crisp_kv_cache& src, const crisp_kv_cache& dst, const float* weights, int keep,
                            int sink, int recent, float* new_weights, int32_t* kept, char* ws, int sms,
                            cudaStream_t st);

}  // namespace crisp
