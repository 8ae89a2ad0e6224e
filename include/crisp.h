/*
 * crisp.h -- C ABI of the CRISP sparse-prefill library (GB300, sm_103a).
 *
 * CRISP ("CRISP: Cliff-awaRe Input-adaptive Sparse Prefilling with
 * Structural-Mass-Motivated Routing", arXiv 2609.01925) decides, per layer and
 * per attention head, which 128x128 blocks of the causal attention matrix to
 * compute, then computes exact softmax attention over those blocks:
 *
 *   A1 crisp_proxy_map          proxy attention map of the last query block
 *   A3 crisp_block_masses       vertical / slash block masses of that map
 *   A1+A3 crisp_proxy_masses    the same masses straight from q and k (map not stored)
 *   A2 crisp_route_cstruct      C_struct routing from the map: Vertical-Slash or Pooled-Estimation
 *      crisp_route_cstruct_masses  the same from the block masses (what the layer runs)
 *      crisp_route_jsd          FlexPrefill's divergence routing (the rule CRISP replaces)
 *   A4 crisp_select_vs          sink-aware noise-floor selection from the map (VS heads)
 *      crisp_select_vs_masses   the same from the block masses (what the layer runs)
 *   A5 crisp_pe_pool            pooled attention estimate (PE heads)
 *   A6 crisp_select_pe          PE block selection (gamma coverage or noise floor)
 *   A7 crisp_build_mask         per-head sparse block mask and attention schedule
 *   A8 crisp_sparse_prefill     causal GQA block-sparse attention over the index sets
 *      crisp_sparse_prefill_mask  the same over a block mask from crisp_build_mask
 *   A9 crisp_dense_prefill      the same kernel over every causal block
 *   crisp_prefill_layer         A1..A8 in order, intermediates in the workspace
 *   crisp_prefill_layer_host    the same from host buffers, copies overlapped with compute
 *   crisp_proxy_map_noalloc     A1 without a caller workspace (static scratch)
 *   crisp_kv_append             new K and V tokens into a paged 8-bit cache
 *   crisp_decode_attention      attention of 1..16 new tokens per sequence over that cache
 *   crisp_kv_evict              keeps a cache's sink, recent and heaviest tokens
 *   crisp_kv_reserve            a batch's pages, slots and positions from its requests' lengths
 *   crisp_kv_append_packed      crisp_kv_append for a batch's tokens in one packed array
 *   crisp_kv_gather             cached tokens back as packed bf16 rows
 *   crisp_packed_prefill        dense causal attention over packed sequences
 *   crisp_wait_selftest         failure detection: a bounded wait that must time out
 *
 * Conventions (every function):
 *  - Pointers are DEVICE pointers unless marked "host". The caller owns and
 *    allocates every buffer, including the workspace; the library allocates
 *    and frees no memory, and creates CUDA objects only in
 *    crisp_host_pipeline_create (three streams and their events).
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *    stream); calls return without synchronising, except crisp_read_status.
 *  - Argument errors are detected on the host, returned synchronously, and
 *    nothing is launched. Errors found on the device (a bounded wait that ran
 *    out) are recorded in the workspace status word; read it with
 *    crisp_read_status. No C++ exception crosses this boundary.
 *  - Fixed sizes: head_dim = 128, block = 128 tokens, batch 1 (a batch is a
 *    loop over calls; the cache and the packed calls take one). seq_len = n
 *    <= 2^20, any n: blocks are aligned at token 0, nb = ceil(n/128), and when
 *    128 does not divide n the last block is short (n - 128*(nb-1) tokens).
 *    The method's steps (A1..A7) need
 *    n >= 256 (the sink block and at least one more); attention, the whole
 *    layer and the workspace sizes take any n >= 0, and n = 0 (an empty
 *    input) launches nothing and returns CRISP_OK.
 *  - bf16 tensors are [heads][tokens][128] with element strides per head and
 *    per token (the 128 features contiguous). For the TMA copies every
 *    pointer must be 16-byte aligned and every stride a multiple of 8
 *    elements.
 *  - Bitsets: bit c of a row is (word[c >> 5] >> (c & 31)) & 1; a row of nb
 *    bits takes W = ceil(nb / 32) uint32 words.
 *  - Rational parameters (tau, alpha, gamma) are compared exactly in integer
 *    arithmetic; masses are integer sums of Q32 quanta, q(p) = round-half-
 *    even(p * 2^32), so index sets do not depend on summation order.
 */
#ifndef CRISP_H_
#define CRISP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define CRISP_API __attribute__((visibility("default")))
#else
#define CRISP_API
#endif

typedef struct CUstream_st* crisp_stream_t; /* same type as cudaStream_t */

typedef enum crisp_status {
  CRISP_OK = 0,
  CRISP_ERR_INVALID_ARG = 1, /* null pointer or parameter out of range */
  CRISP_ERR_SHAPE = 2,       /* unsupported shape (see limits above) */
  CRISP_ERR_ALIGN = 3,       /* pointer or stride not 16-byte aligned */
  CRISP_ERR_WORKSPACE = 4,   /* workspace null or smaller than required */
  CRISP_ERR_CUDA = 5,        /* a CUDA runtime call failed (launch, copy) */
  CRISP_ERR_TIMEOUT = 6,     /* device: a bounded wait inside a kernel ran out */
  CRISP_ERR_DEVICE = 7,      /* the current device is not sm_103 */
  CRISP_ERR_BOUNDS = 8,      /* device: an index fell outside its buffer; the access was skipped. From
                                the cache calls and the packed attention, which read page ids and
                                lengths on the device, in every build; from the others in the
                                bounds-checking build only */
  CRISP_ERR_PAGES = 9        /* device: crisp_kv_reserve needs more pages than are free; it took none */
} crisp_status;

typedef enum crisp_pe_mode {
  CRISP_PE_GAMMA = 0, /* cumulative coverage gamma (the paper's PE rule) */
  CRISP_PE_NOISE = 1  /* the noise-floor rule applied to each pooled row */
} crisp_pe_mode;

/* Head routing: CRISP's structural mass (default) or the Jensen-Shannon
 * divergence rule of FlexPrefill that CRISP replaces (a comparator). */
typedef enum crisp_route_mode {
  CRISP_ROUTE_CSTRUCT = 0,
  CRISP_ROUTE_JSD = 1
} crisp_route_mode;

/* Vertical-Slash block selection: CRISP's sink-aware noise floor (default)
 * or FlexPrefill's cumulative coverage (a comparator). */
typedef enum crisp_vs_mode {
  CRISP_VS_NOISE = 0,
  CRISP_VS_GAMMA = 1
} crisp_vs_mode;

/* Problem shape. Strides are in elements. scale = 0 selects 1/sqrt(128). */
typedef struct crisp_shape {
  int32_t hq;       /* query heads */
  int32_t hkv;      /* key/value heads; hq % hkv == 0 (GQA group G = hq/hkv) */
  int32_t head_dim; /* must be 128 */
  int32_t seq_len;  /* n */
  int32_t block;    /* must be 128 */
  int64_t q_head_stride, q_tok_stride;
  int64_t kv_head_stride, kv_tok_stride; /* shared by K and V */
  int64_t o_head_stride, o_tok_stride;
  float scale;
} crisp_shape;

/* Method parameters; crisp_params_default gives the paper's universal
 * configuration: tau_proxy = 1/5, alpha = 1, gamma = 19/20 (PE only),
 * k_min = 8 blocks (1024 tokens) per direction, pe_mode = CRISP_PE_GAMMA,
 * route_mode = CRISP_ROUTE_CSTRUCT, vs_mode = CRISP_VS_NOISE (the comparator
 * fields default to FlexPrefill's settings as we read them: vs_gamma =
 * 95/100, jsd_tau = 0.1), dense_below = 0 (no length gate; the measured
 * sparse/dense crossover on GB300 lies between 4096 and 8192 tokens, so
 * 8192 is the recommended gate), sink_tokens = recency_tokens = 128 (the
 * paper's two slices: the sink is the first 128 key tokens, the recency
 * window the last 128).
 * crisp_route_cstruct (from the map) takes any slice widths; every call that
 * routes from block masses (crisp_route_cstruct_masses, crisp_prefill_layer,
 * crisp_prefill_layer_host) needs both at 128, one block, and returns
 * CRISP_ERR_INVALID_ARG otherwise. */
typedef struct crisp_params {
  uint32_t tau_num, tau_den;     /* 0 <= tau <= 1, tau_den > 0 */
  uint32_t alpha_num, alpha_den; /* alpha_num, alpha_den <= 65535, alpha_den > 0 */
  uint32_t gamma_num, gamma_den; /* 0 <= gamma <= 1, gamma_den > 0 */
  int32_t kmin_blocks;           /* 0 <= kmin_blocks <= 8192 */
  int32_t pe_mode;               /* crisp_pe_mode */
  int32_t route_mode;            /* crisp_route_mode */
  int32_t vs_mode;               /* crisp_vs_mode */
  uint32_t vs_gamma_num, vs_gamma_den; /* coverage of CRISP_VS_GAMMA, 0 <= gamma <= 1 */
  float jsd_tau;                 /* CRISP_ROUTE_JSD: VS iff sqrt(JSD) >= jsd_tau; 0 <= jsd_tau <= 1 */
  int32_t dense_below;           /* crisp_prefill_layer*: n < dense_below runs dense attention only */
  int32_t sink_tokens;           /* C_struct sink slice: key columns [0, sink_tokens), 0 <= . <= 2^20 */
  int32_t recency_tokens;        /* C_struct recency slice: key columns [n - recency_tokens, n), 0 <= . <= 2^20 */
} crisp_params;

/* Fills *p (host) with the defaults above. */
CRISP_API void crisp_params_default(crisp_params* p);

/* Bytes of workspace the step functions need (status word and scratch). */
CRISP_API crisp_status crisp_workspace_size(const crisp_shape* shape, size_t* bytes /* host */);

/* Bytes of workspace crisp_prefill_layer needs (scratch + every intermediate). */
CRISP_API crisp_status crisp_layer_workspace_size(const crisp_shape* shape, size_t* bytes /* host */);

/* Clears the status word at the start of `ws` (asynchronously on `stream`).
 * Call once after allocating a workspace and after reading an error. */
CRISP_API crisp_status crisp_workspace_init(void* ws, size_t ws_bytes, crisp_stream_t stream);

/* A1. Proxy attention map of the last query block (ai.info page, "Key
 * Contributions" 2 and "Methodology": routing reads the proxy attention map
 * the method already computes). For q-head h (kv head h/G) and the rows
 * i = n-128+r, r in [0,128) (the last 128 tokens):
 *   pmap[h][r][j] = softmax_j(scale * q_i . k_j) over j <= i, and 0 for j > i.
 * q: bf16 [hq][n][128] (only the last 128 rows are read); k: bf16
 * [hkv][n][128]; pmap: fp32 [hq][128][ld], ld = 128*nb (= n when 128
 * divides n; columns n..ld-1 are written as 0), contiguous, 16-byte aligned. */
CRISP_API crisp_status crisp_proxy_map(const crisp_shape* shape, const void* q, const void* k, float* pmap, void* ws,
                             size_t ws_bytes, crisp_stream_t stream);

/* crisp_proxy_map without a caller-provided workspace. The paper has no
 * counterpart to this entry point; it exists for callers that cannot
 * allocate device memory when they run this step -- for example a serving
 * engine that hands all free device memory to its own pool at start-up, or
 * code that must not call cudaMalloc because it synchronises the device and
 * would stall work on other streams. Inputs and the output are as for
 * crisp_proxy_map; q, k and pmap are still the caller's buffers.
 *
 * Scratch: the per-chunk softmax statistics live in one 32 MiB array in the
 * library's static device memory, held on every GPU that loads the library
 * until the process exits. A shape needs 256 + 8*128*hq*(2*ceil(nb/16) + 1)
 * bytes of it, rounded up to 256-byte units (the 512k-token, 32-head layer
 * needs about 16.8 MB); larger shapes are rejected with CRISP_ERR_WORKSPACE
 * and nothing is launched. The first call on a device looks up the array's
 * device address (once per device, with that device current) and keeps it
 * for the life of the process, so make that first call before any stream
 * capture, and make no call on a device after cudaDeviceReset on it (the
 * reset releases the library's static memory and the kept address would
 * point at memory the process no longer owns). Every call shares the one
 * array: calls whose kernels overlap on the GPU (other streams, other
 * threads) race and corrupt each other's statistics; calls serialised on one
 * stream are safe. The status word in the array is cleared by every call; a
 * device wait that times out is recorded there: read it with
 * crisp_noalloc_read_status on the same stream before the next call.
 * Allocates nothing (no cudaMalloc/cudaFree, no allocating library call). */
CRISP_API crisp_status crisp_proxy_map_noalloc(const crisp_shape* shape, const void* q, const void* k, float* pmap,
                                               crisp_stream_t stream);

/* The status word of crisp_proxy_map_noalloc's static scratch on the current
 * device: synchronises `stream` and copies the word to *status (host),
 * CRISP_OK or CRISP_ERR_TIMEOUT after the last call. Allocates nothing.
 * Returns CRISP_ERR_CUDA if the stream or the copy failed. */
CRISP_API crisp_status crisp_noalloc_read_status(crisp_stream_t stream, crisp_status* status /* host */);

/* A3. Block masses of the proxy map ("mass at Vertical-Slash compatible
 * positions", ai-feeds page, "方法"). With q(p) the Q32 quantum and row r
 * standing for token i = n-128+r:
 *   vmass[h][c] = sum over rows r and key columns j of block c of q(pmap[h][r][j])
 *   smass[h][s] = sum over (r, j) with j <= i, j >= 128 and
 *                 floor((i - j)/128) == s of q(pmap[h][r][j])
 *   rmass[h]    = sum over rows r and the recency columns j in [n-128, n)
 *                 (= vmass[h][nb-1] when 128 divides n)
 * Sink columns (j < 128) are left out of the slash masses, so the sink cannot
 * raise the slash noise floor. pmap fp32 [hq][128][ld] as crisp_proxy_map
 * writes it; vmass, smass: uint64 [hq][nb]; rmass: uint64 [hq]. */
CRISP_API crisp_status crisp_block_masses(const crisp_shape* shape, const float* pmap, uint64_t* vmass, uint64_t* smass,
                                uint64_t* rmass, void* ws, size_t ws_bytes, crisp_stream_t stream);

/* A1 and A3 in one pass: the block masses of the proxy map, computed from q
 * and k without storing the map (routing and Vertical-Slash selection read
 * only these masses; ai.info page, "Key Contributions" 2; ai-feeds page,
 * "方法"). Each fp32 probability is formed exactly as crisp_proxy_map stores
 * it and quantised exactly as crisp_block_masses reads it, so vmass and
 * smass (and rmass) are bit-identical to crisp_block_masses(crisp_proxy_map(q,
 * k)). q, k as for crisp_proxy_map; vmass, smass uint64 [hq][nb], rmass
 * uint64 [hq], 8-byte aligned. Saves the 4*hq*128*n-byte map write and its
 * re-read. */
CRISP_API crisp_status crisp_proxy_masses(const crisp_shape* shape, const void* q, const void* k, uint64_t* vmass,
                                          uint64_t* smass, uint64_t* rmass, void* ws, size_t ws_bytes,
                                          crisp_stream_t stream);

/* A2. C_struct routing from the proxy map (ai.info page, "Key Contributions"
 * 2 and "Methodology in Plain English": the share of the map's mass that sits
 * in the sink slice, the first 128 key tokens, and the recency slice, the
 * last 128; tau_proxy = 0.2). With q(p) the Q32 quantum and the slice widths
 * of params (sink_tokens = S, recency_tokens = R; the paper's 128 and 128):
 *   cstruct[h] = sum over rows r and columns j in [0, S) U [n-R, n) of
 *                q(pmap[h][r][j])   (the union: a column in both counts once),
 *   total[h]   = sum over rows r and all columns j of q(pmap[h][r][j]),
 *   route[h]   = 1 (Vertical-Slash) iff tau_den * cstruct >= tau_num * total,
 *                0 (Pooled-Estimation) otherwise.
 * Reads the whole map once (HBM-bound). pmap fp32 [hq][128][ld] as
 * crisp_proxy_map writes it; cstruct, total uint64 [hq], 8-byte aligned;
 * route uint8 [hq]. */
CRISP_API crisp_status crisp_route_cstruct(const crisp_shape* shape, const crisp_params* params, const float* pmap,
                                           uint64_t* cstruct, uint64_t* total, uint8_t* route, void* ws,
                                           size_t ws_bytes, crisp_stream_t stream);

/* A2 from the block masses (what crisp_prefill_layer runs: the masses come
 * from the fused crisp_proxy_masses pass and the map is never stored). With
 * both slices 128 tokens wide the sink slice is key block 0 and the recency
 * slice the recency mass rmass (key block nb-1 when 128 divides n), disjoint
 * for n >= 256:
 *   cstruct[h] = vmass[h][0] + rmass[h],  total[h] = sum_c vmass[h][c],
 *   route[h] as for crisp_route_cstruct; bit-identical to it on the same map.
 * params->sink_tokens and recency_tokens must be 128 (else
 * CRISP_ERR_INVALID_ARG). vmass uint64 [hq][nb]; rmass, cstruct, total
 * uint64 [hq]; route uint8 [hq]. */
CRISP_API crisp_status crisp_route_cstruct_masses(const crisp_shape* shape, const crisp_params* params,
                                                  const uint64_t* vmass, const uint64_t* rmass, uint64_t* cstruct,
                                                  uint64_t* total, uint8_t* route, void* ws, size_t ws_bytes,
                                                  crisp_stream_t stream);

/* A2 comparator: FlexPrefill's routing, which CRISP replaces (ai.info page,
 * "Methodology in Plain English": a pooled attention estimate compared with
 * the per-query attention by Jensen-Shannon divergence). For head h, with
 *   a[c] = vmass[h][c] / sum_c vmass[h][c]   (the last query block's true
 *          attention pooled into key blocks, from the proxy map),
 *   e[c] = pbar[h][nb-1][c]                  (the pooled estimate of that block),
 *   D    = (KL(a || m) + KL(e || m)) / 2,  m = (a + e) / 2, natural log, in fp64,
 *   route[h] = 1 (Vertical-Slash) iff sqrt(D) >= jsd_tau, else 0.
 * pbar: fp32 [hq][nb][nb] holding row nb-1 of EVERY head (crisp_pe_pool with a
 * route array of zeros computes it); jsd: double [hq] (D), or NULL. */
CRISP_API crisp_status crisp_route_jsd(const crisp_shape* shape, const crisp_params* params, const uint64_t* vmass,
                                       const float* pbar, double* jsd, uint8_t* route, void* ws, size_t ws_bytes,
                                       crisp_stream_t stream);

/* A4. Sink-aware noise-floor selection for VS heads, from the block masses
 * (ai.info page, "Methodology in Plain English": a block is kept when its
 * mass is above alpha times the mean background mass of the blocks that are
 * not always retained; k_min is 1024 tokens, 8 blocks, in each direction).
 * Per direction: always-retained vertical {0, nb-1}, slash {0}; candidates
 * [1, nb-2], N of them, mass sum M; keep c iff m[c]*N*alpha_den >
 * alpha_num*M; then fill to min(kmin, available) by (mass desc, index asc).
 * PE heads get empty rows.
 * vs_mode = CRISP_VS_GAMMA (FlexPrefill's cumulative coverage, the rule CRISP
 * replaces): per direction, every block [0, nb-1] is a candidate; keep the
 * shortest (mass desc, index asc) prefix whose mass reaches vs_gamma of the
 * direction's total (vs_gamma_den * prefix >= vs_gamma_num * total), add the
 * always-retained blocks and fill to min(kmin, nb) the same way.
 * vmass, smass: uint64 [hq][nb] (crisp_block_masses or crisp_proxy_masses);
 * vbits, sbits: uint32 [hq][W]. */
CRISP_API crisp_status crisp_select_vs_masses(const crisp_shape* shape, const crisp_params* params,
                                              const uint64_t* vmass, const uint64_t* smass, const uint8_t* route,
                                              uint32_t* vbits, uint32_t* sbits, void* ws, size_t ws_bytes,
                                              crisp_stream_t stream);

/* A4 from the proxy map: crisp_block_masses (A3) then crisp_select_vs_masses,
 * with the masses written out. pmap fp32 [hq][128][ld] as crisp_proxy_map
 * writes it; route uint8 [hq]; vmass, smass uint64 [hq][nb] (outputs);
 * vbits, sbits uint32 [hq][W]. */
CRISP_API crisp_status crisp_select_vs(const crisp_shape* shape, const crisp_params* params, const float* pmap,
                                       const uint8_t* route, uint64_t* vmass, uint64_t* smass, uint32_t* vbits,
                                       uint32_t* sbits, void* ws, size_t ws_bytes, crisp_stream_t stream);

/* A5. Pooled attention estimate for PE heads (the Pooled-Estimation route
 * CRISP keeps from FlexPrefill; ai.info page, "Overview"): block means of q
 * and k (a short last block averaged over its own tokens),
 * pbar[h][b][c] = softmax over c <= b of scale * qbar_b . kbar_c, and 0 for
 * c > b. Rows of VS heads are not written. q, k bf16; pbar fp32
 * [hq][nb][nb], 16-byte aligned. Precision: the means are summed in fp32 and
 * held as hi + lo bf16 pairs (16 significant bits); the logits accumulate
 * hi.hi + hi.lo + lo.hi in fp32 on the tensor cores (lo.lo, 2^-16 of a
 * product, is left out). */
CRISP_API crisp_status crisp_pe_pool(const crisp_shape* shape, const void* q, const void* k, const uint8_t* route,
                                     float* pbar, void* ws, size_t ws_bytes, crisp_stream_t stream);

/* A6. PE block selection per query block b from pbar (ai.info page,
 * "Methodology in Plain English": gamma = 0.95 for the PE path only).
 * CRISP_PE_GAMMA: the shortest prefix of [0, b] ordered by (mass desc, index
 * asc) whose mass reaches gamma of the row (gamma_den*prefix >= gamma_num*
 * total), plus {0, b}. CRISP_PE_NOISE: forced {0, b}, candidates [1, b-1],
 * the A4 rule. Both fill to min(kmin, b+1). VS heads get empty rows.
 * pebits: uint32 [hq][nb][W]. */
CRISP_API crisp_status crisp_select_pe(const crisp_shape* shape, const crisp_params* params, const float* pbar,
                             const uint8_t* route, uint32_t* pebits, void* ws, size_t ws_bytes,
                             crisp_stream_t stream);

/* A7. The per-head sparse mask (ai-feeds page, "方法": the output is a
 * per-head sparse attention mask) as key-block sets per query block qb:
 *   VS head: {kb <= qb : kb in V} U {qb-s, qb-s-1 : s in S} within [0, qb]
 *            (a 128-wide diagonal band at offset block s crosses key blocks
 *            qb-s and qb-s-1);
 *   PE head: pebits row qb within [0, qb].
 * and the attention schedule: kv group by kv group (g = h / G), within a
 * group query blocks descending and the group's heads ascending (a causal
 * row's block count grows with qb, so each group's longest rows run first,
 * and the CTAs in flight gather one kv group's blocks, which stay in L2).
 * rowbits: uint32 [hq][nb][W]; counts: int32 [hq][nb] = blocks per row;
 * order: int32 [hq*nb], order[(g*nb + nb-1-qb)*G + h%G] = h*nb + qb. */
CRISP_API crisp_status crisp_build_mask(const crisp_shape* shape, const uint8_t* route, const uint32_t* vbits,
                                        const uint32_t* sbits, const uint32_t* pebits, uint32_t* rowbits,
                                        int32_t* counts, int32_t* order, void* ws, size_t ws_bytes,
                                        crisp_stream_t stream);

/* A8. Exact causal GQA softmax attention over the selected blocks (ai.info
 * page, "Why This Matters": the attention is exact softmax over the blocks
 * the method keeps), from the index sets of A2, A4 and A6: the mask and the
 * schedule of crisp_build_mask (A7) are built in `ws`, then for token i in
 * query block qb of head h,
 *   out_i = sum_{j in A(i)} softmax_j(scale * q_i . k_j) v_j,
 *   A(i) = { j <= i : block(j) in the head's set for qb (crisp_build_mask) }.
 * Rows with an empty A(i) are written as zeros; only rows i < n are written.
 * q bf16 [hq][n][128]; k, v bf16 [hkv][n][128]; route uint8 [hq]; vbits,
 * sbits uint32 [hq][W]; pebits uint32 [hq][nb][W]; out bf16 [hq][n][128]
 * (o strides). n >= 256 (the index sets need the method's steps). */
CRISP_API crisp_status crisp_sparse_prefill(const crisp_shape* shape, const void* q, const void* k, const void* v,
                                            const uint8_t* route, const uint32_t* vbits, const uint32_t* sbits,
                                            const uint32_t* pebits, void* out, void* ws, size_t ws_bytes,
                                            crisp_stream_t stream);

/* A8 over a block mask: for token i in query block qb of head h,
 *   out_i = sum_{j in A(i)} softmax_j(scale * q_i . k_j) v_j,
 *   A(i) = { j <= i : block(j) in rowbits[h][qb] }.
 * Bits above the diagonal block are ignored; rows with an empty A(i) are
 * written as zeros; only rows i < n are written; any n >= 0. rowbits uint32
 * [hq][nb][W] (crisp_build_mask, or any caller-made mask); order: the
 * schedule from crisp_build_mask, or NULL for the same kv-group-major order
 * (any permutation of the row ids gives the same result). */
CRISP_API crisp_status crisp_sparse_prefill_mask(const crisp_shape* shape, const void* q, const void* k,
                                                 const void* v, const uint32_t* rowbits, const int32_t* order,
                                                 void* out, void* ws, size_t ws_bytes, crisp_stream_t stream);

/* A9. Dense causal attention (A(i) = [0, i]): the exact dense
 * FlashAttention-style baseline the paper measures against (ai.info page,
 * "Methodology in Plain English"). */
CRISP_API crisp_status crisp_dense_prefill(const crisp_shape* shape, const void* q, const void* k, const void* v, void* out,
                                 void* ws, size_t ws_bytes, crisp_stream_t stream);

/* Device views of the intermediates crisp_prefill_layer leaves in `ws`. */
typedef struct crisp_layer_views {
  uint64_t *vmass, *smass, *rmass, *cstruct, *total;
  uint8_t* route;
  uint32_t *vbits, *sbits;
  float* pbar;
  uint32_t *pebits, *rowbits;
  int32_t *counts, *order;
} crisp_layer_views;

/* Fills *views (host) with pointers into `ws` for this shape. */
CRISP_API crisp_status crisp_layer_views_get(const crisp_shape* shape, void* ws, crisp_layer_views* views /* host */);

/* A1..A8 for one layer: block masses of the proxy map (crisp_proxy_masses;
 * the map itself is never stored), routing, VS and PE selection, mask,
 * sparse attention. ws must hold crisp_layer_workspace_size bytes. With
 * route_mode = CRISP_ROUTE_JSD the pooled map is computed for every head and
 * routing is crisp_route_jsd. If seq_len < params->dense_below, or
 * seq_len < 256 (too short for the method, and every block would be kept
 * anyway), the layer is dense attention only and the workspace
 * intermediates are not written. seq_len = 0 launches nothing. */
CRISP_API crisp_status crisp_prefill_layer(const crisp_shape* shape, const crisp_params* params, const void* q, const void* k,
                                 const void* v, void* out, void* ws, size_t ws_bytes, crisp_stream_t stream);

/* Prefill from HOST buffers: the streams and events the host-buffer path
 * uses, created on the current device (the one call of this library that
 * creates CUDA objects; destroy it with crisp_host_pipeline_destroy). */
typedef struct crisp_host_pipeline crisp_host_pipeline;
CRISP_API crisp_status crisp_host_pipeline_create(crisp_host_pipeline** pipeline /* host out */);
/* Waits for the pipeline's streams and destroys them; NULL is a no-op. */
CRISP_API crisp_status crisp_host_pipeline_destroy(crisp_host_pipeline* pipeline);

/* crisp_prefill_layer with q, k, v read from host memory and out written to
 * host memory. The layer is processed in chunks of the query heads of one
 * kv group (half of its G heads when G is even and n >= 131072, with the
 * first and last half group of the layer one head at a time; else all G;
 * every step of the method is per head), the group's K and V uploaded with
 * its first chunk: the upload of chunk c+1 and the download of chunk c-1 run
 * on two of the pipeline's streams while chunk c computes, so the copies
 * overlap the compute. Consecutive chunks compute alternately on `stream`
 * and on the pipeline's third stream, each with its own half of `ws` (when
 * ws holds two chunks' intermediates, as a layer workspace of several
 * chunks does); errors from both land in the status word of `ws`.
 * Results are bit-identical to crisp_prefill_layer.
 * q_host, k_host, v_host, out_host: host, contiguous [heads][n][128] bf16,
 * page-locked for the copies to be asynchronous. q, k, v, out: device
 * buffers of the same sizes (staging; afterwards they hold the inputs and
 * the output). shape: contiguous strides only (else CRISP_ERR_SHAPE). ws:
 * crisp_layer_workspace_size bytes. Ordered after earlier work on `stream`;
 * `stream` completes after the last download. The pipeline must belong to
 * the current device (else CRISP_ERR_DEVICE) and serves one call at a time
 * per stream order. */
CRISP_API crisp_status crisp_prefill_layer_host(crisp_host_pipeline* pipeline, const crisp_shape* shape,
                                                const crisp_params* params, const void* q_host, const void* k_host,
                                                const void* v_host, void* out_host, void* q, void* k, void* v,
                                                void* out, void* ws, size_t ws_bytes, crisp_stream_t stream);

/* ---- A paged key/value cache held in 8 bits --------------------------------
 * What a prefilled layer leaves for decoding. Page p of kv head h holds 128
 * tokens of 128 e4m3 codes; one power-of-two scale per page and head, K and V
 * apart, gives the values: value = code * scale. The scale is 2^e with the
 * smallest integer e >= -100 for which amax <= 448 * 2^e, amax the largest
 * finite magnitude: scaling by it is exact, each stored element is off by at
 * most half an e4m3 step (2^-4 of itself, or 2^-10 scales where it is
 * below 2^-6 scales), and a page's scale can grow without a second rounding
 * of codes of at least 2^-6 scales. A non-finite element is stored as NaN.
 *
 * Token j of sequence b is row j % 128 of page table[b][j / 128]. Entries of
 * the table past a sequence's last page are not read. A page id outside [0,
 * num_pages) or a length outside [0, 128 * max_pages] sets CRISP_ERR_BOUNDS in
 * the status word: such a page reads as holding no tokens and is not written,
 * such a length counts as the nearest one inside. A page may stand in several
 * sequences' tables (a shared prefix) as long as no call writes it; a page
 * written by a call (crisp_kv_append, the destination of crisp_kv_evict) must
 * stand there once, and its contents are unspecified otherwise.
 *
 * lens[b] counts the tokens held, the ones being appended or asked about
 * included: advance it, then append, then attend. Rows of a page at or past
 * lens[b] may hold anything. batch <= 1024, hkv <= 4096, max_pages <= 8192,
 * num_pages < 2^24, batch * hkv * max_pages < 2^31 (else CRISP_ERR_SHAPE). k and
 * v and their strides are 16-byte aligned, the other pointers 4-byte aligned. */
typedef struct crisp_kv_cache {
  int32_t batch;        /* sequences */
  int32_t hkv;          /* key/value heads */
  int32_t head_dim;     /* must be 128 */
  int32_t block;        /* tokens of a page; must be 128 */
  int32_t num_pages;    /* pages of the pool */
  int32_t max_pages;    /* entries of a table row */
  int64_t page_stride;  /* bytes from page to page, k and v alike */
  int64_t head_stride;  /* bytes from head to head of a page; a head's 128 x 128 codes are contiguous */
  void* k;              /* e4m3 [num_pages][hkv][128][128] */
  void* v;
  float* k_scale;       /* fp32 [num_pages][hkv], contiguous */
  float* v_scale;
  const int32_t* table; /* int32 [batch][max_pages], contiguous */
  int32_t* lens;        /* int32 [batch]; written by crisp_kv_evict on its destination only */
} crisp_kv_cache;

/* bf16 [batch][heads][tokens][128] with element strides (the 128 features
 * contiguous): the pointer 16-byte aligned, strides multiples of 8 and at least
 * 128 (that of an axis of one entry is not used). */
typedef struct crisp_tokens {
  const void* data;
  int64_t batch_stride, head_stride, tok_stride;
} crisp_tokens;

/* Workspace bytes of the three cache calls (as for the other steps, call
 * crisp_workspace_init once after allocating). with_weights: whether the
 * decode call gets weights_out. */
CRISP_API crisp_status crisp_kv_append_workspace_size(const crisp_kv_cache* cache, size_t* bytes /* host */);
CRISP_API crisp_status crisp_decode_workspace_size(const crisp_kv_cache* cache, int32_t hq, int32_t q_len,
                                                   int32_t with_weights, size_t* bytes /* host */);
CRISP_API crisp_status crisp_kv_evict_workspace_size(const crisp_kv_cache* cache, int32_t keep,
                                                     size_t* bytes /* host */);

/* Writes new tokens into the cache: with c = new_lens[b] (NULL: n_new for
 * every sequence; clamped to [0, min(n_new, lens[b])], CRISP_ERR_BOUNDS if it
 * was outside), token i < c of sequence b goes to position lens[b] - c + i.
 * The scale of a page that already held tokens below the first new position
 * only grows; when it does, those tokens' codes are rounded again at the new
 * scale. Rows at or past lens[b] are left as they were. k_new, v_new: bf16
 * [batch][hkv][n_new][128], 0 <= n_new <= 128 * max_pages. */
CRISP_API crisp_status crisp_kv_append(const crisp_kv_cache* cache, const crisp_tokens* k_new,
                                       const crisp_tokens* v_new, int32_t n_new, const int32_t* new_lens, void* ws,
                                       size_t ws_bytes, crisp_stream_t stream);

/* Exact softmax attention of the last q_len tokens of every sequence over the
 * cache (the dense step's formula, over the values the cache stands for).
 * Query token i of sequence b sees the keys j < lens[b] - (q_len - 1 - i); with
 * s_j = scale * q . k_j (scale 0: 1/sqrt(128)), kv head h / (hq / hkv):
 *   out[b][h][i] = sum_j softmax_j(s) v_j,       zeros where no key is seen,
 *   weights_out[b][g][j] = weights_in[b][g][j] + sum over the heads h of kv head
 *                g and the tokens i of softmax_j(s),     j < lens[b],
 * the second only with weights_out (weights_in NULL counts as zeros; the two
 * may be the same array; entries at or past lens[b] are left as they were).
 * No call clears an entry: where weights accumulate from call to call, the
 * caller sets those at or past lens[b] to zero before tokens are appended there.
 * q, out: bf16 [batch][hq][q_len][128], 1 <= q_len <= 16, hq % hkv == 0;
 * weights: fp32 [batch][hkv][128 * max_pages], contiguous, 16-byte aligned.
 * Precision: q is held as two e4m3 pieces, exact down to 2^-13 of the row's
 * largest element and below that off by at most 2^-21 of it. p is held as two
 * in the product with V, off by at most 2^-8 of itself or, where that is more,
 * 2^-22 of the row's largest p among the keys of the product (256 at most, in
 * two neighbouring pages): a p behind a neighbour that is 2^14 times as large
 * reaches out with fewer bits, at 2^-22 of it as zero, which shows in out only
 * where V of the large one is near zero. The sums and the weights count every p
 * in full. Products and sums are fp32. Limits: with rows = (hq / hkv) * q_len,
 * rows <= 1024, hq <= 4096, batch * hkv * max_pages * ceil(rows / 32) < 2^31 and
 * batch * hkv * (rows + max_pages) < 2^31 (else CRISP_ERR_SHAPE). The result
 * does not depend on timing: the same call gives the same bits. */
CRISP_API crisp_status crisp_decode_attention(const crisp_kv_cache* cache, int32_t hq, int32_t q_len, float scale,
                                              const crisp_tokens* q, const crisp_tokens* out,
                                              const float* weights_in, float* weights_out, void* ws, size_t ws_bytes,
                                              crisp_stream_t stream);

/* Cuts every sequence to at most `keep` tokens by accumulated attention weight
 * (crisp_decode_attention's weights). With n = src->lens[b], per sequence and kv
 * head: all tokens if n <= keep; else the first `sink`, the last `recent`, and
 * the keep - sink - recent others of largest weight (equal weights: the lowest
 * position; NaN counts as larger than any number). The kept tokens go, in their
 * order, to positions 0, 1, .. of dst: each of its pages gets the scale its
 * values need, codes rounded again where that differs. dst->lens[b] = min(n,
 * keep). dst->lens is not src->lens. dst may share the pools with src (k, v,
 * scales); its table's pages must then not stand in any src table. new_weights
 * fp32 [batch][hkv][128 * dst->max_pages] (16-byte aligned) and kept int32
 * [batch][hkv][128 * dst->max_pages] (each kept token's old position) are
 * written below the new length and left as they were from there on (so
 * new_weights starts as zeros, if decoding goes on with it); either may be
 * NULL. 1 <= keep <= 128 * dst->max_pages, sink + recent
 * <= keep. weights: as for crisp_decode_attention, not the same array as
 * new_weights. */
CRISP_API crisp_status crisp_kv_evict(const crisp_kv_cache* src, const crisp_kv_cache* dst, const float* weights,
                                      int32_t keep, int32_t sink, int32_t recent, float* new_weights, int32_t* kept,
                                      void* ws, size_t ws_bytes, crisp_stream_t stream);

/* ---- Batches of packed sequences -------------------------------------------
 * Requests of different lengths in one call, token by token with no padding:
 * sequence b of a packed tensor is its rows [cu[b], cu[b + 1]), cu an int32
 * array of batch + 1 running sums on the device. A packed tensor is a
 * crisp_tokens of one batch entry, [heads][rows][128] (its batch_stride is not
 * used), and its rows may be more than cu[batch]: those behind the last sequence
 * are neither read nor written, so that a captured graph serves any batch that
 * fits. A step of a server is: crisp_kv_reserve, once; then for every layer
 * crisp_kv_append_packed and crisp_packed_prefill (over the new keys, or over all
 * of them read back by crisp_kv_gather where the prompts go on from cached
 * tokens) or crisp_decode_attention. */

/* What crisp_kv_reserve finds out for a step; device arrays, contiguous, 4-byte
 * aligned. runs: one entry more than the pages that max_new tokens of the
 * batch can touch, R = min(max_new, max_new / 128 + 2 * batch). */
typedef struct crisp_kv_step {
  int32_t max_new;    /* new tokens there is room for, 0 .. 2^24 */
  int32_t max_all;    /* room for the slots of all tokens, 0 .. 2^24; 0: not wanted */
  int32_t* cu_new;    /* int32 [batch + 1]  where each sequence's new tokens begin */
  int32_t* cu_all;    /* int32 [batch + 1]  the same of all its tokens, old and new */
  int32_t* slots;     /* int32 [max_new]    new token i is row slots[i] % 128 of page slots[i] / 128 */
  int32_t* positions; /* int32 [max_new]    its position in its sequence */
  int32_t* runs;      /* int32 [R + 1]      the first new token of each page touched; from there on the total */
  int32_t* all_slots; /* int32 [max_all]    the slot of every token, in order */
} crisp_kv_step;

/* Hands out the cache's pages for a step. Sequence b keeps its first k =
 * min(keep[b], lens[b]) tokens (keep NULL: all; 0: the request is done or replaced;
 * fewer than lens[b]: drafted tokens are taken back) and gets new_lens[b] more
 * (NULL: none). Pages past ceil(k / 128) go back to the free pages, missing ones
 * are taken from them; table (the cache's own, entries given back become -1) and
 * cache->lens = k + new_lens[b] are updated, and *step is filled: entries of
 * slots, positions and all_slots at or past their totals are left as they were.
 *
 * free_pages int32 [num_pages] holds the *num_free (int32, device) free page ids
 * as a stack. In the order of sequences and their pages, the pages given back are
 * pushed last first, then those needed are popped first to last: a call that
 * takes back what the one before took leaves the stack as it was. A page that
 * stands in several tables must not be given back.
 *
 * Where the step cannot be, the status word says so, cu_new, cu_all and runs become
 * zeros (crisp_kv_append_packed, crisp_kv_gather over cu_all and crisp_packed_prefill,
 * which go by them, do nothing), and nothing else changes. crisp_decode_attention goes
 * by cache->lens, which stay: it would attend over the tokens from before the step, so
 * read the status word before it. The reasons:
 * CRISP_ERR_PAGES if too few pages are free; CRISP_ERR_BOUNDS for a length or
 * new_lens outside [0, 128 * max_pages], a negative keep, more than 128 * max_pages
 * tokens in a sequence, max_new or (where it is not 0) max_all exceeded, num_free outside [0,
 * num_pages], or a page to be given back that is none. A page id on the stack or
 * in the table that is none gives slots of -1. Workspace: as for crisp_kv_append.
 * keep, new_lens: int32 [batch], neither of them cache->lens. */
CRISP_API crisp_status crisp_kv_reserve(const crisp_kv_cache* cache, int32_t* table, int32_t* free_pages,
                                        int32_t* num_free, const int32_t* keep, const int32_t* new_lens,
                                        const crisp_kv_step* step, void* ws, size_t ws_bytes, crisp_stream_t stream);

/* crisp_kv_append for packed tokens: token i < cu_new[batch] of k_new and v_new
 * ([hkv][max_new][128] bf16) goes to slots[i]. Reads runs and slots of the step
 * only: a run's tokens stand in its page from its first one's slot on, and the
 * page's scale only grows where that is not the page's row 0. A run that is
 * outside [0, max_new], or does not fit its page, is CRISP_ERR_BOUNDS and not
 * written. */
CRISP_API crisp_status crisp_kv_append_packed(const crisp_kv_cache* cache, const crisp_kv_step* step,
                                              const crisp_tokens* k_new, const crisp_tokens* v_new, void* ws,
                                              size_t ws_bytes, crisp_stream_t stream);

/* Reads cached tokens back: row i of k_out and v_out ([hkv][n][128] bf16) becomes
 * code * scale of slot slots[i], exactly, for i < min(n, *count) (count: int32 on
 * the device, NULL: n; after crisp_kv_reserve, all_slots and cu_all + batch). A
 * negative slot leaves its row as it was; one outside the pool is
 * CRISP_ERR_BOUNDS and does too. 0 <= n <= 2^24. The cache's table and lens are
 * not read, and its batch may be 0. Workspace: as for crisp_kv_append. */
CRISP_API crisp_status crisp_kv_gather(const crisp_kv_cache* cache, const int32_t* slots, int32_t n,
                                       const int32_t* count, const crisp_tokens* k_out, const crisp_tokens* v_out,
                                       void* ws, size_t ws_bytes, crisp_stream_t stream);

typedef struct crisp_packed {
  int32_t batch;        /* sequences, at most 1024; an empty one costs as much of a call's start as others (5 us of
                           it with 256, 30 with 512, 131 with 1024) */
  int32_t hq;           /* query heads, at most 4096 */
  int32_t hkv;          /* key/value heads; hq % hkv == 0 */
  int32_t head_dim;     /* must be 128 */
  int32_t total_q;      /* rows of q and out, at most 2^24 */
  int32_t total_k;      /* rows of k and v, at most 2^24 */
  int32_t max_k;        /* about the most keys of a sequence (0: total_k): decides how work is split, and with it
                           the workspace; no limit */
  float scale;          /* 0: 1/sqrt(128) */
  const int32_t* cu_q;  /* int32 [batch + 1] */
  const int32_t* cu_k;  /* int32 [batch + 1]; may be cu_q */
} crisp_packed;

/* The status word, and room for the unfinished rows of tiles whose keys are split over
 * several parts: parts x total_q x hq rows of 520 bytes. The number of parts goes by
 * total_q, total_k and max_k, not by the lengths on the device. Without max_k a step
 * with room for many tokens counts as one long sequence: 64 requests of 32/8 heads with
 * room for 8192 new tokens and 400000 in all take 818 MB, and 256 bytes with a max_k of
 * 16384. */
CRISP_API crisp_status crisp_packed_workspace_size(const crisp_packed* packed, size_t* bytes /* host */);

/* Exact causal softmax attention of every sequence of a batch: with nq and nk its
 * rows in cu_q and cu_k, its query i sees its keys j <= nk - nq + i (the whole
 * prompt where nq = nk; a chunk that goes on from nk - nq earlier tokens where
 * not), and
 *   out_i = sum_j softmax_j(scale * q_i . k_j) v_j,    zeros where no key is seen,
 * kv head h / (hq / hkv). q bf16 [hq][total_q][128], k, v [hkv][total_k][128], out
 * as q, and none of the inputs (equal pointers are CRISP_ERR_INVALID_ARG; no element
 * may be shared). What a row does not see does not reach it, infinities and NaN in v
 * included. A sequence whose running sums descend, leave [0, total_q] or [0,
 * total_k], or are more than 2^20 rows apart is CRISP_ERR_BOUNDS and counts as
 * empty, and so does one that begins in cu_q before the end of an earlier one
 * whose sums do none of that: their rows are left as they were. Precision:
 * products of bf16 in fp32, p rounded to bf16 (2^-8 of itself) for the product
 * with v, sums in fp32. Scores scale * q_i . k_j that are finite stay below 2^30
 * in magnitude (beyond, fp32 no longer tells a row's scores from its largest
 * one's by an exponent). A row that sees keys, all of them with a score of -inf,
 * becomes zeros; v that is not finite may or may not reach a row through a score
 * of -inf. The result does not depend on timing. Calls that may run at the same
 * time (on two streams, in two captured graphs) take a workspace each. */
CRISP_API crisp_status crisp_packed_prefill(const crisp_packed* packed, const crisp_tokens* q, const crisp_tokens* k,
                                            const crisp_tokens* v, const crisp_tokens* out, void* ws, size_t ws_bytes,
                                            crisp_stream_t stream);

/* Synchronises `stream` and copies the workspace status word to *status
 * (host). Returns CRISP_ERR_CUDA if the stream or the copy failed. */
CRISP_API crisp_status crisp_read_status(const void* ws, crisp_stream_t stream, crisp_status* status /* host */);

/* Failure-detection self-test: launches one kernel that waits, through the
 * same bounded mbarrier wait every pipeline kernel uses, on a barrier that
 * nothing arrives at, for limit_ns (0 < limit_ns <= 10 s). The wait gives up,
 * the kernel records CRISP_ERR_TIMEOUT in the status word of ws and returns,
 * and the context stays usable (crisp_read_status then reports the timeout;
 * crisp_workspace_init clears it). */
CRISP_API crisp_status crisp_wait_selftest(void* ws, size_t ws_bytes, int64_t limit_ns, crisp_stream_t stream);

/* Static description of a status code (never NULL). */
CRISP_API const char* crisp_status_string(crisp_status status);

#ifdef __cplusplus
}
#endif

#endif /* CRISP_H_ */
