/*
 * rvqmoe -- Mixture-of-Experts expert FFN on 3-stage residual-vector-quantised
 * (RVQ) weights, for NVIDIA GB300 (sm_103a).  C ABI.
 *
 * Method (sources are public web pages on the WASTE inference engine):
 *  - Expert weights are coded by 3-stage residual vector quantisation of
 *    8-dimensional sub-vectors with 256-entry codebooks: one uint8 code per
 *    stage per sub-vector, 3.00 bits per weight, no entropy coding
 *    ["WASTE Inference Engine: Running Kimi K3 2.78T on Consumer Hardware",
 *    section "Residual Vector Quantization (RVQ)"; GeekNews topic 32035,
 *    section "Quantization and accuracy"].
 *  - The weight matrix is never materialised: a partial-dot lookup table is
 *    built per codebook and position, T_s[j][k] = <x[8j..8j+7], C_s[k]>, and
 *    each output row is a sum over positions j of three table reads
 *    ["Running a 2.78-Trillion-Parameter Model on a Laptop: Inside WASTE's
 *    NVMe-Streaming Engine", section "Technical Insight"].
 *  - An expert is gate, up and down projection matrices stored together in
 *    one record with its codebooks and a checked header [same page, section
 *    "Technical Insight"; GeekNews topic 32035, section "Disk streaming
 *    structure"]; the router picks 16 experts per layer [GeekNews topic
 *    32035, section "Read-ahead and router prediction"].
 *  Readings where the pages are silent (sub-vectors along the input
 *  dimension, one codebook set per matrix, top-k softmax renormalised over
 *  the selected experts with ties to the lower index, SwiGLU, weighted
 *  combine plus residual) are stated at the calls below.
 *
 * Conventions for every call:
 *  - Pointers marked (dev) are device memory, (host) host memory.  The caller
 *    owns every buffer; the library allocates no device or host buffers (the
 *    tiered expert store's handle and its copy streams, created by
 *    moe_cache_create and released by moe_cache_destroy, are the exception).
 *  - Batch sizes (n tokens) are at least 1: an empty batch is an argument
 *    error (RVQ_EINVAL), so a caller with no tokens skips the call.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *    default stream), except where "synchronous" is stated.
 *  - Arguments are checked on the host before anything is launched; a bad
 *    argument returns RVQ_EINVAL (shape, null pointer, range) or RVQ_EALIGN
 *    (a pointer that is not 16-byte aligned) and launches nothing.
 *  - Conditions only the device can see (an expert index outside the bank, a
 *    corrupted record header, a non-finite router logit) set bits of the
 *    status word at the start of the caller's workspace; rvq_ws_status()
 *    reads them.  No call traps, aborts or exits.
 *  - rvq_last_error() returns a thread-local message for the last failure.
 *  - Calls on different streams with different buffers are thread-safe.
 */
#ifndef RVQMOE_H
#define RVQMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *rvq_stream_t; /* identical to cudaStream_t */

typedef enum rvq_status {
    RVQ_OK = 0,
    RVQ_EINVAL = 1,   /* invalid argument (shape, range, null pointer)          */
    RVQ_EALIGN = 2,   /* pointer not 16-byte aligned                             */
    RVQ_ENOMEM = 3,   /* caller-provided workspace or buffer too small           */
    RVQ_ECORRUPT = 4, /* bank record header failed validation                    */
    RVQ_EDEVICE = 5,  /* a kernel flagged a bad index or non-finite input        */
    RVQ_ETIMEOUT = 6, /* a bounded device-side wait gave up                      */
    RVQ_ECUDA = 7,    /* a CUDA runtime call failed (message in rvq_last_error)  */
    RVQ_ENOTIMPL = 8  /* configuration not supported by this build               */
} rvq_status;

typedef enum rvq_dtype {
    RVQ_F32 = 0,
    RVQ_BF16 = 1,
    RVQ_F16 = 2 /* the dense operators (moe_linear, moe_gated_linear, moe_norm_join) only */
} rvq_dtype;

/* Bits of the device status word (first 4 bytes of every workspace). */
#define RVQ_DEV_ERR_INDEX 0x1u    /* expert index / offsets outside range      */
#define RVQ_DEV_ERR_NONFINITE 0x2u /* router logit NaN or infinite             */
#define RVQ_DEV_ERR_CORRUPT 0x4u  /* expert record header mismatch             */
#define RVQ_DEV_ERR_TIMEOUT 0x8u  /* bounded spin-wait expired                 */

/* Bytes at the start of every workspace reserved for the status block. */
#define RVQ_WS_STATUS_BYTES 256u

const char *rvq_status_string(rvq_status s);
const char *rvq_last_error(void);
/* Library version, e.g. 0x000100 for 0.1.0. */
uint32_t rvq_version(void);

/* --------------------------------------------------------------------------
 * Packed code layout ("RVQ tile layout").  A matrix of `rows` x `cols`
 * weights has cols/8 sub-vectors ("chunks") per row and 3 codes per chunk.
 * Requirements: rows % 32 == 0, cols % 512 == 0.  Size: exactly
 * 3 * rows * cols / 8 bytes (3.00 bits per weight).
 *   tile (g, b), g < cols/256 (32-chunk group), b < rows/32 (32-row block),
 *   starts at byte ((g * rows/32) + b) * 3072.  Inside a tile, byte
 *   ((s*2 + h)*32 + l)*16 + i  (stage s < 3, half h < 2, lane l < 32, i < 16)
 *   holds the stage-s code of row 32b + l, chunk 32g + ((16h + i + l) mod 32).
 * The per-row rotation (l) makes the 32 lanes of a warp read 32 different
 * table columns at every step, so shared-memory lookups never conflict.
 *
 * Packed codebook layout: fp32 [3][128][8][2]; element (stage s, entry k,
 * dimension i) sits at ((s*128 + k/2)*8 + i)*2 + (k & 1), i.e. entries are
 * interleaved in pairs so that two table entries are built per packed
 * fp32x2 FMA.  Size RVQ_CODEBOOK_BYTES.
 * ------------------------------------------------------------------------ */
#define RVQ_CODEBOOK_BYTES 24576u

/* 3 * rows * cols / 8; 0 if rows/cols do not satisfy the layout rules. */
size_t rvq_code_bytes(int32_t rows, int32_t cols);

/* Canonical codes (dev) uint8 [rows][cols/8][3] -> packed codes (dev).
 * dst_bytes must be >= rvq_code_bytes(rows, cols).  src and dst must not
 * overlap.  EINVAL on shape, ENOMEM if dst_bytes is short. */
rvq_status rvq_pack(const uint8_t *codes_dev, int32_t rows, int32_t cols,
                    uint8_t *packed_dev, size_t dst_bytes, rvq_stream_t stream);

/* Inverse of rvq_pack (used by round-trip tests). */
rvq_status rvq_unpack(const uint8_t *packed_dev, int32_t rows, int32_t cols,
                      uint8_t *codes_dev, size_t dst_bytes, rvq_stream_t stream);

/* Canonical codebooks (dev) fp32 [3][256][8] -> packed codebooks (dev). */
rvq_status rvq_pack_codebooks(const float *cb_dev, float *cb_packed_dev, rvq_stream_t stream);

/* --------------------------------------------------------------------------
 * Partial-dot lookup table, "per codebook and position" [starlog page,
 * "Technical Insight"]: lut[t][j][s][k] = sum_{i<8} x[t][8j+i] * C_s[k][i]
 * for every token t < n, chunk j < cols/8, stage s < 3, entry k < 256, fp32.
 * codebooks: canonical fp32 [3][256][8] (dev); x: [n][cols] of xdt (dev);
 * lut: fp32 [n][cols/8][3][256] (dev).  cols % 8 == 0.  The fused GEMV and
 * FFN calls build the same table tile by tile in shared memory and never
 * write it out; this call exists to expose and test that step on its own.
 * ------------------------------------------------------------------------ */
rvq_status rvq_lut_build(const float *codebooks_dev, const void *x_dev, rvq_dtype xdt,
                         int32_t n, int32_t cols, float *lut_dev, rvq_stream_t stream);

/* --------------------------------------------------------------------------
 * One RVQ matrix times n input vectors, on the codes directly:
 * y[t][r] = sum_j sum_s T^t_s[j][code(r,j,s)] (== W x with W the residual
 * decode) [agentlenshq page, "Residual Vector Quantization (RVQ)"].
 * packed codes + packed codebooks (dev); x [n][cols] of xdt (dev); y fp32
 * [n][rows] (dev).  Workspace (dev) of at least
 * rvq_gemv_workspace_bytes(rows, cols, n) bytes, 256-byte aligned; its
 * status block must have been cleared once with rvq_ws_clear().
 * ------------------------------------------------------------------------ */
size_t rvq_gemv_workspace_bytes(int32_t rows, int32_t cols, int32_t n);
rvq_status rvq_gemv(const uint8_t *packed_codes_dev, const float *packed_cb_dev,
                    int32_t rows, int32_t cols, const void *x_dev, rvq_dtype xdt, int32_t n,
                    float *y_dev, void *ws_dev, size_t ws_bytes, rvq_stream_t stream);

/* --------------------------------------------------------------------------
 * rvq_gemv for callers that cannot allocate device memory (for example a
 * plug-in inside a framework that owns all device memory, or a loop where an
 * allocation and its implicit synchronisation are not allowed).  The source
 * pages have no counterpart to this call; it is an addition of this library.
 * Same operation, arguments, layouts and results as rvq_gemv, without the
 * workspace: the split-K scratch is a fixed RVQ_NOALLOC_SCRATCH_BYTES device
 * array inside the library, held by every GPU that loads the library until
 * the process exits.  Calls no cudaMalloc/cudaFree or allocating routine.
 *  - Argument checks as rvq_gemv (EINVAL / EALIGN), then RVQ_ENOMEM when
 *    rows x cols x n would need more scratch than the fixed maximum
 *    (rvq_gemv_workspace_bytes > max).  A rejected call launches nothing.
 *  - The first call on a device (and the first after the device's context
 *    was replaced, e.g. by cudaDeviceReset) looks up the array's device
 *    address with that device current; make that first call before any
 *    stream capture.
 *  - Every call shares the one array: calls whose work overlaps on the GPU
 *    (other streams, other threads) race and give wrong results; serialise
 *    them.  Each call clears the status block it needs at the start, so a
 *    call's device status must be read before the next call.
 * rvq_gemv_noalloc_status: synchronous; waits for `stream`, then reads the
 * device status word of the array (what rvq_ws_status reads from a
 * workspace) and returns RVQ_OK, RVQ_EDEVICE, RVQ_ECORRUPT or RVQ_ETIMEOUT,
 * storing the raw bits in *bits_out if not NULL and clearing them.  The
 * single-matrix GEMV reads no expert records, offsets or pair lists and has
 * no bounded waits, so its launches detect no device-side error and the word
 * reads 0 after them; the call is there so that a caller never has to assume
 * that (and reads any bit a later kernel of the path might set).
 * ------------------------------------------------------------------------ */
#define RVQ_NOALLOC_SCRATCH_BYTES 4194304u /* 4 MiB */
rvq_status rvq_gemv_noalloc(const uint8_t *packed_codes_dev, const float *packed_cb_dev,
                            int32_t rows, int32_t cols, const void *x_dev, rvq_dtype xdt,
                            int32_t n, float *y_dev, rvq_stream_t stream);
rvq_status rvq_gemv_noalloc_status(uint32_t *bits_out, rvq_stream_t stream);

/* --------------------------------------------------------------------------
 * Offline RVQ encoder: the pages' conversion step (GeekNews topic 32035,
 * "Quantization and accuracy", "Conversion": every expert matrix is encoded
 * once, offline, into 3 x 256 codewords of 8 dimensions).  Residual k-means,
 * one stage at a time: codebook = the residual sub-vectors at indices
 * floor(k N / 256) (N = rows * cols / 8, sub-vector i = W[i / (cols/8)]
 * [8 (i % (cols/8)) ..]), then `iters` rounds of nearest codeword (fp32
 * distance, fused multiply-adds in dimension order, ties to the lower index)
 * and mean of each codeword's members (int64 fixed point x 2^32 summed, then
 * divided by the count in double, rounded to fp32), a last assignment for the
 * stage's codes, and the residual minus the chosen codewords.  Reproducible:
 * bit-identical from run to run and to the same steps on the CPU.
 * w fp32 [rows][cols] (dev), |w| < 128, cols % 8 == 0, 256 <= N <= 2^21
 * (N = rows * cols / 8 sub-vectors; the bounds keep the fixed-point member
 * sums inside int64, and a 7168 x 2048 expert matrix is N = 1,835,008);
 * codes uint8 [rows][cols/8][3] and codebooks fp32 [3][256][8] (dev) in the
 * canonical layout rvq_pack / moe_bank_write_expert take; ws of
 * rvq_encode_workspace_bytes(rows, cols) bytes, 256-byte aligned. */
size_t rvq_encode_workspace_bytes(int32_t rows, int32_t cols);
rvq_status rvq_encode(const float *w_dev, int32_t rows, int32_t cols, int32_t iters,
                      uint8_t *codes_dev, float *codebooks_dev, void *ws_dev, size_t ws_bytes,
                      rvq_stream_t stream);

/* --------------------------------------------------------------------------
 * Expert bank: n_experts records of record_bytes each, contiguous in HBM.
 * Record = [rvq_expert_header, 128 B][packed codebooks gate, up, down]
 *          [packed codes gate f x d][up f x d][down d x f]; every part starts
 * on a 128-byte boundary, records on a 256-byte boundary.  gate, up and down
 * of one expert are adjacent, as in the pages' one-read expert record.
 * ------------------------------------------------------------------------ */
#define RVQ_BANK_MAGIC 0x31515652u /* "RVQ1" little-endian */
#define RVQ_HDR_FLAG_CRC32 0x1u    /* header crc32 holds the payload checksum  */

typedef struct rvq_expert_header {
    uint32_t magic;        /* RVQ_BANK_MAGIC                                  */
    uint32_t version;      /* 1                                               */
    int32_t layer;         /* layer id given to moe_bank_init                 */
    int32_t expert;        /* expert id == record index                       */
    int32_t d, f;          /* hidden and intermediate size                    */
    uint32_t flags;        /* RVQ_HDR_FLAG_CRC32 once sealed, else 0          */
    uint32_t crc32;        /* payload checksum once sealed (moe_bank_seal)    */
    uint64_t cb_off;       /* byte offsets from the record start             */
    uint64_t gate_off, up_off, down_off;
    uint64_t record_bytes;
    uint8_t pad[56];
} rvq_expert_header;       /* 128 bytes */

typedef struct rvq_moe_bank {
    uint8_t *base;         /* (dev) first record, 256-byte aligned            */
    uint64_t record_bytes; /* moe_bank_record_bytes(d, f)                     */
    int32_t n_experts, d, f, layer;
} rvq_moe_bank;

uint64_t moe_bank_record_bytes(int32_t d, int32_t f);

/* Fill *bank for a device buffer of `bytes` bytes (host-side only, launches
 * nothing).  d % 512 == 0, f % 512 == 0, 1 <= n_experts <= 256.  ENOMEM if
 * bytes < n_experts * record_bytes. */
rvq_status moe_bank_init(rvq_moe_bank *bank, uint8_t *base_dev, uint64_t bytes,
                         int32_t n_experts, int32_t d, int32_t f, int32_t layer);

/* Write one expert record: packs canonical codes (dev) gate/up [f][d/8][3],
 * down [d][f/8][3] and canonical codebooks (dev) fp32 [3 matrices][3][256][8]
 * (gate, up, down), and writes the header. */
rvq_status moe_bank_write_expert(const rvq_moe_bank *bank, int32_t expert,
                                 const uint8_t *gate_codes_dev, const uint8_t *up_codes_dev,
                                 const uint8_t *down_codes_dev, const float *codebooks_dev,
                                 rvq_stream_t stream);

/* Synchronous: copies every record header to the host and checks magic,
 * version, layer, expert id, shape and offset ranges.  ECORRUPT on mismatch
 * (message names the first bad record). */
rvq_status moe_bank_validate(const rvq_moe_bank *bank, rvq_stream_t stream);

/* Payload checksums: the pages' opt-in CRC check of each expert record
 * (GeekNews topic 32035, "Disk streaming structure").  CRC-32 (ISO-HDLC:
 * reflected polynomial 0xEDB88320, register preset to all ones, result
 * complemented) over each record's bytes [128, record_bytes), computed on the
 * device, one block per record.  Both calls are asynchronous on `stream`.
 *  - moe_bank_seal writes the value to every header (crc32) and sets
 *    RVQ_HDR_FLAG_CRC32.  Seal after the last moe_bank_write_expert (a write
 *    replaces the header and so clears the seal of that record).
 *  - moe_bank_verify recomputes it.  crc_dev (uint32 [n_experts], dev, or
 *    NULL) receives the computed values; a sealed record whose value differs
 *    sets RVQ_DEV_ERR_CORRUPT in the status word of ws_dev (ws_bytes >=
 *    RVQ_WS_STATUS_BYTES; read it with rvq_ws_status; the call does not clear
 *    it).  Unsealed records are only reported in crc_dev.
 * One pass reads the whole bank (4.2 GB for 256 K3-shaped experts), so the
 * check is an explicit pass, not part of the layer call. */
rvq_status moe_bank_seal(const rvq_moe_bank *bank, rvq_stream_t stream);
rvq_status moe_bank_verify(const rvq_moe_bank *bank, uint32_t *crc_dev, void *ws_dev,
                           size_t ws_bytes, rvq_stream_t stream);

/* --------------------------------------------------------------------------
 * Tiered expert store: the pages' streaming engine with host memory in place
 * of NVMe ("Running a 2.78-Trillion-Parameter Model on a Laptop", "Technical
 * Insight"; GeekNews topic 32035, "Read-ahead and router prediction").  A
 * host-resident bank holds every layer's expert records; an HBM cache of
 * record slots holds recently used ones, keyed by (layer, expert), least
 * recently used replaced first.
 *  - host_bank: pinned host memory (cudaHostAlloc or registered), records
 *    [layer][expert], moe_bank_record_bytes(d, f) each, byte-identical to a
 *    device bank written by moe_bank_write_expert (copy one over).
 *  - slots_dev: device buffer (256-byte aligned) of slots_bytes; it holds
 *    slots_bytes / record_bytes slots.
 *  - slot_map_dev: int32 [n_layers][n_experts] (dev), kept by the cache: the
 *    slot of each resident record, -1 otherwise.  The kernels address records
 *    through it and still check every header (expert id, layer), so a record
 *    that is not resident is reported (RVQ_DEV_ERR_CORRUPT), never used.
 * The cache owns host-side state; calls on one cache must not overlap.
 * ------------------------------------------------------------------------ */
typedef struct rvq_expert_cache rvq_expert_cache;
typedef struct rvq_cache_stats {
    uint64_t hits;          /* routed experts found resident                  */
    uint64_t misses;        /* routed experts copied in on demand             */
    uint64_t prefetched;    /* records copied in by router lookahead          */
    uint64_t prefetch_used; /* of those, later routed while still resident    */
    uint64_t bytes_copied;  /* host -> HBM record bytes                       */
    int32_t slots;
    int32_t pad;
} rvq_cache_stats;
rvq_status moe_cache_create(rvq_expert_cache **cache, const uint8_t *host_bank, int32_t n_layers,
                            int32_t n_experts, int32_t d, int32_t f, uint8_t *slots_dev,
                            uint64_t slots_bytes, int32_t *slot_map_dev);
rvq_status moe_cache_destroy(rvq_expert_cache *cache);
rvq_status moe_cache_stats(const rvq_expert_cache *cache, rvq_cache_stats *stats);
/* The bank view of layer `layer` (base = the slots), e.g. for
 * moe_workspace_bytes. */
rvq_status moe_cache_bank(const rvq_expert_cache *cache, int32_t layer, rvq_moe_bank *bank);
/* One MoE layer on cached records.  Synchronous on the host: after routing it
 * reads the expert counts back to decide the copies.  Router logits -> top-k
 * and grouping -> the routed experts made resident (misses copied
 * host -> HBM on the cache's own copy streams (four, one per slot residue,
 * so several copy engines run at once); `stream` waits for the slots it
 * needs) ->
 * expert FFN on the cached records (lookup tables; tensor cores for groups of
 * >= tc_min_tokens when > 0) -> combine + residual.  Other arguments as in
 * moe_layer_forward_ex, with ws_bytes >= moe_workspace_bytes of the cache's
 * bank view.  Router lookahead: with next_wr_dev non-NULL and lookahead > 0,
 * the next layer's router (next_wr_dev, next_bias_dev) runs on this layer's
 * input (next_logits_dev: fp32 [n][n_experts] scratch, dev), and each
 * token's `lookahead` highest-scoring experts of the next layer are copied in
 * while this layer's FFN runs (never replacing this layer's records; skipped
 * when no slot is free).  ENOMEM when this layer's experts do not fit. */
rvq_status moe_layer_forward_streamed(rvq_expert_cache *cache, int32_t layer,
                                      const float *wr_dev, const float *bias_dev,
                                      const void *x_dev, rvq_dtype xdt, int32_t n, int32_t k,
                                      float *logits_dev, int32_t *topk_idx_dev, float *topk_w_dev,
                                      int32_t *offsets_dev, int32_t *pairs_dev, float *out_dev,
                                      void *ws_dev, size_t ws_bytes, const void *residual_dev,
                                      rvq_dtype rdt, int32_t tc_min_tokens,
                                      const float *next_wr_dev, const float *next_bias_dev,
                                      int32_t lookahead, float *next_logits_dev,
                                      rvq_stream_t stream);

/* --------------------------------------------------------------------------
 * Router.  logits[t][e] = sum_c Wr[e][c] * x[t][c] (+ bias[e]), fp32
 * accumulate.  Wr fp32 [E][d] (dev); bias fp32 [E] (dev) or NULL; x [n][d]
 * of xdt (dev); logits fp32 [n][E] (dev).  1 <= E <= 256, d % 8 == 0.
 * ------------------------------------------------------------------------ */
rvq_status moe_router_logits(const float *wr_dev, const float *bias_dev, const void *x_dev,
                             rvq_dtype xdt, int32_t n, int32_t E, int32_t d,
                             float *logits_dev, rvq_stream_t stream);

/* Top-k selection, weights and token grouping.
 * Selection: the k largest fp32 logits of each token, equal logits ordered by
 * the lower expert index; slots are written in that order.  Weights:
 * w = exp(l - l_max) / sum over the k selected (softmax renormalised over
 * the selection).  Grouping: offsets[E+1] = exclusive prefix of per-expert
 * counts; pairs[n*k] sorted by (expert, token), entry = t*k + slot.
 * topk_idx int32 [n][k], topk_w fp32 [n][k], offsets int32 [E+1], pairs int32
 * [n*k] (all dev).  1 <= k <= min(E, 32), E <= 256, 1 <= n <= moe_route_max_tokens(E).
 * A non-finite logit sets RVQ_DEV_ERR_NONFINITE in the workspace status word
 * (ws >= RVQ_WS_STATUS_BYTES); outputs are then unspecified but in range. */
int32_t moe_route_max_tokens(int32_t E);
rvq_status moe_route(const float *logits_dev, int32_t n, int32_t E, int32_t k,
                     int32_t *topk_idx_dev, float *topk_w_dev, int32_t *offsets_dev,
                     int32_t *pairs_dev, void *ws_dev, size_t ws_bytes, rvq_stream_t stream);

/* Routing by scores with a balance bias and groups of experts (moe_route's selection by
 * logits is the pages' reading; this call is an addition for routers trained so):
 *   p_e = softmax(l)_e over all E, or sigmoid(l_e);   c_e = p_e + bias[e]
 *   the E experts are `groups` runs of equal size; a group's value is the sum of its two
 *   largest c (its c where it is one expert); the top_groups groups of largest value stay
 *   the k largest c of those groups are chosen, in descending order
 *   w_j = scale * p_j, or with renorm scale * p_j / sum_i p_i of the chosen
 * Ties go to the lower group and the lower expert.  The choice is that of 64-bit
 * arithmetic (without a bias experts are compared by their logits); weights are fp32.
 * The bias takes part in the choice alone.  Renormalised sigmoids of very negative logits
 * keep their ratios. */
typedef enum moe_score { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;
typedef struct moe_route_rule {
    moe_score score;
    const float *bias_dev;       /* fp32 [E] (dev), or NULL                      */
    int32_t groups, top_groups;  /* 1 <= top_groups <= groups <= 32, E % groups == 0 */
    int32_t renorm;
    float scale;
} moe_route_rule;

/* 0 for sizes the call refuses; for up to n tokens. */
size_t moe_route_scored_workspace_bytes(int32_t n, int32_t E);

/* topk_idx int32 [n][k], topk_w fp32 [n][k], offsets int32 [E+1], pairs int32 [n*k] as
 * moe_route writes them; logits fp32 [n][E] (all dev).  1 <= k <= min(32, experts of
 * top_groups groups), E <= 256, n <= 262144.  The outputs overlap nothing (EINVAL); ws
 * 256-byte aligned, moe_route_scored_workspace_bytes long, its status block cleared once;
 * calls that share it run one after another.  A logit or bias that is not
 * finite sets RVQ_DEV_ERR_NONFINITE and counts as 0. */
rvq_status moe_route_scored(const float *logits_dev, int32_t n, int32_t E, int32_t k,
                            const moe_route_rule *rule, int32_t *topk_idx_dev, float *topk_w_dev,
                            int32_t *offsets_dev, int32_t *pairs_dev, void *ws_dev,
                            size_t ws_bytes, rvq_stream_t stream);

/* Gradient of the logits (fp32 [n][E], every element written) from that of topk_w, for
 * the choice topk_idx (which has no gradient; indices outside 0 .. E-1 take no part):
 *   dp_j = scale dw_j, or with renorm scale (dw_j - sum_i dw_i p_i / P) / P, P = sum_i p_i
 *   sigmoid: dl_j = dp_j p_j (1 - p_j);  softmax: dl_e = p_e (dp_e - sum_j dp_j p_j)
 * A logit that is not finite counts as 0 here too (the choice reported it).
 * dlogits may take the place of logits and overlaps nothing else (EINVAL). */
rvq_status moe_route_scored_backward(const float *dtopk_w_dev, const float *logits_dev,
                                     const int32_t *topk_idx_dev, int32_t n, int32_t E, int32_t k,
                                     const moe_route_rule *rule, float *dlogits_dev,
                                     rvq_stream_t stream);

/* --------------------------------------------------------------------------
 * Expert FFN on the grouped pairs: for every pair entry p = t*k + slot with
 * expert e, y_pair[p] = Wd_e (silu(Wg_e x_t) * (Wu_e x_t)), silu(g) =
 * g / (1 + exp(-g)), all matrices evaluated on their RVQ codes through
 * shared-memory lookup tables with fp32 accumulation.  Reads offsets [E+1]
 * and pairs [n*k] from moe_route (dev); x [n][d] of xdt (dev); y_pair fp32
 * [n*k][d] (dev).  Each block checks its expert's record header on read and
 * sets RVQ_DEV_ERR_CORRUPT / RVQ_DEV_ERR_INDEX instead of computing with a bad
 * record.  ws >= moe_workspace_bytes(bank, n, k), 256-byte aligned.
 * ------------------------------------------------------------------------ */
size_t moe_workspace_bytes(const rvq_moe_bank *bank, int32_t n, int32_t k);
rvq_status moe_expert_ffn(const rvq_moe_bank *bank, const void *x_dev, rvq_dtype xdt,
                          int32_t n, int32_t k, const int32_t *offsets_dev,
                          const int32_t *pairs_dev, float *y_pair_dev, void *ws_dev,
                          size_t ws_bytes, rvq_stream_t stream);

/* A starting point for tc_min_tokens, measured on GB300 with K3-shaped
 * experts (d = 7168, f = 2048): at 64 tokens per step a threshold of 6 was
 * the fastest tried (4 and 8 within 4 %), while at 32 tokens the lookup
 * tables alone were fastest; a 2048-token prefill chunk is fastest with every
 * expert on the tensor cores (1).  The crossover depends on the shapes and
 * on the group sizes of the step. */
#define RVQMOE_PREFILL_MIN_TOKENS 6

/* As moe_expert_ffn, with per-expert dispatch to the tensor-core path.
 * Experts whose group holds at least tc_min_tokens tokens are computed by
 * the prefill path: their codes are decoded tile by tile to fp16 on chip
 * (W = C1[c1] + C2[c2] + C3[c3] from fp16 shared-memory codebooks, summed in
 * fp16, held in tensor memory as the MMA's A operand) and multiplied with the
 * tokens converted to fp16 on the tensor cores (tcgen05, fp32 accumulators in
 * TMEM): gate and up GEMMs, h = silu(g) * u rounded to fp16, down GEMM.
 * Results of those experts carry 16-bit rounding (the tests hold them to
 * 2e-2 x RMS).  A token or h value beyond the fp16 range (65504) saturates
 * and sets RVQ_DEV_ERR_NONFINITE.
 * tc_min_tokens <= 0: every expert takes the lookup-table path (identical to
 * moe_expert_ffn); 1: every expert takes the tensor-core path.  A bounded
 * device wait that expires sets RVQ_DEV_ERR_TIMEOUT. */
rvq_status moe_expert_ffn_ex(const rvq_moe_bank *bank, const void *x_dev, rvq_dtype xdt,
                             int32_t n, int32_t k, const int32_t *offsets_dev,
                             const int32_t *pairs_dev, float *y_pair_dev, void *ws_dev,
                             size_t ws_bytes, int32_t tc_min_tokens, rvq_stream_t stream);

/* Weighted combine plus residual: out[t][c] = residual[t][c] +
 * sum_slot topk_w[t][slot] * y_pair[t*k + slot][c], fp32.  residual [n][d]
 * of rdt (dev), out fp32 [n][d] (dev); out may alias residual only if rdt is
 * RVQ_F32. */
rvq_status moe_combine(const float *y_pair_dev, const float *topk_w_dev, int32_t n, int32_t k,
                       int32_t d, const void *residual_dev, rvq_dtype rdt, float *out_dev,
                       rvq_stream_t stream);

/* One whole MoE layer: router logits, routing and grouping, expert FFN and
 * combine, with the last reduction of the FFN fused into the combine.
 * Outputs as the separate calls (logits, topk_idx, topk_w, offsets, pairs,
 * out; all dev).  x is also the residual.  bias may be NULL.
 * ws >= moe_workspace_bytes(bank, n, k).  If `events` is not NULL it must
 * hold MOE_LAYER_EVENTS cudaEvent_t handles, recorded on `stream` before
 * the first kernel and after each kernel (for per-kernel timing). */
#define MOE_LAYER_EVENTS 8
rvq_status moe_layer_forward(const rvq_moe_bank *bank, const float *wr_dev, const float *bias_dev,
                             const void *x_dev, rvq_dtype xdt, int32_t n, int32_t k,
                             float *logits_dev, int32_t *topk_idx_dev, float *topk_w_dev,
                             int32_t *offsets_dev, int32_t *pairs_dev, float *out_dev,
                             void *ws_dev, size_t ws_bytes, void **events,
                             rvq_stream_t stream);

/* As moe_layer_forward, with two additions.
 *  - residual_dev (dtype rdt, [n][d], 16-byte aligned; NULL: x itself) is the
 *    stream the combine adds to: out = residual + sum_slot w * expert(x).  A
 *    layer stack passes the normalised stream as x and the raw stream here.
 *    A bf16 residual must not alias out (EINVAL).
 *  - the per-expert tensor-core dispatch of moe_expert_ffn_ex (tc_min_tokens
 *    <= 0: lookup tables only).  With dispatch the event marks are: 0 start,
 *    1 router logits, 2 routing, 3 lookup-table experts done, 4 tensor-core
 *    gate/up GEMM, 5 tensor-core down GEMM, 6 = 5, 7 combine. */
rvq_status moe_layer_forward_ex(const rvq_moe_bank *bank, const float *wr_dev,
                                const float *bias_dev, const void *x_dev, rvq_dtype xdt, int32_t n,
                                int32_t k, float *logits_dev, int32_t *topk_idx_dev,
                                float *topk_w_dev, int32_t *offsets_dev, int32_t *pairs_dev,
                                float *out_dev, void *ws_dev, size_t ws_bytes,
                                const void *residual_dev, rvq_dtype rdt, int32_t tc_min_tokens,
                                void **events, rvq_stream_t stream);

/* moe_layer_forward_ex with the experts chosen by `rule` (moe_route_scored) in the
 * place of moe_route; bias_dev is the router's own bias, added to the logits.  Sizes
 * are those of the layer calls, n <= moe_route_max_tokens(E) (4224 for 256 experts) among
 * them, though moe_route_scored by itself takes more; more are refused (EINVAL). */
rvq_status moe_layer_forward_scored(const rvq_moe_bank *bank, const float *wr_dev,
                                    const float *bias_dev, const moe_route_rule *rule,
                                    const void *x_dev, rvq_dtype xdt, int32_t n, int32_t k,
                                    float *logits_dev, int32_t *topk_idx_dev, float *topk_w_dev,
                                    int32_t *offsets_dev, int32_t *pairs_dev, float *out_dev,
                                    void *ws_dev, size_t ws_bytes, const void *residual_dev,
                                    rvq_dtype rdt, int32_t tc_min_tokens, void **events,
                                    rvq_stream_t stream);

/* One whole MoE layer with its input and output in host memory, for callers
 * whose tokens arrive from and leave to the host.  The call queues, all on
 * `stream` and asynchronous (synchronise the stream before reading out_host):
 *  - a copy of x_host (n x d of xdt) into x_dev;
 *  - the layer of moe_layer_forward_ex (x is also the residual; no event
 *    marks);
 *  - a copy of out (fp32 n x d) from out_dev back to out_host.
 * A transfer of up to 1 MiB whose host buffer the device maps (pinned memory,
 * which is mapped on systems with unified addressing) at a 16-byte aligned
 * address is made by the call's own kernels: the input by a copy kernel that
 * waits for the preceding kernel on the stream like the layer's kernels, the
 * output by the combine, which writes it to out_host beside out_dev.  The
 * step thus stays one chain of dependent launches.  Larger transfers, and any
 * other host buffer, go through cudaMemcpyAsync: pageable memory works, with
 * the driver's staging.
 * x_dev (dev, >= n x d x sizeof(xdt) bytes, 16-byte aligned) and the other
 * device buffers are the caller's, as in moe_layer_forward_ex.  Every
 * argument is checked before the first copy (EINVAL / EALIGN / ENOMEM,
 * nothing queued). */
rvq_status moe_layer_forward_host(const rvq_moe_bank *bank, const float *wr_dev,
                                  const float *bias_dev, const void *x_host, rvq_dtype xdt,
                                  int32_t n, int32_t k, void *x_dev, float *logits_dev,
                                  int32_t *topk_idx_dev, float *topk_w_dev, int32_t *offsets_dev,
                                  int32_t *pairs_dev, float *out_dev, float *out_host, void *ws_dev,
                                  size_t ws_bytes, int32_t tc_min_tokens, rvq_stream_t stream);

/* A CUDA graph of one layer call, for loops that run the same layer on the
 * same buffers step after step (decode).  moe_layer_graph_create records the
 * launches of moe_layer_forward_ex (x is also the residual; no event marks)
 * once, by stream capture on `stream`, and instantiates them; each
 * moe_layer_graph_launch then runs the whole layer as one graph launch on the
 * stream it is given, without the per-kernel host launch cost.
 *  - x_host and out_host both non-NULL: the graph also holds the copy of
 *    x_host (n x d of xdt) into x_dev before the layer and of out_dev (fp32
 *    n x d) into out_host after it, as moe_layer_forward_host; both NULL: the
 *    layer reads x_dev as it is when the graph runs.  One of them NULL: EINVAL.
 *  - The graph records pointers, not contents: every buffer must outlive the
 *    graph, and each launch reads what they hold when it runs.
 *  - Creating queues no work.  `stream` must be a stream that can be captured
 *    (not the legacy default stream): otherwise RVQ_ECUDA, nothing recorded.
 *  - Arguments are checked as in moe_layer_forward_host before the capture
 *    starts (EINVAL / EALIGN / ENOMEM; *graph_out is set to NULL on error).
 * moe_layer_graph_destroy frees the graph (NULL: no-op); it must not run
 * while a launch of it is pending on a stream that has not been synchronised.
 * The pages have no counterpart: this is how the library replays its launch
 * sequence on the GPU. */
typedef struct rvq_layer_graph rvq_layer_graph;
rvq_status moe_layer_graph_create(const rvq_moe_bank *bank, const float *wr_dev,
                                  const float *bias_dev, const void *x_host, rvq_dtype xdt,
                                  int32_t n, int32_t k, void *x_dev, float *logits_dev,
                                  int32_t *topk_idx_dev, float *topk_w_dev, int32_t *offsets_dev,
                                  int32_t *pairs_dev, float *out_dev, float *out_host, void *ws_dev,
                                  size_t ws_bytes, int32_t tc_min_tokens, rvq_stream_t stream,
                                  rvq_layer_graph **graph_out);
rvq_status moe_layer_graph_launch(const rvq_layer_graph *graph, rvq_stream_t stream);
rvq_status moe_layer_graph_destroy(rvq_layer_graph *graph);

/* A pre-norm layer of a stack in one call: xn = bf16(h / sqrt(mean(h^2) +
 * eps)) row by row (the values moe_rms_norm gives), then moe_layer_forward_ex
 * with x = xn (bf16) and residual = h: out = h + sum_slot w * expert(xn).
 * The stack's reading of the pages' per-layer input (they show no
 * normalisation; the stream grows without bound otherwise).
 *  - h_dev: dtype hdt (fp32 or bf16) [n][d], 16-byte aligned; out may alias an
 *    fp32 h (each element is read before it is written), not a bf16 one.
 *  - xn_dev: bf16 [n][d] (dev, 16-byte aligned), written; must not alias h or
 *    out.
 *  - eps > 0.  Other arguments as in moe_layer_forward_ex (no event marks).
 * For one token the norm runs inside the router launch (every router block
 * derives the same factor; block 0 writes xn), one launch less on the decode
 * critical path; larger batches launch the norm first. */
rvq_status moe_layer_forward_prenorm(const rvq_moe_bank *bank, const float *wr_dev,
                                     const float *bias_dev, const void *h_dev, rvq_dtype hdt,
                                     int32_t n, int32_t k, float eps, uint16_t *xn_dev,
                                     float *logits_dev, int32_t *topk_idx_dev, float *topk_w_dev,
                                     int32_t *offsets_dev, int32_t *pairs_dev, float *out_dev,
                                     void *ws_dev, size_t ws_bytes, int32_t tc_min_tokens,
                                     rvq_stream_t stream);

/* Row-wise RMS normalisation without a gain, the pre-norm of a layer stack:
 * out[t][c] = x[t][c] / sqrt(mean_c x[t][c]^2 + eps), sums in fp32.
 * The pages describe no normalisation: a stack of their layers (router,
 * top-k, RVQ SwiGLU experts, combine + residual) without one grows without
 * bound (the expert FFN is quadratic in its input), so the stack applies
 * this before each layer, as pre-norm transformer blocks do.
 * x: dtype xdt [n][d]; out: dtype odt [n][d]; d % 4 == 0; both 16-byte
 * aligned (EALIGN); eps >= 0; x may alias out only when both are fp32. */
rvq_status moe_rms_norm(const void *x_dev, rvq_dtype xdt, int32_t n, int32_t d, float eps,
                        void *out_dev, rvq_dtype odt, rvq_stream_t stream);

/* --------------------------------------------------------------------------
 * Dense operators beside the routed experts: the two halves of a shared
 * (always active, unquantised) expert, and the norms, gate and residual that
 * join one block to the next, each with its gradients.  The pages have no
 * counterpart; the formulas are stated at each call.  A block with a shared
 * expert runs them as
 *     moe_norm_join -> moe_gated_linear -> moe_linear -> moe_layer_forward_ex
 * with the shared expert's output as the layer's residual.
 *
 * Matrices are row-major with a row pitch `ld*` in elements: ld >= columns,
 * ld % 8 == 0, base pointers 16-byte aligned (EALIGN).  n (tokens) is
 * from 1 to 2^24 - 256; rows and cols are multiples of 8 in that range (EINVAL).
 * Matrices of one pitch in different columns of a wider one do not overlap.
 * Element types are
 * RVQ_BF16 or RVQ_F16 for the operands of a product (one type for x, w, bias
 * and, in a gradient, dout and every output); products accumulate in fp32 on
 * the tensor cores and each output is rounded once.
 *
 * `ws` (dev, 256-byte aligned) starts with the status block: rvq_ws_clear()
 * once, then any number of calls on one stream.  A bounded device wait that
 * expires sets RVQ_DEV_ERR_TIMEOUT; the outputs are then undefined.
 * ------------------------------------------------------------------------ */
/* Activations are evaluated in fp32 to a relative error of about (16 + 3 |a|)
 * 2^-23, a the argument of their exponential (-v; -v^2/2; the tanh form's
 * 2 sqrt(2/pi) (v + 0.044715 v^3)): also in the tails, down to |a| = 87, past
 * which their value is 0 (or v). */
typedef enum moe_act {
    MOE_ACT_NONE = 0,
    MOE_ACT_RELU = 1,     /* max(v, 0); slope 0 at 0                            */
    MOE_ACT_SILU = 2,     /* v / (1 + exp(-v))                                  */
    MOE_ACT_GELU = 3,     /* v/2 (1 + erf(v / sqrt 2))                          */
    MOE_ACT_GELU_TANH = 4 /* v/2 (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3)))      */
} moe_act;

/* Workspace of moe_linear (backward = 0), or of moe_linear_backward and
 * moe_linear (1), for up to n tokens.  It depends on the current device's SM count.
 * 0 for a shape the calls refuse. */
size_t moe_linear_workspace_bytes(int32_t n, int32_t rows, int32_t cols, int32_t backward);

/* out[t][r] = residual[t][r] + alpha * act(sum_c x[t][c] w[r][c] + bias[r])
 *  - x [n][cols], w [rows][cols] of dt; bias [rows] of dt or NULL.
 *  - residual [n][rows] of rdt, or NULL; out [n][rows] of odt; rdt and odt are
 *    fp32 or 16-bit (any mix).  out may alias residual if type and pitch agree
 *    (each element is read before it is written); out and pre overlap nothing
 *    else (EINVAL).
 *  - pre: fp32 [n][rows] without padding, or NULL; receives x w^T + bias, which
 *    moe_linear_backward needs for act != MOE_ACT_NONE. */
rvq_status moe_linear(const void *x_dev, int64_t ldx, const void *w_dev, int64_t ldw,
                      const void *bias_dev, rvq_dtype dt, int32_t n, int32_t rows, int32_t cols,
                      moe_act act, float alpha, const void *residual_dev, rvq_dtype rdt,
                      int64_t ldr, void *out_dev, rvq_dtype odt, int64_t ldo, float *pre_dev,
                      void *ws_dev, size_t ws_bytes, rvq_stream_t stream);

/* Gradients of moe_linear, with dp = alpha * dout * act'(pre):
 *   dx = dp w, dw = dp^T x, dbias[r] = sum_t dp[t][r]
 * dout [n][rows]; dx [n][cols], dw [rows][cols], dbias [rows], all of dt, each
 * NULL when not wanted (one at least is).  The gradient of the residual is dout
 * itself.  pre: as written by the forward call (NULL for MOE_ACT_NONE).  With
 * an activation dp is rounded to dt once as an operand of the products (fp16: a dp
 * beyond 65504 becomes infinite there, as any fp16 gradient does; scale dout).
 * The gradients overlap neither each other nor dout, nor w (with dx), nor x
 * (with dw): the products may run in one launch (EINVAL). */
rvq_status moe_linear_backward(const void *dout_dev, int64_t lddo, const void *x_dev, int64_t ldx,
                               const void *w_dev, int64_t ldw, const float *pre_dev, rvq_dtype dt,
                               int32_t n, int32_t rows, int32_t cols, moe_act act, float alpha,
                               void *dx_dev, int64_t lddx, void *dw_dev, int64_t lddw,
                               void *dbias_dev, void *ws_dev, size_t ws_bytes,
                               rvq_stream_t stream);

/* Workspace of moe_gated_linear / moe_gated_linear_backward, as above. */
size_t moe_gated_linear_workspace_bytes(int32_t n, int32_t rows, int32_t cols, int32_t backward);

/* The first half of a gated feed-forward block in one kernel (a second one adds
 * partial sums where the tokens are too few to fill the GPU with tiles):
 *   g = x wg^T + bg, u = x wu^T + bu, out = act(g) * u
 *  - x [n][cols], wg and wu [rows][cols] (one pitch ldw), bg and bu [rows] or
 *    NULL (each by itself), out [n][rows], all of dt.
 *  - pre: fp32 [2][n][rows] or NULL; receives g and u for the gradients.
 *  - out and pre overlap nothing (EINVAL). */
rvq_status moe_gated_linear(const void *x_dev, int64_t ldx, const void *wg_dev,
                            const void *wu_dev, int64_t ldw, const void *bg_dev,
                            const void *bu_dev, rvq_dtype dt, int32_t n, int32_t rows,
                            int32_t cols, moe_act act, void *out_dev, int64_t ldo, float *pre_dev,
                            void *ws_dev, size_t ws_bytes, rvq_stream_t stream);

/* Gradients of moe_gated_linear, with dg = dout * u * act'(g) and
 * du = dout * act(g) (each rounded to dt once as an operand of the products, as dp
 * of moe_linear_backward):
 *   dx = dg wg + du wu, dwg = dg^T x, dwu = du^T x, dbg, dbu = sums over t
 * Outputs are NULL when not wanted; dwg and dwu go together (one pitch lddw).
 * The gradients overlap neither each other, nor wg and wu (with dx), nor x (with
 * dwg and dwu) (EINVAL). */
rvq_status moe_gated_linear_backward(const void *dout_dev, int64_t lddo, const void *x_dev,
                                     int64_t ldx, const void *wg_dev, const void *wu_dev,
                                     int64_t ldw, const float *pre_dev, rvq_dtype dt, int32_t n,
                                     int32_t rows, int32_t cols, moe_act act, void *dx_dev,
                                     int64_t lddx, void *dwg_dev, void *dwu_dev, int64_t lddw,
                                     void *dbg_dev, void *dbu_dev, void *ws_dev, size_t ws_bytes,
                                     rvq_stream_t stream);

/* How the gate of moe_norm_join is broadcast over [n][d]. */
typedef enum moe_gate {
    MOE_GATE_NONE = 0,    /* no gate (1)              */
    MOE_GATE_SCALAR = 1,  /* one value                */
    MOE_GATE_TOKEN = 2,   /* [n], one per token       */
    MOE_GATE_CHANNEL = 3, /* [d], one per channel     */
    MOE_GATE_FULL = 4     /* [n][d]                   */
} moe_gate;

/* Joins a block's output y to the residual stream h and norms the result for
 * the next block, in one pass (norm(v) = v / sqrt(mean_c v^2 + eps)):
 *   z      = post_norm ? norm(y) * w_post : y
 *   h_out  = alpha * h + gate * z
 *   xn     = norm(h_out) * w_pre          (of h_out before its rounding)
 *  - h, h_out: [n][d] of hdt; y: [n][d] of ydt; xn: [n][d] of xdt; gate of gdt;
 *    w_post, w_pre: [d] of wdt, NULL = 1.  Types are fp32, bf16 or fp16.  Rows
 *    are contiguous, as in moe_rms_norm; d % 8 == 0 and d <= 16384 (EINVAL).
 *  - h may be NULL (no residual), h_out or xn may be NULL (not both).
 *  - rstd: fp32 [2][n] or NULL; receives 1/rms of y (1 without a post norm) and
 *    of h_out, for the gradients.
 *  - h_out and xn may each take the place of h, y or a full gate of the same
 *    type; the outputs (rstd too) overlap nothing else (EINVAL).  Sums and
 *    statistics are fp32.  eps >= 0; a row of zeros with eps = 0 gives NaN, as
 *    the formula does. */
rvq_status moe_norm_join(const void *h_dev, rvq_dtype hdt, const void *y_dev, rvq_dtype ydt,
                         int32_t n, int32_t d, float alpha, const void *gate_dev,
                         moe_gate gate_kind, rvq_dtype gdt, int32_t post_norm,
                         const void *w_post_dev, const void *w_pre_dev, rvq_dtype wdt, float eps,
                         void *h_out_dev, void *xn_dev, rvq_dtype xdt, float *rstd_dev,
                         rvq_stream_t stream);

/* Workspace of moe_norm_join_backward (partial sums over tokens). */
size_t moe_norm_join_workspace_bytes(int32_t n, int32_t d);

/* Gradients of moe_norm_join from dh_out [n][d] of hdt and dxn [n][d] of xdt
 * (each may be NULL: no gradient arrives there, not both), with the forward's
 * inputs and rstd:
 *   e      = dh_out + r2 (dxn w_pre) - h_out r2^3 mean(dxn w_pre h_out)
 *   dh     = alpha e (hdt);  dgate = e z, summed over the gate's broadcast (gdt)
 *   dz     = gate e;  dw_post = sum_t dz y r1;  dw_pre = sum_t dxn h_out r2 (wdt)
 *   dy     = post_norm ? r1 (dz w_post) - y r1^3 mean(dz w_post y) : dz  (ydt)
 * h_out is recomputed from h, y and rstd.  Outputs are NULL when not wanted.
 * Sums over tokens run in a fixed order: results repeat bit for bit.  dh, dy and
 * dgate (per token or full) may each take the place of h, y, gate, dh_out or dxn of
 * the same type and shape, and overlap no other input; the gradients do not overlap
 * each other (EINVAL). */
rvq_status moe_norm_join_backward(const void *dh_out_dev, const void *dxn_dev, rvq_dtype xdt,
                                  const void *h_dev, rvq_dtype hdt, const void *y_dev,
                                  rvq_dtype ydt, int32_t n, int32_t d, float alpha,
                                  const void *gate_dev, moe_gate gate_kind, rvq_dtype gdt,
                                  int32_t post_norm, const void *w_post_dev,
                                  const void *w_pre_dev, rvq_dtype wdt, const float *rstd_dev,
                                  void *dh_dev, void *dy_dev, void *dgate_dev, void *dw_post_dev,
                                  void *dw_pre_dev, void *ws_dev, size_t ws_bytes,
                                  rvq_stream_t stream);

/* --------------------------------------------------------------------------
 * Microscaled operators: the dense operators above for matrices held in 8 or 4 bits
 * (the pages have no counterpart; formats as in the Open Compute Project's
 * "Microscaling Formats (MX)" specification, 1.0).  Blocks of 32 values along a row
 * share a scale 2^(byte - 127); a value is its code times that scale.  A block with
 * scale byte 255 is NaN.
 *  - codes: uint8, row-major, columns padded to a multiple of 128 (the padding holds
 *    zeros): one byte per MOE_MX_F8 value, one for two MOE_MX_F4 values, the lower
 *    column in the lower half.  moe_mx_code_bytes(fmt, rows, cols) bytes.
 *  - scales: uint8, in tiles of 128 rows x 4 blocks (128 columns), 512 bytes each;
 *    tile (r / 128, c / 128) is number (r / 128) * ceil(cols / 128) + c / 128, and in it
 *    row r, column c has byte (r % 32) * 16 + (r / 32 % 4) * 4 + c / 32 % 4.
 *    moe_mx_scale_bytes(rows, cols) bytes.  Bytes of rows behind the last are neither
 *    written nor used; those of padded columns are written (0).
 * Both start on 32 bytes (EALIGN).  Rows from 1, columns multiples of 8, up to
 * 2^24 - 256 each.  Other matrices have row pitches as in the dense operators.
 * ------------------------------------------------------------------------ */
typedef enum moe_mx {
    MOE_MX_F8 = 0, /* e4m3: 4-bit exponent, 3-bit mantissa, up to 448           */
    MOE_MX_F4 = 1  /* e2m1: 0, 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives      */
} moe_mx;

/* 0 for a shape or format that the calls refuse. */
size_t moe_mx_code_bytes(moe_mx fmt, int32_t rows, int32_t cols);
size_t moe_mx_scale_bytes(int32_t rows, int32_t cols);

/* x [rows][cols] of xdt (fp32, bf16 or fp16) -> codes and scales.  With m the largest
 * magnitude of a block, its scale is 2^(floor(log2 m) - 8) (F8) or 2^(floor(log2 m) - 2)
 * (F4), at least 2^-127 (so too where m = 0); values over their scale are rounded to
 * the nearest code, ties to even, and end at the largest one.  A block that holds a
 * NaN or an infinity gets scale 255 and codes 0.  No sums: the result is exact.
 * codes and scales overlap neither x nor each other (EINVAL). */
rvq_status moe_mx_quantize(const void *x_dev, int64_t ldx, rvq_dtype xdt, int32_t rows,
                           int32_t cols, moe_mx fmt, uint8_t *codes_dev, uint8_t *scales_dev,
                           rvq_stream_t stream);

/* The inverse: out [rows][cols] of odt = codes times scales (in fp32, rounded once). */
rvq_status moe_mx_dequantize(const uint8_t *codes_dev, const uint8_t *scales_dev, moe_mx fmt,
                             int32_t rows, int32_t cols, void *out_dev, rvq_dtype odt, int64_t ldo,
                             rvq_stream_t stream);

/* Workspaces of the products below, for up to n tokens (256-byte aligned; rvq_ws_clear()
 * once, then any number of calls on one stream; a bounded device wait that expires sets
 * RVQ_DEV_ERR_TIMEOUT, and the outputs are undefined).  0 for a shape they refuse. */
size_t moe_mx_linear_workspace_bytes(int32_t n, int32_t rows, int32_t cols);
size_t moe_mx_gated_linear_workspace_bytes(int32_t n, int32_t rows, int32_t cols);

/* out[t][r] = residual[t][r] + alpha * act(sum_c x[t][c] w[r][c] + bias[r])
 *  - x [n][cols] and w [rows][cols] microscaled, each in either format (two MOE_MX_F4
 *    operands are multiplied at twice the rate); bias fp32 [rows] or NULL.
 *  - residual [n][rows] of rdt, or NULL; out [n][rows] of odt; rdt and odt are fp32 or
 *    16-bit (any mix).  out may alias residual if type and pitch agree (each element is
 *    read before it is written) and overlaps nothing else (EINVAL).
 * Products of codes are exact, sums are fp32 on the tensor cores, and each output is
 * rounded once.  A block of NaN makes its token's (or its weight row's) outputs NaN. */
rvq_status moe_mx_linear(const uint8_t *x_dev, const uint8_t *x_scales_dev, moe_mx xfmt,
                         const uint8_t *w_dev, const uint8_t *w_scales_dev, moe_mx wfmt,
                         const float *bias_dev, int32_t n, int32_t rows, int32_t cols, moe_act act,
                         float alpha, const void *residual_dev, rvq_dtype rdt, int64_t ldr,
                         void *out_dev, rvq_dtype odt, int64_t ldo, void *ws_dev, size_t ws_bytes,
                         rvq_stream_t stream);

/* The first half of a gated feed-forward block:
 *   g = x wg^T + bg, u = x wu^T + bu, act(g) * u
 * into out [n][rows] of odt (fp32 or 16-bit), or, with out NULL, microscaled in ofmt
 * (codes, scales: moe_mx_quantize of the fp32 values) for the next product.
 * wg and wu [rows][cols] share wfmt; bg, bu fp32 [rows] or NULL, each by itself.  The
 * outputs overlap nothing (EINVAL). */
rvq_status moe_mx_gated_linear(const uint8_t *x_dev, const uint8_t *x_scales_dev, moe_mx xfmt,
                               const uint8_t *wg_dev, const uint8_t *wg_scales_dev,
                               const uint8_t *wu_dev, const uint8_t *wu_scales_dev, moe_mx wfmt,
                               const float *bg_dev, const float *bu_dev, int32_t n, int32_t rows,
                               int32_t cols, moe_act act, void *out_dev, rvq_dtype odt, int64_t ldo,
                               uint8_t *codes_dev, uint8_t *scales_dev, moe_mx ofmt, void *ws_dev,
                               size_t ws_bytes, rvq_stream_t stream);

/* moe_norm_join with the normed rows microscaled on the way out: h_out as there, and
 * codes, scales = moe_mx_quantize(norm(h_out) * w_pre), of the fp32 values.
 *  - h_out and xn (those values in xdt, for a router or routed experts beside the
 *    microscaled product) may be NULL; codes and scales ([n][d]) may not, and overlap
 *    nothing.  Other arguments and overlaps as in moe_norm_join.
 *  - rstd as there: moe_norm_join_backward takes it, with the gradient of the
 *    microscaled rows in dxn (straight through the rounding). */
rvq_status moe_norm_join_mx(const void *h_dev, rvq_dtype hdt, const void *y_dev, rvq_dtype ydt,
                            int32_t n, int32_t d, float alpha, const void *gate_dev,
                            moe_gate gate_kind, rvq_dtype gdt, int32_t post_norm,
                            const void *w_post_dev, const void *w_pre_dev, rvq_dtype wdt, float eps,
                            void *h_out_dev, void *xn_dev, rvq_dtype xdt, moe_mx fmt,
                            uint8_t *codes_dev, uint8_t *scales_dev, float *rstd_dev,
                            rvq_stream_t stream);

/* How the current device computes the products of moe_linear or (gated)
 * moe_gated_linear, or (backward) those of their gradients, both wanted: lets a test
 * say which way it ran.  Launches nothing.  out[0]: 1 if dx and dw share a launch; then for
 * the forward product or dx, and (backward) for dw: a moe_way, the parts or the pairs
 * of CTAs that a tile is cut into, the tile's columns (0 for MOE_WAY_STREAM). */
typedef enum moe_way {
    MOE_WAY_STREAM = 0, /* weights streamed past the tokens                     */
    MOE_WAY_TILES = 1,  /* whole tiles                                          */
    MOE_WAY_PARTS = 2,  /* tiles cut by depth, added by a second launch         */
    MOE_WAY_SPLIT = 3   /* tiles split by depth among the pairs of a cluster    */
} moe_way;
rvq_status rvq_selftest_dense_plan(int32_t gated, int32_t backward, int32_t n, int32_t rows,
                                   int32_t cols, int32_t out[7]);

/* The same of moe_mx_linear or (gated) moe_mx_gated_linear: out[0] is MOE_WAY_STREAM or
 * MOE_WAY_TILES, out[1] the CTAs that the depth of a streamed product is split among. */
rvq_status rvq_selftest_mx_plan(int32_t gated, moe_mx xfmt, moe_mx wfmt, int32_t n, int32_t rows,
                                int32_t cols, int32_t out[2]);

/* Self-test of the failure path of the tensor-core kernel (no counterpart in
 * the pages): launches the prefill GEMM on one zero token routed to expert 0
 * with its MMA role first waiting for an mbarrier arrival that nothing makes.
 * The bounded wait (1 s) expires, every role of every block gives up, the
 * kernel frees its tensor memory and returns; afterwards rvq_ws_status()
 * reports RVQ_ETIMEOUT (bit RVQ_DEV_ERR_TIMEOUT) and the context stays usable.
 * No GPU fault, trap or hang is involved.  ws: as for moe_layer_forward with
 * n = 1, k = 1 (its contents are overwritten).  Synchronises the stream once
 * before the launch. */
rvq_status rvq_selftest_prefill_timeout(const rvq_moe_bank *bank, void *ws_dev, size_t ws_bytes,
                                        rvq_stream_t stream);

/* --------------------------------------------------------------------------
 * Workspace status block.
 * rvq_ws_clear: zero the status block (async).  Call once per workspace.
 * rvq_ws_status: synchronous; waits for `stream`, reads the status word,
 * returns RVQ_OK, RVQ_EDEVICE (index / non-finite), RVQ_ECORRUPT or
 * RVQ_ETIMEOUT, stores the raw bits in *bits_out if not NULL, and clears it.
 * ------------------------------------------------------------------------ */
rvq_status rvq_ws_clear(void *ws_dev, rvq_stream_t stream);
rvq_status rvq_ws_status(void *ws_dev, uint32_t *bits_out, rvq_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* RVQMOE_H */
