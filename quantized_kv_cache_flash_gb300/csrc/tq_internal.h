// Host <-> device parameter blocks and launcher entry points (internal).
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "tq.h"

namespace tq {

// Decode (split-K) kernel parameters.  A row group is up to group_rows (4, 8
// or 16) query rows (GQA heads x Tq) of one KV head: the N dimension of the
// warp-level MMAs, whose M dimension is 16 tokens.  The CTAs split the
// context's 32-token chunks of all (batch, kv head, row group) units evenly.
struct DecodeParams {
    const uint8_t* k_codes;   // packed K codes (unused for fp16 K)
    const __half* k_norm;     // fp16 K norms (unused for fp16 K)
    const uint8_t* v_codes;   // packed V codes
    const __half* v_norm;     // fp16 V norms
    const int32_t* lengths;   // [B]
    const __half* q;          // [B, Hq, Tq, 128]
    float* part_o;            // [num_ctas + units, 16, 128], units = batch * hkv * row_groups
    float* part_ml;           // [num_ctas + units, 16, 2]  (running max in log2 units, sum)
    uint32_t* status;
    int32_t batch, hkv, hq, group, tq, rows, row_groups, group_rows, cap, max_len;
    int32_t num_ctas;         // decode grid (one wave of token-balanced CTAs)
    float scale_log2e;        // softmax scale * log2(e)
    float sparse_tau;         // sparse-V threshold on the softmax weight (0: off)
    uint32_t* sparse_tiles;   // sparse V: [0] += 16-token tiles skipped, [1] += tiles judged
    int32_t table;            // 1: records carry their centroid x norm table (no norms)
    uint32_t ktab[4];         // prmt byte tables of the K codebook (lo0, lo1, hi0, hi1)
    uint32_t vtab[4];
    uint32_t signs[4];        // bit d set <=> s_d = -1
    // K centroids' rounding residuals c - fp16(c), scaled by 2^res_shift, as
    // e4m3 bytes (3-bit: indexed by the signed code; 4-bit: by magnitude rank)
    uint32_t ktab8[2];
    int32_t res_shift;
    int32_t k_res;            // 1: the K codebook has entries that are not fp16 values
    // Tree attention (tree != null): the last tq tokens are a drafted block,
    // row j sees every token before it and token i of it where bit i of its
    // words tree[b * tree_per_seq + j * tree_words ..] is set.
    const uint32_t* tree;
    int32_t tree_words, tree_per_seq;   // tree_per_seq 0: one mask for all sequences
};

constexpr int kMaxTreeGroup = 128;      // query heads per KV head of a tree

struct CombineParams {
    const float* part_o;
    const float* part_ml;
    const int32_t* lengths;
    __half* out;              // [B, Hq, Tq, 128]
    uint32_t* status;
    int32_t batch, hkv, hq, group, tq, row_groups, group_rows, max_len, num_ctas;
    int32_t nan_rows;         // 1 (a tree's call): a row with a NaN sum is NaN, not a row that sees no token
    float v_rescale;
    uint32_t signs[4];
};

struct EncodeParams {
    const __half* k_new;      // [B, Hkv, T, 128]
    const __half* v_new;
    uint8_t* k_codes;         // packed codes or fp16 K rows (fp16 K mode)
    __half* k_norm;
    uint8_t* v_codes;
    __half* v_norm;
    int32_t* lengths;
    uint32_t* status;
    uint32_t* counter;        // zero between calls; the last CTA resets it
    uint32_t* tiles_next;     // large appends: the next tile to hand out (zero between calls, reset likewise)
    int32_t batch, hkv, t_new, cap;
    // n / t_new and n / hkv for 0 <= n < 2^31 as (n * m) >> s (see div_magic)
    uint32_t div_t_m, div_h_m;
    int32_t div_t_s, div_h_s;
    uint32_t signs[4];
    // decision thresholds on |u| over the positive half of the codebook:
    // a > tau_k  <=>  a >= gt[k];   a >= tau_k  <=>  a >= ge[k]   (fp32, exact)
    float k_gt[7], k_ge[7], v_gt[7], v_ge[7];
    // table records: 48 bytes of 3-bit codes + fp16(c_j * n16), j = 0..7
    int32_t table;
    float k_cb[8], v_cb[8];
    // packed appends (cu != null): k_new, v_new are [total, Hkv, 128] and
    // sequence b's tokens are rows cu[b] .. cu[b + 1] - 1 (t_new is not used)
    const int32_t* cu;        // [B + 1]
    int32_t total;
    float k_mag[8], v_mag[8]; // the positive half of the codebooks, ascending
    // a value this close to a threshold (times the norm) is decided exactly; large appends:
    // the second one for vectors without entries below fine_min (times the norm)
    float k_near, v_near, k_near_fine, v_near_fine, k_fine_min, v_fine_min;
};

// Chunked-prefill attention (tcgen05) parameters.  One CTA = one (query
// tile of pos_per_tile positions x group heads, batch * kv head).
struct PrefillParams {
    const uint8_t* k_codes;   // packed K codes, or fp16 K rows (read through the tensor map)
    const __half* k_norm;
    const uint8_t* v_codes;
    const __half* v_norm;
    const int32_t* lengths;   // [B]
    const __half* q;          // [B, Hq, Tq, 128]
    __half* out;              // [B, Hq, Tq, 128]
    uint32_t* status;
    int32_t batch, hkv, hq, group, tq, cap, max_len;
    int32_t pos_per_tile;     // query positions per 128-row tile (128 / group)
    int32_t mtiles;           // tiles per kv head
    float scale_log2e, v_rescale;
    uint32_t ktab[4], vtab[4], signs[4];
    // packed sequences (tq_packed_prefill.cu; cu != null): q and out are [total, Hq, 128], sequence
    // b's rows cu[b] .. cu[b + 1] - 1 (tq and mtiles are not used)
    const int32_t* cu;        // [B + 1]
    int32_t total;
    int32_t slots;            // query tile pairs of all sequences, at most
    int32_t span;             // positions per pair
    uint32_t span_inv;        // 2^32 / span, rounded up
};

// Tree attention on the tensor cores (tq_tree.cu): units are (batch, kv head,
// tile of 128 query rows), a row of a unit is node * group + head of the group.
struct TreeParams {
    const uint8_t* k_codes;   // packed K codes (fp16 K: read through the tensor map)
    const __half* k_norm;
    const uint8_t* v_codes;
    const __half* v_norm;
    const int32_t* lengths;   // [B]
    const __half* q;          // [B, Hq, Tq, 128]
    __half* out;
    const uint32_t* tree;     // as in DecodeParams
    int32_t tree_words, tree_per_seq;
    float* part_o;            // [num_ctas + units, 128, 128]
    float* part_ml;           // [num_ctas + units, 128, 2]
    uint8_t* q_tiles;         // per unit Q' (q_hi, q_lo): 64 KB (fp16 K: 32 KB)
    uint32_t* status;
    int32_t batch, hkv, hq, group, tq, cap, max_len;
    int32_t rows;             // group * tq
    int32_t row_tiles, per_b; // tiles of rows per KV head, units per sequence
    int32_t num_ctas;
    float scale_log2e, v_rescale;
    uint32_t ktab[4], vtab[4], signs[4];
};

// Keeping the accepted tokens of a drafted block (see tq_cache_compact).
struct CompactParams {
    uint8_t* k_data;          // packed codes, table records or fp16 K rows
    uint8_t* v_data;
    __half* k_norm;           // null where the mode has none
    __half* v_norm;
    int32_t* lengths;
    const int32_t* start;     // [B] first token of the drafted block
    const int32_t* keep;      // [B, max_keep] places in the block, ascending
    const int32_t* num_keep;  // [B]
    uint32_t* status;
    int32_t batch, hkv, cap, rbk, rbv, max_keep, num_drafted;
};

// Copying sequences (see tq_cache_copy).
struct CopyParams {
    const uint8_t* k_src;
    const uint8_t* v_src;
    const __half* kn_src;     // null where the mode has none
    const __half* vn_src;
    uint8_t* k_dst;
    uint8_t* v_dst;
    __half* kn_dst;
    __half* vn_dst;
    const int32_t* src_lengths;
    int32_t* dst_lengths;
    const int32_t* src;       // [pairs] sequence of the source cache
    const int32_t* dst;       // [pairs] sequence of the destination cache
    const int32_t* num_tokens;  // [pairs], or null: the whole source
    uint32_t* status;
    int32_t pairs, hkv, src_batch, dst_batch, src_cap, dst_cap, rbk, rbv, max_len;
    int32_t same;             // 1: source and destination are one cache
};

// The softmax weights that tokens get (see tq_attention_weights).  A row of a (batch, KV
// head) unit is head of the group * tq + query position; 256 rows are a pair of query tiles.
//  A call takes the pairs pair0 .. pair0 + pairs - 1.
struct WeightsParams {
    const uint8_t* k_codes;   // packed K codes (fp16 K: read through the tensor map)
    const __half* k_norm;
    const int32_t* lengths;   // [B]
    const __half* q;          // [B, Hq, Tq, 128]
    const int32_t* seen;      // [B] tokens that have a weight already, or null: all but the last tq
    float* weights;           // [B, Hkv, cap]
    // workspace
    uint8_t* q_tiles;         // [units][pairs] Q': q_hi and q_lo of 256 rows, 64 KB each (quantized K)
    float2* part_ml;          // [ctas + units * pairs][256] a run's (maximum, sum) of each row
    float* part_w;            // [units][pairs][part_len] sums per pair; null: one pair, added at once
    uint32_t* status;
    int32_t batch, hkv, hq, group, tq, rows, cap, max_len;
    int32_t pairs, pair0, part_len, ctas;
    uint32_t div_tq_m, div_pairs_m;   // n / tq and n / pairs as (n * m) >> s (see div_magic)
    int32_t div_tq_s, div_pairs_s;
    float scale_log2e, decay;
    uint32_t ktab[4], signs[4];
};

// The same for up to 16 rows per KV head (tq_weights_step.cu), in groups as the decode's
// (group_rows_for).
struct StepParams {
    const uint8_t* k_codes;
    const __half* k_norm;
    const int32_t* lengths;
    const __half* q;
    const int32_t* seen;
    float* weights;
    float* scores;            // workspace: [units][score_len][group rows], log2 units
    float2* part_ml;          // workspace: [ctas + units][group rows]
    uint32_t* status;
    int32_t batch, hkv, hq, group, tq, rows, cap, max_len, score_len, ctas;
    int32_t span;             // tokens per CTA of the second kernel
    float scale_log2e, decay;
    uint32_t ktab[4], signs[4];
};

// Eviction by weight (see tq_cache_evict).
struct EvictParams {
    const uint8_t* k_src;
    const uint8_t* v_src;
    const __half* kn_src;     // null where the mode has none
    const __half* vn_src;
    uint8_t* k_dst;
    uint8_t* v_dst;
    __half* kn_dst;
    __half* vn_dst;
    const int32_t* src_lengths;
    int32_t* dst_lengths;
    const float* weights;     // [B, Hkv, src_cap]
    float* new_weights;       // [B, Hkv, dst_cap], or null
    const int32_t* num_keep;  // [B]
    int32_t* kept;            // [B, Hkv, max_keep]
    int32_t* counts;          // workspace: tokens kept per sequence, -1 where it is left as it was
    uint32_t* status;
    int32_t batch, hkv, src_cap, dst_cap, rbk, rbv, max_keep, max_len, sinks, recent;
    int32_t same;             // 1: in place
    int32_t move_ctas;        // CTAs per unit of the move to another cache
};

// Verification of drafted tokens (see tq_verify_tree).
struct VerifyParams {
    const int32_t* tokens;    // [B, N]
    const int32_t* parents;   // [1 or B, N]
    const float* target;      // [B, N] rows of ld_target floats
    const float* draft;       // [B, N] rows of ld_draft floats, or null
    const float* uniforms;    // [B, N]
    int32_t* keep;            // [B, N]
    int32_t* num_keep;        // [B]
    int32_t* next;            // [B]
    uint32_t* status;
    int64_t ld_target, ld_draft;
    int32_t batch, nodes, vocab, parents_per_seq;
};

// Division of 0 <= n < 2^31 by a constant d >= 1 as a multiply-high: with
// l = ceil(log2 d), s = 31 + l and m = ceil(2^s / d) (below 2^32),
// floor(n m / 2^s) = floor(n / d), because m d - 2^s < d <= 2^l and
// n < 2^31 keep the error term n (m d - 2^s) / (d 2^s) below 1/d.
inline void div_magic(uint32_t d, uint32_t* m, int32_t* s) {
    int l = 0;
    while ((1ull << l) < d) ++l;
    *s = 31 + l;
    *m = static_cast<uint32_t>(((1ull << *s) + d - 1) / d);
}

// Launchers (return a cudaError_t value).
// group_rows (p.group_rows) selects the 4-, 8- or 16-row variant.
int launch_decode(int kbits, int vbits, const DecodeParams& p, const CUtensorMap* kmap,
                  cudaStream_t stream, cudaEvent_t ev_begin, cudaEvent_t ev_end);
int launch_combine(const CombineParams& p, cudaStream_t stream);
// Appends of more than kEncodeSmallMax vectors per stream run on the tensor
// cores and read their inputs through kmap / vmap (encode_rows_map of k_new /
// v_new); smaller ones ignore the maps.  (Packed, 4 bits: 1024 vectors 7.0 us a warp
// each and 13.1 on the tensor cores, 4096 10.3 and 13.1, 3 bits 9.7 and 10.4.)
constexpr long long kEncodeSmallMax = 4096;
int launch_encode(int kbits, int vbits, const EncodeParams& p, const CUtensorMap* kmap,
                  const CUtensorMap* vmap, cudaStream_t stream);
// The same for packed appends (p.cu); nvec = p.total * p.hkv decides the kernel.
int launch_encode_packed(int kbits, int vbits, const EncodeParams& p, const CUtensorMap* kmap,
                         const CUtensorMap* vmap, cudaStream_t stream);

// Resident CTAs per SM of a decode variant (for the host split planner);
// res: the variant with the centroid residual product.
int decode_ctas_per_sm(int kbits, int vbits, int group_rows, bool table, bool res);
int launch_prefill(int kbits, int vbits, const PrefillParams& p, const CUtensorMap* kmap,
                   cudaStream_t stream);
int launch_packed_prefill(int kbits, int vbits, const PrefillParams& p, const CUtensorMap* kmap, cudaStream_t stream);
int launch_tree(int kbits, int vbits, const TreeParams& p, const CUtensorMap* kmap, cudaStream_t stream,
                cudaEvent_t ev0, cudaEvent_t ev1);
int launch_compact(const CompactParams& p, cudaStream_t stream);
// CTAs = pairs * hkv * ceil(max_len / kCopyTokens), below 2^31
constexpr int kCopyTokens = 256;
int launch_copy(const CopyParams& p, cudaStream_t stream);
int launch_weights(int kbits, const WeightsParams& p, const CUtensorMap* kmap, const CUtensorMap* qmap,
                   cudaStream_t stream);
int launch_weights_step(int kbits, int group_rows, const StepParams& p, const CUtensorMap* kmap, cudaStream_t stream);
int weights_step_ctas_per_sm(int kbits, int group_rows);
constexpr int kEvictMoveCtas = 8;   // of the cluster that moves a unit's records in place
int launch_evict(EvictParams p, cudaStream_t stream);
int launch_verify(const VerifyParams& p, cudaStream_t stream);
int launch_selftest_stall(uint32_t* status, uint64_t limit_ns, cudaStream_t stream);

// Query rows per row group for `rows` query rows of one KV head: 4 when K is
// quantized and at most 4 rows share a KV head (the low halves of the rotated
// query then ride in the score MMA's spare columns), else 8, or 16 per group.
inline int group_rows_for(int rows, int kbits) {
    return (rows <= 4 && kbits != 16) ? 4 : rows <= 8 ? 8 : 16;
}

// Launch with programmatic stream serialization: the kernel may be scheduled
// while its predecessor in the stream finishes (every kernel of this library
// waits for its predecessor with griddep_wait() before touching memory).
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The same with clusters of `cluster` CTAs.
template <typename... Params, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(Params...), dim3 grid, dim3 block, int cluster, size_t smem,
                               cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Opt a kernel into clusters of more than 8 CTAs on the current device, once per device
// (`done` as in set_smem_attr_once).
template <typename Kernel>
cudaError_t allow_large_clusters_once(Kernel kernel, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

// Opt a kernel into `bytes` of dynamic shared memory (and, carveout >= 0, a
// preferred shared-memory carveout) on the current device, once per device:
// `done` keeps one bit per device ordinal (devices past 63 set it every call).
// min_regs: the registers per thread that a kernel's split between its warp groups
// counts on; built with fewer it would wait for them for ever, so it is refused.
template <typename Kernel>
cudaError_t set_smem_attr_once(Kernel kernel, int bytes, std::atomic<uint64_t>& done, int carveout = -1,
                               int min_regs = 0) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && carveout >= 0)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, carveout);
    if (e == cudaSuccess && min_regs > 0) {
        cudaFuncAttributes a;
        e = cudaFuncGetAttributes(&a, kernel);
        if (e == cudaSuccess && a.numRegs < min_regs) e = cudaErrorInvalidKernelImage;
    }
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

// Records that carry a centroid x norm table instead of a norm.
inline bool mode_table(int mode) { return mode == TQ_TURBO3_TABLE; }

// (K bits, V bits) of a mode; 16 = fp16 K.
inline int mode_bits(int mode, int* kb, int* vb) {
    switch (mode) {
        case TQ_TURBO4_ASYM: *kb = 16; *vb = 4; return TQ_OK;
        case TQ_TURBO3: *kb = 3; *vb = 3; return TQ_OK;
        case TQ_TURBO4: *kb = 4; *vb = 4; return TQ_OK;
        case TQ_TURBO3_ASYM: *kb = 16; *vb = 3; return TQ_OK;
        case TQ_TURBO4K_3V: *kb = 4; *vb = 3; return TQ_OK;
        case TQ_TURBO3_TABLE: *kb = 3; *vb = 3; return TQ_OK;
        default: return TQ_ERR_UNSUPPORTED;
    }
}

// ---------------------------------------------------------------------------
// Host helpers shared by the entry points (defined in tq_api.cu)
// ---------------------------------------------------------------------------
namespace host {

// Kernel-side forms of a checked codebook.
struct CodebookTables {
    bool valid = false;
    int bits = 0;
    float cb[16] = {};
    uint32_t tab[4] = {};  // prmt byte tables of the fp16 centroids (lo0, lo1, hi0, hi1)
    float gt[7] = {}, ge[7] = {};  // encode decision thresholds (see EncodeParams)
    // e4m3 bytes of (c - fp16(c)) * 2^res_shift (3-bit: by signed code; 4-bit:
    // by magnitude rank), for the score's fp8 residual product
    uint32_t tab8[2] = {};
    int res_shift = 0;
    // how far an encode's value and a threshold may be off together, as a multiple of
    // the vector's norm: the warp-per-vector kernel and the tensor-core one (and that one
    // where no entry is below fine_min times the norm)
    float near_small = 0.f, near_tc = 0.f, near_fine = 0.f, fine_min = 0.f;
};

constexpr int kSMs = 152;  // GB300 (only used to size the split grids)

int cuda_err_code(cudaError_t e);
bool aligned16(const void* p);
// Non-null and 4-byte aligned: a list of 32-bit numbers that a kernel reads.
bool list_ok(const void* p);
// Mode, shape, pointers and codebooks of a cache; *kb, *vb = its bits (16 = fp16 K).
int check_cache(const tq_cache* c, int* kb, int* vb);
// (Re)builds *t unless it already holds this codebook.
int build_tables(const float* cb, int n, int bits, CodebookTables* t);
// s_d = -1 <=> bit d of out (splitmix64 of the rotation seed).
void make_signs(uint64_t seed, uint32_t out[4]);
// Tensor map of the fp16 K rows of a cache (driver entry point looked up once).
int encode_kmap(CUtensorMap* map, const tq_cache* c);
// Tensor map of `rows` fp16 vectors of 128 dims at `base` (16-byte aligned),
// boxes of 128 rows x 64 halves (128-byte swizzle): the encode's input tiles.
int encode_rows_map(CUtensorMap* map, const void* base, uint64_t rows);
// Tensor map of fp16 vectors [tokens, heads, 128] at `base`, boxes of 128 tokens
// of one head x 64 halves: a packed append's input tiles.
int encode_tokens_map(CUtensorMap* map, const void* base, uint64_t heads, uint64_t tokens);
// Whether every entry of a codebook is an fp16 value (no rounding residual).
bool codebook_is_fp16(const float* cb, int n);

// One decode call's checked arguments and the row grouping and grid derived
// from them.
struct DecodePlan {
    int kb, vb;
    bool res;          // quantized K whose codebook is not all fp16 values
    int group, rows, group_rows, row_groups;
    long long units;   // (batch, kv head, row group) units
    int ctas;          // decode grid
};
// (max_rows: query rows per KV head that the caller takes)
int plan_decode(const tq_cache* c, const void* q, const void* out, int num_q_heads, int tq_rows,
                int max_len_hint, float scale, DecodePlan* pl, int max_rows = 256);
// The mask of a drafted tree: words[(shared ? 0 : b)][tq][ceil(tq / 32)].
struct TreeMask {
    const uint32_t* words;
    bool shared;
};
// Split-K scratch of a plan: (ctas + units) slots of 16 rows x (128 + 2) floats.
inline size_t decode_slots(const DecodePlan& pl) { return size_t(pl.ctas + pl.units) * 16; }
// Launch the decode and combine kernels of a plan on `stream`, the partials
// in `part` (decode_slots(pl) * 130 floats), device status bits ORed into
// `status`; ev0/ev1 (optional) bracket the decode kernel.
int launch_decode_plan(const DecodePlan& pl, const tq_cache* c, const CodebookTables& kt,
                       const CodebookTables& vt, const uint32_t signs[4], const CUtensorMap* kmap,
                       const void* q, int num_q_heads, int tq_rows, int max_len_hint, float scale,
                       float tau, void* out, float* part, uint32_t* status, cudaStream_t stream,
                       cudaEvent_t ev0, cudaEvent_t ev1, uint32_t* sparse_tiles = nullptr,
                       const TreeMask* tree = nullptr);

}  // namespace host

}  // namespace tq
