// Attention of a drafted tree over the packed cache on the 5th-generation
// tensor cores: split over the context, for blocks of more than 16 query rows
// per KV head (fewer run on the decode kernel, whose warp MMAs hold 16).
//
// Per 128 query rows (drafted nodes x heads of the group) and 128 tokens:
//   S[128 x 128] = Q' . K^T          (8 or 16 MMAs of K = 16, fp32 in tensor memory)
//   P[r][t]      = 2^(S n_k scale log2 e - base_r) n_v    (rounded to fp16)
//   O[128 x 128] += P . C_v          (8 MMAs, fp32 in tensor memory)
// with Q' = Rot(q) as two fp16 halves (quantized K: K's tile holds the fp16
// centroids, the norm goes to the fp32 scores) or q (fp16 K).  V's tile holds
// the centroids themselves, exact in fp16, and the V norm goes into P, so a
// term is rounded once.  With e the exponent of a tile's largest V norm, the base of a
// row may trail its scores by 14 - e (log2; p n_v stays below 2^15), and where it moves
// it stops 10 short of that, so the largest weights' terms start at 2^4 or above whatever
// the norms' size (a term loses bits below 2^-18, and less than 2^-29 of the largest norm
// where it vanishes).  With a margin of 4 every third tile had a row that moved its base,
// with 10 hardly any has.
//
// A CTA is a pipeline over the 128-token tiles of its share, a stage per kind of
// warp, with two K, V, S and P tiles between them: four warps dequantise K and
// four V, eight run the softmax (fragments of 16 rows x 128 tokens per warp), a warp
// each issues S, P.V, the K copies and the V copies.  So S(n + 1) and P.V(n - 1) run
// under softmax(n).
//
// What bounds it: a tile takes 3000 cycles.  Its 24 MMAs are 1536 of the tensor core
// (52% active measured); shared memory moves 2000 wavefronts of loads and stores and
// 1024 of MMA operands (K, V and P, so Q' lies in tensor memory), together nine tenths of
// the time; the schedulers issue 65% of it, half on the ALU's byte permutes.  All kinds of
// warp share the instruction caches, so loops are rolled where they can be.  Measured:
// 64 nodes, 8 sequences of 4000 to 16384 tokens, turbo4, 32 / 8 heads, 143 us (661 TFLOP/s,
// q_lo's products not counted); 33 nodes, three of 777 to 16351, fp16 K, 28 / 4 heads,
// 36 us; 16 nodes, one of 8192, turbo3, 16.7 us.  P over S in tensor memory took 147 us
// for the first, Q' in shared memory besides 149.
//
// Split: the (batch, kv head, row tile) units lie end to end as 128-token
// chunks, and CTA c of P takes [c C / P, (c + 1) C / P) of the C chunks, from
// the actual lengths; it writes one partial (m, l, O) per unit that it touches,
// which tq_tree_combine_kernel merges, normalises and rotates back.  Q' is
// rotated and split by a small kernel before, while this one sets up and
// dequantises its first tiles.
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kTok = 128;            // tokens per tile (chunk)
constexpr int kTreeRows = 128;       // query rows per unit
constexpr int kMargin = 10;            // log2 by which scores may grow before their row's base moves again

template <int KB, int VB>
struct TreeCfg {
    static constexpr int kRbK = (KB == 0) ? 256 : KB * 16;
    static constexpr int kRbV = VB * 16;
    static constexpr int kVtOff = 0;                                  // two V^T tiles [dim][token] (32 KB each)
    static constexpr int kPOff = kVtOff + 65536;                      // two P tiles [row][token]
    static constexpr int kKOff = kPOff + 65536;                       // two K tiles [token][dim] (fp16 K: as copied)
    static constexpr int kSKOff = kKOff + 65536;                      // two tiles of K records (quantized K)
    static constexpr int kSK = (KB == 0) ? 0 : kTok * kRbK;
    static constexpr int kSVOff = kSKOff + 2 * kSK;                   // two tiles of V records
    static constexpr int kSV = kTok * kRbV;
    static constexpr int kColOff = kSVOff + 2 * kSV;                  // two tiles of n_k scale log2 e [128]
    static constexpr int kNvOff = kColOff + 2 * kTok * 4;             // two tiles of n_v [128]
    static constexpr int kNmOff = kNvOff + 2 * kTok * 4;              // two tiles of the largest n_v of 32 tokens [4]
    // mbarriers, of even and odd tiles: K copied, V copied, K (and norms) stored,
    // V stored, P stored, S done, P.V done; Q' stored, all MMAs done [2] (after
    // a time-out)
    static constexpr int kBarOff = kNmOff + 32;
    static constexpr int kBars = 20;
    static constexpr int kSmem = kBarOff + 8 * kBars + 8;             // and the TMEM slot
    static constexpr int kSmemAlloc = kSmem + 256;   // to a 1024-byte boundary: the base is one, but for 256 bytes at most
    static_assert(kSmemAlloc <= 232448, "227 KB per CTA");
    static constexpr uint32_t kIdesc = umma_idesc_f16_f32(128, 128);
};

// Warp groups of four warps: 0 and 1 softmax, 2 dequantises K, 3 V, 4 has the
// issuing threads.  Registers per thread after the split (their sum times 128
// is at most the launch's 640 x 96).
constexpr int kTreeThreads = 640;
constexpr int kRegsLaunch = 96, kRegsSoftmax = 136, kRegsDequant = 72, kRegsIssue = 64;
static_assert(2 * kRegsSoftmax + 2 * kRegsDequant + kRegsIssue <= 5 * kRegsLaunch, "within the launch's registers");

__device__ __forceinline__ int tree_chunks(int L, int max_len) {
    const int n = min(L, max_len);
    return n > 0 ? (n + kTok - 1) / kTok : 0;
}

__device__ __forceinline__ int lane_prefix(int v, int lane) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// The sequences' lengths and chunks laid end to end (whole warp; the first 32
// sequences in registers, one per lane, so that batches of up to 32 read
// `lengths` once).
struct TreeScan {
    int len, inc, v;   // this lane's sequence: length, chunks up to and with it, its own
    int total;         // of all sequences

    __device__ __forceinline__ void init(const TreeParams& p, int lane) {
        len = lane < p.batch ? p.lengths[lane] : 0;
        v = tree_chunks(len, p.max_len) * p.per_b;
        inc = lane_prefix(v, lane);
        int more = 0;
        for (int b = 32 + lane; b < p.batch; b += 32) more += tree_chunks(p.lengths[b], p.max_len) * p.per_b;
        if (p.batch > 32) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) more += __shfl_xor_sync(0xffffffffu, more, o);
        }
        total = __shfl_sync(0xffffffffu, inc, 31) + more;
    }

    // the sequence that holds chunk pos < total, its length and the chunks before it
    __device__ __forceinline__ void locate(const TreeParams& p, int pos, int lane, int& b, int& before, int& L) const {
        unsigned hit = __ballot_sync(0xffffffffu, inc > pos);
        if (hit) {
            b = __ffs(hit) - 1;
            before = __shfl_sync(0xffffffffu, inc - v, b);
            L = __shfl_sync(0xffffffffu, len, b);
            return;
        }
        int cum = __shfl_sync(0xffffffffu, inc, 31);
#pragma unroll 1
        for (int b0 = 32; b0 < p.batch; b0 += 32) {
            const int l2 = b0 + lane < p.batch ? p.lengths[b0 + lane] : 0;
            const int v2 = tree_chunks(l2, p.max_len) * p.per_b;
            const int inc2 = lane_prefix(v2, lane);
            hit = __ballot_sync(0xffffffffu, cum + inc2 > pos);
            if (hit) {
                const int l = __ffs(hit) - 1;
                b = b0 + l;
                before = cum + __shfl_sync(0xffffffffu, inc2 - v2, l);
                L = __shfl_sync(0xffffffffu, l2, l);
                return;
            }
            cum += __shfl_sync(0xffffffffu, inc2, 31);
        }
        b = 0;   // pos past the end (not reached by the callers)
        before = L = 0;
    }
};

// 32 bits of visibility for drafted tokens i0 .. i0 + 31 of a mask row of W
// words: i < 0 are context tokens, all seen.
__device__ __forceinline__ uint32_t tree_window(const uint32_t* row, int W, int i0) {
    if (i0 <= -32) return 0xffffffffu;
    if (i0 < 0) return (row[0] << -i0) | ((1u << -i0) - 1u);
    const int k = i0 >> 5;
    const uint32_t lo = k < W ? row[k] : 0u, hi = k + 1 < W ? row[k + 1] : 0u;
    return __funnelshift_r(lo, hi, i0 & 31);
}

}  // namespace

// Q' of every unit, fp16 (q_hi, then q_lo): a warp per row (the rows past the
// last one are zero), lane l dims 4l .. 4l + 3, stored as [16 pieces of 8 dims]
// [128 rows], so that the rows' threads read 16 bytes each, together.
template <bool ROTATE>
__global__ void __launch_bounds__(256) tq_tree_q_kernel(const __grid_constant__ TreeParams p) {
    const int lane = threadIdx.x & 31;
    const int row = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    griddep_wait();
    griddep_launch_dependents();   // (what came before this call is done now: the next kernel may read the cache)
    const int unit = row / kTreeRows, r = row - unit * kTreeRows;
    const int b = unit / p.per_b, ui = unit - b * p.per_b;
    const int h = ui / p.row_tiles, rr = (ui - h * p.row_tiles) * kTreeRows + r;
    uint2 hv = make_uint2(0u, 0u), lv = hv;
    if (rr < p.rows) {
        const int j = rr / p.group, hl = rr - j * p.group;
        hv = reinterpret_cast<const uint2*>(
            p.q + ((static_cast<size_t>(b) * p.hq + h * p.group + hl) * p.tq + j) * kD)[lane];
        if constexpr (ROTATE) {
            const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&hv.x));
            const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&hv.y));
            float x[4] = {f0.x, f0.y, f1.x, f1.y};
            const uint32_t sn = sign_nibble(p.signs, lane);
#pragma unroll
            for (int d = 0; d < 4; ++d) x[d] = ((sn >> d) & 1u) ? -x[d] : x[d];
            wht128_lane4(x, lane);
#pragma unroll
            for (int d = 0; d < 4; ++d) x[d] *= 0.08838834764831845f;   // 1/sqrt(128)
            hv = make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
            // q_lo = Rot(q) - q_hi (exact in fp32), rounded once more
            const float2 h0 = __half22float2(*reinterpret_cast<const __half2*>(&hv.x));
            const float2 h1 = __half22float2(*reinterpret_cast<const __half2*>(&hv.y));
            lv = make_uint2(pack_half2(x[0] - h0.x, x[1] - h0.y), pack_half2(x[2] - h1.x, x[3] - h1.y));
        }
    }
    uint8_t* tile = p.q_tiles + static_cast<size_t>(unit) * (ROTATE ? 65536 : 32768) +
                    ((lane >> 1) * kTreeRows + r) * 16 + (lane & 1) * 8;
    *reinterpret_cast<uint2*>(tile) = hv;
    if constexpr (ROTATE) *reinterpret_cast<uint2*>(tile + 32768) = lv;
}

template <int KB, int VB>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tq_tree_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap kmap) {
    using C = TreeCfg<KB, VB>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int lane = tid & 31;
    const int wg = warp >> 2;

    // (The cache, lengths and mask come from work before the Q' kernel, whose
    // CTAs waited for it before they let this grid launch; the Q' tiles are read
    // behind griddep_wait.)
    const int P = static_cast<int>(gridDim.x), c_me = static_cast<int>(blockIdx.x);
    TreeScan scan;
    scan.init(p, lane);
    // floor(c total / P): c (total mod P) < P^2 is small
    const int per_cta = scan.total / P, over = scan.total - per_cta * P;
    const int lo = __shfl_sync(0xffffffffu, c_me * per_cta + c_me * over / P, 0);
    const int hi = __shfl_sync(0xffffffffu, (c_me + 1) * per_cta + (c_me + 1) * over / P, 0);
    // (uniform over the CTA; a grid without work ends after its predecessor all
    // the same.  The base of dynamic shared memory is a 1024-byte boundary.)
    if (lo >= hi || smem - smem_raw > 256) {
        griddep_wait();
        if (lo < hi && tid == 0) atomicOr(p.status, kStatusPipelineStall);
        return;
    }

    const uint32_t bars = smem_u32(smem + C::kBarOff);
    const uint32_t bar_k = bars, bar_v = bars + 16, bar_kr = bars + 32, bar_vr = bars + 48, bar_p = bars + 64,
                   bar_s = bars + 80, bar_o = bars + 96, bar_q = bars + 112, bar_x = bars + 120,
                   bar_n = bars + 136;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 8 * C::kBars);
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(bar_k + 8 * i, 1);      // K copied, V copied
        for (int i = 0; i < 4; ++i) mbar_init(bar_kr + 8 * i, 128);   // K stored, V stored
        for (int i = 0; i < 2; ++i) mbar_init(bar_p + 8 * i, 256);    // P stored
        for (int i = 0; i < 4; ++i) mbar_init(bar_s + 8 * i, 1);      // S done, P.V done
        mbar_init(bar_q, 256);                                        // Q' stored
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_x + 8 * i, 1);
            mbar_init(bar_n + 8 * i, 128);                            // scales and norms stored
        }
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(smem_u32(tslot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // tensor memory: S of even and odd tiles (128 columns each), O (128), q_hi and
    // q_lo (64 each)
    const uint32_t tmem = *tslot, tm_o = tmem + 256, tm_q = tmem + 384;

    bool stalled = false;   // once set, waits return at once and nothing more is issued
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!stalled && !mbar_wait_bounded(bar, parity)) stalled = true;
    };
    // Tile n of a segment is tile t = tbase + n of the CTA: it takes the buffers
    // t & 1, whose barriers' phase is t >> 1.
    int tbase = 0, pos = lo;
    uint32_t segs = 0;

    // The segment at pos: chunks [k0, k0 + ntiles) of unit (b, h, rt).
    struct Segment {
        int b, ui, k0, ntiles, L, t_lim;
        size_t row0;
    };
    auto segment = [&]() {
        Segment s;
        int before;
        scan.locate(p, pos, lane, s.b, before, s.L);
        s.b = __shfl_sync(0xffffffffu, s.b, 0);
        before = __shfl_sync(0xffffffffu, before, 0);
        s.L = __shfl_sync(0xffffffffu, s.L, 0);
        const int nch = tree_chunks(s.L, p.max_len);
        s.ui = (pos - before) / nch;   // h * row_tiles + rt
        s.k0 = (pos - before) - s.ui * nch;
        s.ntiles = min(nch - s.k0, hi - pos);
        s.t_lim = min(s.L, p.max_len);
        s.row0 = (static_cast<size_t>(s.b) * p.hkv + s.ui / p.row_tiles) * p.cap;
        return s;
    };
    // all warps: the end of a segment; true when some wait timed out
    auto end_segment = [&](int ntiles) {
        tc_fence_before();
        const bool bad = __syncthreads_or(stalled) != 0;
        tc_fence_after();
        tbase += ntiles;
        pos += ntiles;
        ++segs;
        return bad;
    };

    if (wg == 4) {
        // ---- issuing warps: S, the K copies, the V copies, P.V ----
        regs_dec<kRegsIssue>();
        const int role = warp & 3;
        bool bad = false;
        while (pos < hi && !bad) {
            const Segment s = segment();
            if (role == 0 || role == 3) {
                // S(n) and P.V(n) by a warp each, so that the tensor core has the
                // other's products while one waits.  The whole warp runs the loop, so
                // that addresses and descriptors stay in uniform registers, and one
                // lane issues.
                const uint32_t one = lane == 0 ? 1u : 0u;
                const uint32_t tmu = __shfl_sync(0xffffffffu, tmem, 0);
                const uint64_t adesc = umma_desc_sw128(__shfl_sync(0xffffffffu, smem_u32(smem + C::kPOff), 0));
                const uint64_t bdesc =
                    umma_desc_sw128(__shfl_sync(0xffffffffu, smem_u32(smem + (role == 0 ? C::kKOff : C::kVtOff)), 0));
                if (role == 0) wait(bar_q, segs & 1);
#pragma unroll 1
                for (int n = 0; n < s.ntiles; ++n) {
                    const int t = tbase + n, u = t & 1;
                    const uint32_t off = static_cast<uint32_t>(u) * (32768 >> 4);
                    if (role == 0) {
                        wait((KB == 0 ? bar_k : bar_kr) + 8 * u, (t >> 1) & 1);
                        if (t >= 2) wait(bar_p + 8 * u, ((t >> 1) - 1) & 1);   // softmax(t - 2) has read this S tile
                    } else {
                        wait(bar_vr + 8 * u, (t >> 1) & 1);
                        wait(bar_p + 8 * u, (t >> 1) & 1);
                    }
                    if (__any_sync(0xffffffffu, stalled)) break;
                    tc_fence_after();
                    if (role == 0) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint64_t d = bdesc + off + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
                            umma_f16_ts_if(one, tmu + 128 * u, tmu + 384 + 8 * kk, d, C::kIdesc, kk > 0 ? 1u : 0u);
                            if constexpr (KB != 0) umma_f16_ts_if(one, tmu + 128 * u, tmu + 448 + 8 * kk, d, C::kIdesc, 1u);
                        }
                    } else {
                        const uint32_t more = n > 0 ? 1u : 0u;
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint32_t k = off + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
                            umma_f16_if(one, tmu + 256, adesc + k, bdesc + k, C::kIdesc, kk > 0 ? 1u : more);
                        }
                    }
                    if (lane == 0) umma_commit((role == 0 ? bar_s : bar_o) + 8 * u);
                    __syncwarp();
                }
                // on a time-out, what is in flight ends before the memory goes
                // away: a last commit completes behind all of this warp's products
                if (__any_sync(0xffffffffu, stalled)) {
                    stalled = true;
                    if (lane == 0) {
                        atomicOr(p.status, kStatusPipelineStall);
                        umma_commit(bar_x + 8 * (role >> 1));
                        (void)mbar_wait_bounded(bar_x + 8 * (role >> 1), 0);
                    }
                }
            } else if (role == 1 && lane == 0) {
                int sent = 0;
#pragma unroll 1
                for (int n = 0; n < s.ntiles; ++n, ++sent) {   // K records (fp16 K: MMA tiles)
                    const int t = tbase + n, tok0 = (s.k0 + n) * kTok;
                    const uint32_t bar = bar_k + 8 * (t & 1);
                    if constexpr (KB == 0) {
                        if (t >= 2) wait(bar_s + 8 * (t & 1), ((t >> 1) - 1) & 1);   // S(t - 2) has read its K tile
                        if (stalled) break;
                        const uint32_t dst = smem_u32(smem + C::kKOff + (t & 1) * 32768);
                        mbar_arrive_expect_tx(bar, 32768);
#pragma unroll 1
                        for (int q = 0; q < 8; ++q)
                            tma_g2s_2d(dst + q * 4096, &kmap, (q >> 2) * 64,
                                       static_cast<int32_t>(s.row0 + tok0 + (q & 3) * 32), bar);
                    } else {
                        if (t >= 2) wait(bar_kr + 8 * (t & 1), ((t >> 1) - 1) & 1);   // the records of tile t - 2 are read
                        if (stalled) break;
                        const uint32_t bytes = min(kTok, s.t_lim - tok0) * C::kRbK;
                        fence_proxy_async();
                        mbar_arrive_expect_tx(bar, bytes);
                        bulk_g2s(smem_u32(smem + C::kSKOff + (t & 1) * C::kSK), p.k_codes + (s.row0 + tok0) * C::kRbK, bytes,
                                 bar);
                    }
                }
                if (stalled) {   // the copies in flight land first
                    for (int n = max(0, sent - 2); n < sent; ++n)
                        (void)mbar_wait_bounded(bar_k + 8 * ((tbase + n) & 1), ((tbase + n) >> 1) & 1);
                }
            } else if (role == 2 && lane == 0) {
                int sent = 0;
#pragma unroll 1
                for (int n = 0; n < s.ntiles; ++n, ++sent) {   // V records
                    const int t = tbase + n, tok0 = (s.k0 + n) * kTok;
                    if (t >= 2) wait(bar_vr + 8 * (t & 1), ((t >> 1) - 1) & 1);
                    if (stalled) break;
                    const uint32_t bytes = min(kTok, s.t_lim - tok0) * C::kRbV, bar = bar_v + 8 * (t & 1);
                    fence_proxy_async();
                    mbar_arrive_expect_tx(bar, bytes);
                    bulk_g2s(smem_u32(smem + C::kSVOff + (t & 1) * C::kSV), p.v_codes + (s.row0 + tok0) * C::kRbV, bytes,
                             bar);
                }
                if (stalled)
                    for (int n = max(0, sent - 2); n < sent; ++n)
                        (void)mbar_wait_bounded(bar_v + 8 * ((tbase + n) & 1), ((tbase + n) >> 1) & 1);
            }
            __syncwarp();
            bad = end_segment(s.ntiles);
        }
    } else if (wg >= 2) {
        // ---- dequantising warps: K(n) (quantized K) with both norms of the tile's
        // tokens, one per thread, and V(n)^T ----
        regs_dec<kRegsDequant>();
        const int r = tid & 127;
        bool bad = false;
        while (pos < hi && !bad) {
            const Segment s = segment();
            // the tile's scales and norms, a token per thread: by the warps that have less
            // to do (raw halves, a tile ahead, converted where they are used)
            __half nk = __ushort_as_half(0), nv = nk;
            auto load_norms = [&](int n) {   // (0 past the end)
                const int t = (s.k0 + n) * kTok + r;
                const bool in = n < s.ntiles && t < s.t_lim;
                if constexpr (KB != 0) nk = in ? p.k_norm[s.row0 + t] : __ushort_as_half(0);
                nv = in ? p.v_norm[s.row0 + t] : __ushort_as_half(0);
            };
            auto store_norms = [&](int n) {
                const int t = tbase + n, u = t & 1;
                if (t >= 2) wait(bar_p + 8 * u, ((t >> 1) - 1) & 1);   // softmax(t - 2) has read its own
                if constexpr (KB != 0)
                    (reinterpret_cast<float*>(smem + C::kColOff) + u * kTok)[frag_place(r)] =
                        __half2float(nk) * p.scale_log2e;
                const float x = __half2float(nv);
                // (an infinite or NaN norm counts as +-65504: 0 * inf would be NaN in
                // the rows that do not see the token; it does not count for the
                // slack, so the rows that do may overflow)
                (reinterpret_cast<float*>(smem + C::kNvOff) + u * kTok)[frag_place(r)] =
                    fmaxf(fminf(x, 65504.f), -65504.f);
                // (non-negative floats order like their bits)
                const uint32_t nmax = __reduce_max_sync(0xffffffffu, fabsf(x) < 65536.f ? __float_as_uint(fabsf(x)) : 0u);
                if (lane == 0) (reinterpret_cast<uint32_t*>(smem + C::kNmOff) + 4 * u)[warp & 3] = nmax;
                mbar_arrive(bar_n + 8 * u);
                load_norms(n + 1);
            };
            if (wg == 2) {
                if constexpr (KB == 0) load_norms(0);
#pragma unroll 1
                for (int n = 0; n < s.ntiles; ++n) {
                    if constexpr (KB == 0) {
                        store_norms(n);
                        continue;
                    }
                    const int t = tbase + n, u = t & 1;
                    wait(bar_k + 8 * u, (t >> 1) & 1);
                    if (t >= 2) wait(bar_s + 8 * u, ((t >> 1) - 1) & 1);   // S(t - 2) has read its K tile
                    // a token per thread; the quarters are taken in an order that
                    // differs between lanes whose records start in the same banks
                    const Tables kt{p.ktab[0], p.ktab[1], p.ktab[2], p.ktab[3]};
                    const uint8_t* rec = smem + C::kSKOff + u * C::kSK + r * C::kRbK;
                    uint8_t* sK = smem + C::kKOff + u * 32768;
                    const int turn = KB == 4 ? r >> 1 : r >> 3;
                    // (rolled: unrolled by two the CTA's warps took 150 us at 64 nodes, 8
                    // sequences of 24,000 tokens, so 142: what the instruction caches hold)
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        const int quarter = (q + turn) & 3;
                        uint32_t hh[16];
                        dequant_q32<(KB == 0 ? 4 : KB)>(rec + quarter * (C::kRbK / 4), kt, hh);
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            *reinterpret_cast<uint4*>(sK + sw128_offset(r, 32 * quarter + 8 * m)) =
                                make_uint4(hh[4 * m], hh[4 * m + 1], hh[4 * m + 2], hh[4 * m + 3]);
                    }
                    fence_proxy_async();
                    mbar_arrive(bar_kr + 8 * u);
                }
            } else {
                const Tables vt{p.vtab[0], p.vtab[1], p.vtab[2], p.vtab[3]};
                if constexpr (KB != 0) load_norms(0);
#pragma unroll 1
                for (int n = 0; n < s.ntiles; ++n) {
                    const int t = tbase + n, u = t & 1;
                    if constexpr (KB != 0) store_norms(n);
                    wait(bar_v + 8 * u, (t >> 1) & 1);
                    if (t >= 2) wait(bar_o + 8 * u, ((t >> 1) - 1) & 1);   // P.V(t - 2) has read its V tile
                    store_vt<VB>(smem + C::kSVOff + u * C::kSV, smem + C::kVtOff + u * 32768, vt, warp & 3, lane);
                    fence_proxy_async();
                    mbar_arrive(bar_vr + 8 * u);
                }
            }
            bad = end_segment(s.ntiles);
        }
    } else {
        // ---- softmax warps: warp w has rows 32 (w & 3) + 16 (w >> 2) .. + 15 as MMA
        // fragments: lane 4v + c has rows v and v + 8 and columns 2c, 2c + 1 of every
        // eight, so a thread reads a quarter of the tile's scales and norms (with a row
        // per thread, their broadcast reads took a third of the shared-memory bandwidth
        // that the MMAs need) ----
        regs_inc<kRegsSoftmax>();
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const int c4 = 4 * (lane & 3);   // this thread's place in a tile's scales and norms
        bool bad = false;
        while (pos < hi && !bad) {
            const Segment s = segment();
            const int base = s.L - p.tq;                   // first drafted token
            const int full_below = min(base, s.t_lim);     // tokens below this are seen by every row
            const int row32 = (s.ui % p.row_tiles) * kTreeRows + 32 * quad;
            const int row16 = row32 + 16 * half;           // this warp's first row
            const bool live = row16 < p.rows;
            const uint32_t* mask = p.tree + static_cast<size_t>(s.b) * p.tree_per_seq;
            // Q' of the unit into tensor memory: lane = row, q_hi by the first four
            // warps, q_lo by the others
            if (segs == 0) griddep_wait();
            if (KB != 0 || half == 0) {
                const uint4* q16 = reinterpret_cast<const uint4*>(
                                       p.q_tiles + static_cast<size_t>(s.b * p.per_b + s.ui) * (KB == 0 ? 32768 : 65536) +
                                       half * 32768) + 32 * quad + lane;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t w[32];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint4 x = __ldcg(q16 + (8 * c + e) * kTreeRows);
                        w[4 * e] = x.x, w[4 * e + 1] = x.y, w[4 * e + 2] = x.z, w[4 * e + 3] = x.w;
                    }
                    tmem_st32(tm_q + lanes + 64 * half + 32 * c, w);
                }
            }
            tc_fence_before();
            mbar_arrive(bar_q);
            float m_base[2], l_sum[2];   // base (log2) and this thread's part of the sum of rows v + 8q
            const uint32_t* mrow[2];     // and their masks
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                m_base[q] = -INFINITY, l_sum[q] = 0.f;
                const int rr = row16 + (lane >> 2) + 8 * q;
                mrow[q] = rr < p.rows ? mask + (rr / p.group) * p.tree_words : nullptr;
            }
#pragma unroll 1
            for (int n = 0; n < s.ntiles; ++n) {
                const int t = tbase + n, u = t & 1;
                const int tok0 = (s.k0 + n) * kTok;
                wait(bar_n + 8 * u, (t >> 1) & 1);                     // scales and norms
                if (t >= 2) wait(bar_o + 8 * u, ((t >> 1) - 1) & 1);   // P.V(t - 2) has read its P
                wait(bar_s + 8 * u, (t >> 1) & 1);
                tc_fence_after();
                if (live) {   // (warp-uniform)
                    const uint32_t t_s = tmem + 128 * u + lanes + (static_cast<uint32_t>(16 * half) << 16);
                    const float* col = reinterpret_cast<const float*>(smem + C::kColOff) + u * kTok + c4;
                    const float* nvs = reinterpret_cast<const float*>(smem + C::kNvOff) + u * kTok + c4;
                    // how far a score may pass its row's base: p n_v stays below 2^15 (from the
                    // largest norm's exponent, -24 at least), and how far the largest one does
                    // where the base moves
                    const uint4 nm = *reinterpret_cast<const uint4*>(smem + C::kNmOff + 16 * u);
                    const int spare = 14 + 127 - static_cast<int>(max(max(nm.x, nm.y), max(nm.z, nm.w)) >> 23);
                    const int slack_i = max(0, min(14 + 24, spare));
                    const float slack = static_cast<float>(slack_i), most = __int_as_float((slack_i + 127) << 23);
                    // stmatrix: lane 8m + k gives row k of matrix m: rows 0-7 and 8-15 of
                    // eight tokens, then of the next eight
                    const uint32_t prow =
                        smem_u32(smem + C::kPOff + u * 32768) + (32 * quad + 16 * half + (lane & 15)) * 128;
                    const bool masked = tok0 + kTok > full_below;   // some row sees the tile in part
                    float2 nb[2], sum[2];
                    auto scale4 = [&](int c) {
                        if constexpr (KB != 0) return *reinterpret_cast<const float4*>(col + 16 * c);
                        return make_float4(p.scale_log2e, p.scale_log2e, p.scale_log2e, p.scale_log2e);
                    };
                    auto norm4 = [&](int c) { return *reinterpret_cast<const float4*>(nvs + 16 * c); };
                    // x of columns 16c .. 16c + 15 from S, x[2i + q], and P from x
                    auto scores = [&](const float4& s4, const uint32_t* v, float2 (&x)[4]) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = e >> 1, q = e & 1;
                            x[e] = __ffma2_rn(make_float2(__uint_as_float(v[4 * i + 2 * q]), __uint_as_float(v[4 * i + 2 * q + 1])),
                                              i ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y), nb[q]);
                        }
                    };
                    auto hide = [&](int c, float2 (&x)[4]) {   // tokens that a row does not see
                        const int t0 = tok0 + 16 * c;
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t w = 0u;
                            if (mrow[q] != nullptr && t0 < s.t_lim) {
                                w = tree_window(mrow[q], p.tree_words, t0 - base);
                                if (t0 + 16 > s.t_lim) w &= (1u << (s.t_lim - t0)) - 1u;
                            }
                            w >>= 2 * (lane & 3);   // this thread's columns: bits 0, 1, 8, 9
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                if (!((w >> (8 * i)) & 1u)) x[2 * i + q].x = -INFINITY;
                                if (!((w >> (8 * i)) & 2u)) x[2 * i + q].y = -INFINITY;
                            }
                        }
                    };
                    auto weigh = [&](int c, const float4& w4, const float2 (&x)[4]) {
                        uint32_t pk[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int q = e & 1;
                            const float2 pe = make_float2(fast_exp2(x[e].x), fast_exp2(x[e].y));
                            sum[q] = __fadd2_rn(sum[q], pe);
                            const float2 w = __fmul2_rn(pe, e >> 1 ? make_float2(w4.z, w4.w) : make_float2(w4.x, w4.y));
                            pk[e] = pack_half2(w.x, w.y);
                        }
                        stsm_x4(prow + (c >> 2) * 16384 + (((2 * (c & 3) + (lane >> 4)) ^ (lane & 7)) << 4), pk[0], pk[1],
                                pk[2], pk[3]);
                    };
                    auto set_base = [&]() {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const float b0 = m_base[q] == -INFINITY ? 0.f : -m_base[q];
                            nb[q] = make_float2(b0, b0);
                            sum[q] = make_float2(0.f, 0.f);
                        }
                    };
                    // P against the rows' bases.  A score that passes its base by more
                    // than the slack shows in the thread's sum (which may also pass
                    // 2^slack without one); then, and on a row's first tile, the bases
                    // move to the tile's maxima before (another) pass.
                    bool move = __any_sync(0xffffffffu, m_base[0] == -INFINITY || m_base[1] == -INFINITY);
#pragma unroll 1
                    for (;;) {
                        set_base();
                        if (move) {
                            float mq[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
                            for (int c = 0; c < 8; ++c) {
                                uint32_t v[8];
                                tmem_ld_frag_issue(t_s + 16 * c, v);
                                tmem_ld_wait(v);
                                float2 x[4];
                                scores(scale4(c), v, x);
                                if (masked) hide(c, x);
#pragma unroll
                                for (int e = 0; e < 4; ++e) mq[e & 1] = fmaxf(mq[e & 1], fmaxf(x[e].x, x[e].y));
                            }
                            float alpha[2];
                            bool grow = false;
#pragma unroll
                            for (int q = 0; q < 2; ++q) {   // the row's maximum is spread over its four lanes
                                float mx = fmaxf(mq[q], __shfl_xor_sync(0xffffffffu, mq[q], 1));
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                                const bool fresh = m_base[q] == -INFINITY;
                                const bool up = mx > (fresh ? -INFINITY : slack);
                                mx -= fmaxf(0.f, slack - kMargin);   // (what the base moves by)
                                alpha[q] = up ? (fresh ? 0.f : fast_exp2(-mx)) : 1.f;
                                l_sum[q] *= alpha[q];
                                if (up) m_base[q] = (fresh ? 0.f : m_base[q]) + mx;
                                grow |= up;
                            }
                            if (n > 0 && __any_sync(0xffffffffu, grow)) {   // rescale the rows of O
                                wait(bar_o + 8 * (1 - u), ((t - 1) >> 1) & 1);   // P.V(t - 1) is done
                                tc_fence_after();
                                const uint32_t t_or = tm_o + lanes + (static_cast<uint32_t>(16 * half) << 16);
#pragma unroll 1
                                for (int c = 0; c < 8; ++c) {
                                    uint32_t o[8];
                                    tmem_ld_frag_issue(t_or + 16 * c, o);
                                    tmem_ld_wait(o);
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha[(e >> 1) & 1]);
                                    tmem_st_frag256(t_or + 16 * c, o);
                                }
                                tmem_st_wait();
                            }
                            set_base();
                        }
                        if (!masked) {
                            uint32_t v[2][32];   // 64 columns each
                            tmem_ld_frag_issue(t_s, v[0]);
                            float4 s4 = scale4(0), w4 = norm4(0);
                            tmem_ld_wait(v[0]);
                            tmem_ld_frag_issue(t_s + 64, v[1]);
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const float4 sn = scale4((c + 1) & 7), wn = norm4((c + 1) & 7);   // of the next columns
                                if (c == 4) tmem_ld_wait(v[1]);
                                float2 x[4];
                                scores(s4, v[c >> 2] + 8 * (c & 3), x);
                                weigh(c, w4, x);
                                s4 = sn;
                                w4 = wn;
                            }
                        } else {
#pragma unroll 1
                            for (int c = 0; c < 8; ++c) {
                                uint32_t v[8];
                                tmem_ld_frag_issue(t_s + 16 * c, v);
                                tmem_ld_wait(v);
                                float2 x[4];
                                scores(scale4(c), v, x);
                                hide(c, x);
                                weigh(c, norm4(c), x);
                            }
                        }
                        const float s0 = sum[0].x + sum[0].y, s1 = sum[1].x + sum[1].y;
                        if (move || !__any_sync(0xffffffffu, fmaxf(s0, s1) > most)) {
                            l_sum[0] += s0;
                            l_sum[1] += s1;
                            break;
                        }
                        move = true;
                    }
                    fence_proxy_async();   // the MMA reads P through the async proxy
                }
                tc_fence_before();
                mbar_arrive(bar_p + 8 * u);   // P(t) is stored, S(t), the scales and norms are read
            }

            // ---- write the unit's partial: each warp its rows' 64 columns through
            // shared memory (over the V^T tiles; 16-byte pieces XORed with the row),
            // then a row at a time, 512 bytes together ----
            const int tl = tbase + s.ntiles - 1;
            wait(bar_o + 8 * (tl & 1), (tl >> 1) & 1);
            tc_fence_after();
            if (pos + s.ntiles >= hi || stalled) griddep_launch_dependents();   // last segment: let the merge launch
            const int late = named_bar_or(5, 256, stalled);                  // (both V^T tiles are free)
            if (row32 < p.rows && !late) {
                float2* sml = reinterpret_cast<float2*>(smem + C::kColOff) + 32 * quad;   // (the scales and norms are read)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float l = l_sum[q] + __shfl_xor_sync(0xffffffffu, l_sum[q], 1);
                    l += __shfl_xor_sync(0xffffffffu, l, 2);
                    if ((lane & 3) == 0) sml[16 * half + (lane >> 2) + 8 * q] = make_float2(m_base[q], l);
                }
                const int r = 32 * quad + lane;
                uint8_t* xo = smem + C::kVtOff + r * 512;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t v[32];
                    tmem_ld32(tm_o + lanes + 64 * half + 32 * c, v);
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4*>(xo + (((16 * half + 8 * c + e / 4) ^ lane) << 4)) =
                            make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
                named_bar_sync(1 + quad, 64);
                const size_t slot_row = (static_cast<size_t>(c_me) + s.b * p.per_b + s.ui) * kTreeRows + 32 * quad;
                // dims 4 lane .. + 3 lie in columns pi(d): pairs flipped by the 32-dim
                // block lane >> 3
                const int c0 = (4 * lane) ^ (2 * (lane >> 3)), c1 = (4 * lane + 2) ^ (2 * (lane >> 3));
                const int nrows = min(32, p.rows - row32);
#pragma unroll 4
                for (int row = half; row < nrows; row += 2) {
                    const uint8_t* src = smem + C::kVtOff + (32 * quad + row) * 512;
                    const float2 a = *reinterpret_cast<const float2*>(src + (((c0 >> 2) ^ row) << 4) + (c0 & 2) * 4);
                    const float2 b = *reinterpret_cast<const float2*>(src + (((c1 >> 2) ^ row) << 4) + (c1 & 2) * 4);
                    reinterpret_cast<float4*>(p.part_o + (slot_row + row) * kD)[lane] = make_float4(a.x, a.y, b.x, b.y);
                }
                if (half == 0 && lane < nrows)
                    reinterpret_cast<float2*>(p.part_ml)[slot_row + lane] = sml[lane];
            }
            bad = end_segment(s.ntiles);   // everything is free for the next segment
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// A warp per output row: merge the partials of the CTAs over the row's unit by
// their log-sum-exp weights, four or eight at a time, apply v_rescale / l, leave the
// rotated basis and store fp16.  Rows of one unit read neighbouring partials.
__global__ void __launch_bounds__(256) tq_tree_combine_kernel(const __grid_constant__ TreeParams p) {
    const int lane = threadIdx.x & 31;
    const int row = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5);   // (b, kv head, node, head of the group)
    const int per_unit = p.rows;
    const int bh = row / per_unit, rr = row - bh * per_unit;
    const int b = bh / p.hkv, h = bh - b * p.hkv;
    if (b >= p.batch) return;
    const int rt = rr / kTreeRows, r = rr - rt * kTreeRows;
    const int ui = h * p.row_tiles + rt, unit = b * p.per_b + ui;
    // (`lengths` may be read before the dependency wait: the split kernel's CTAs
    // waited for the work that wrote it before any let this grid launch)
    int before = 0, all = 0;
    for (int bb = lane; bb < p.batch; bb += 32) {
        const int v = tree_chunks(p.lengths[bb], p.max_len) * p.per_b;
        all += v;
        if (bb < b) before += v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    const int nch = tree_chunks(p.lengths[b], p.max_len);
    const int P = p.num_ctas;
    int c0 = 0, n = 0;
    if (nch > 0) {
        const long long first = before + static_cast<long long>(ui) * nch;
        c0 = static_cast<int>(((first + 1) * P - 1) / all);
        n = static_cast<int>(((first + nch) * P - 1) / all) - c0 + 1;
    }
    auto has = [&](int i) {   // whether CTA c0 + i had chunks at all (where every one had, without the divisions)
        const long long c = c0 + i;
        return i < n && (all >= P || c * all / P < (c + 1) * all / P);
    };
    const size_t row0 = (static_cast<size_t>(c0) + unit) * kTreeRows + r;
    griddep_wait();
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    bool nan = false;   // a partial's sum is NaN (its base is -inf where all its scores were): so is the row
    auto merge = [&](auto ahead) {   // with so many partials in flight
        constexpr int kAhead = decltype(ahead)::value;
        for (int i0 = 0; i0 < n; i0 += kAhead) {
            float2 ml[kAhead];
            float4 o[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const bool u = has(i0 + k);
                const size_t at = row0 + static_cast<size_t>(i0 + k) * kTreeRows;
                ml[k] = u ? __ldcg(reinterpret_cast<const float2*>(p.part_ml) + at) : make_float2(-INFINITY, 0.f);
                o[k] = u ? __ldcg(reinterpret_cast<const float4*>(p.part_o + at * kD) + lane)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float Mn = M;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                Mn = fmaxf(Mn, ml[k].x);
                nan = nan || ml[k].y != ml[k].y;
            }
            if (Mn == -INFINITY) continue;
            const float sc = M == -INFINITY ? 0.f : fast_exp2(M - Mn);
            acc.x *= sc; acc.y *= sc; acc.z *= sc; acc.w *= sc;
            den *= sc;
            M = Mn;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (ml[k].x == -INFINITY) continue;
                const float w = fast_exp2(ml[k].x - M);
                den += w * ml[k].y;
                acc.x += w * o[k].x; acc.y += w * o[k].y;
                acc.z += w * o[k].z; acc.w += w * o[k].w;
            }
        }
    };
    // (32 partials a row, 112 rows of one sequence of 8,192 tokens and 4 KV heads: 17.1 us
    // with eight in flight, 18.2 with four; two or three a row: no difference)
    if (n > 4) merge(std::integral_constant<int, 8>{});
    else merge(std::integral_constant<int, 4>{});
    float inv = 0.f;
    if (nan) inv = __int_as_float(0x7fffffff);
    else if (den > 0.f) inv = p.v_rescale / den;
    else if (lane == 0) atomicOr(p.status, kStatusShortContext);
    float v[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
    wht128_lane4(v, lane);
    const uint32_t sn = sign_nibble(p.signs, lane);
    const float nrm = 0.08838834764831845f;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ((sn >> i) & 1u) ? -v[i] * nrm : v[i] * nrm;
    const int j = rr / p.group, hl = rr - j * p.group;
    __half* op = p.out + ((static_cast<size_t>(b) * p.hq + h * p.group + hl) * p.tq + j) * kD + lane * 4;
    *reinterpret_cast<uint2*>(op) = make_uint2(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]));
}

template <int KB, int VB>
static int launch_tree_t(const TreeParams& p, const CUtensorMap* kmap, cudaStream_t stream, cudaEvent_t ev0,
                         cudaEvent_t ev1) {
    using C = TreeCfg<KB, VB>;
    static std::atomic<uint64_t> attr_done{0};
    cudaError_t e = set_smem_attr_once(tq_tree_kernel<KB, VB>, C::kSmemAlloc, attr_done, -1, kRegsLaunch);
    if (e != cudaSuccess) return e;
    if (ev0) cudaEventRecord(ev0, stream);
    e = launch_pdl(tq_tree_q_kernel<KB != 0>, dim3(p.batch * p.per_b * (kTreeRows / 8)), dim3(256), 0, stream, p);
    if (e != cudaSuccess) return e;
    e = launch_pdl(tq_tree_kernel<KB, VB>, dim3(p.num_ctas), dim3(kTreeThreads), C::kSmemAlloc, stream, p, *kmap);
    if (ev1) cudaEventRecord(ev1, stream);
    if (e != cudaSuccess) return e;
    const long long rows = 1ll * p.batch * p.hkv * p.rows;
    return launch_pdl(tq_tree_combine_kernel, dim3(static_cast<unsigned int>((rows + 7) / 8)), dim3(256), 0, stream, p);
}

int launch_tree(int kbits, int vbits, const TreeParams& p, const CUtensorMap* kmap, cudaStream_t stream,
                cudaEvent_t ev0, cudaEvent_t ev1) {
    if (kbits == 16 && vbits == 4) return launch_tree_t<0, 4>(p, kmap, stream, ev0, ev1);
    if (kbits == 16 && vbits == 3) return launch_tree_t<0, 3>(p, kmap, stream, ev0, ev1);
    if (kbits == 3 && vbits == 3) return launch_tree_t<3, 3>(p, kmap, stream, ev0, ev1);
    if (kbits == 4 && vbits == 4) return launch_tree_t<4, 4>(p, kmap, stream, ev0, ev1);
    if (kbits == 4 && vbits == 3) return launch_tree_t<4, 3>(p, kmap, stream, ev0, ev1);
    return cudaErrorInvalidValue;
}

}  // namespace tq
