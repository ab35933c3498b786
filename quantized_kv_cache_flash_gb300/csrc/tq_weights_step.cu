// tq_attention_weights for few rows per KV head (a decode step): up to 16.
//
// Two kernels.  The first is the decode kernel's K half: CTAs with equal shares of all
// units' 32-token chunks, their warps streaming chunks through private rings of bulk
// copies, dequantising in registers, scores by warp MMAs with 16 tokens as M.  It writes
// the scores (fp32, log2 units) to the workspace and a (maximum, sum of exp2) per row and
// share.  A thread keeps its own tokens' maximum and sum of each of its rows, so no lane
// waits for another until the share ends.  The second joins a unit's shares to the rows'
// log-sum-exp and turns the scores into the tokens' weights, a token a thread.  (Scores
// of 4 to 8 rows are 16 to 32 bytes a token, mostly served by L2; reading K once more
// would be 48 to 256 and another dequantisation.)
//
// Where a cluster of 16 CTAs per unit fits the GPU at once (few units), one kernel does
// both: the scores stay in shared memory, and the CTAs of a cluster exchange their
// (maximum, sum) pairs there.
//
// 32 sequences of 4,000 to 16,384 tokens, 32/8 heads, turbo4: 66 us, the scores 52 (K's 193 MB
// would take 28), the sums 15 (scores and weights through L2).  Nothing is full in the scores
// kernel: issue 0.57, the integer pipe 0.58, DRAM 0.47; its warps wait for the integer pipe
// (1.5 cycles an instruction), for their turn (1.7) and for results (1.0) more than for memory
// (0.7).  One sequence of 8,177, 28/4 heads, turbo3: 7.6 us in a graph (launch, one trip to
// memory, two cluster barriers); 5 with fp16 K: 18 (50 MB, 7.4).
// 64 units of 10,000 tokens with 4, 8, 16 rows: 30, 36, 45 us (turbo4; fp16 K 49, 50, 61); the kernel
// for blocks of queries, which reads K twice, takes 75 with 20 rows (fp16 K 73).
#include <cooperative_groups.h>

#include <algorithm>

#include "tq_decode_kernel.cuh"

namespace tq {

namespace cg = cooperative_groups;

constexpr int kStepCluster = 16;   // CTAs per unit of the one-kernel form
constexpr int kStepOneTokens = 1024;   // tokens of such a CTA, at most

template <int KB, int ROWS>
struct StepCfg {
    static constexpr int kWarps = 4;
    static constexpr int NT = ROWS == 16 ? 2 : 1;           // 8-column MMA n-tiles
    static constexpr bool kPair = KB != 0 && ROWS == 4;     // column 2i: q_hi of row i, 2i + 1: q_lo
    static constexpr bool kQlo = KB != 0 && ROWS != 4;      // q_lo as a second B operand
    static constexpr int NE = kPair ? 1 : 2;                // query rows per thread per n-tile
    static constexpr int kTok = KB == 0 ? 32 : 64;          // tokens per stage
    static constexpr int kStages = 2;
    static constexpr int kMinCtas = KB == 0 ? 3 : NT == 2 ? 4 : 6;   // resident CTAs per SM, at least
    static constexpr int kRbK = KB == 0 ? 256 : KB * 16;
    static constexpr int kKnOff = kTok * kRbK;
    static constexpr int kStageRaw = kKnOff + (KB == 0 ? 0 : kTok * 2);
    static constexpr int kStageAlign = KB == 0 ? 1024 : 128;
    static constexpr int kStage = (kStageRaw + kStageAlign - 1) / kStageAlign * kStageAlign;
    static constexpr int kPipe = kWarps * kStages * kStage;
    static constexpr int kQStride = kD + 8;                 // (16-byte pads: columns on different banks)
    static constexpr int kQOff = kPipe;
    static constexpr int kQloOff = kQOff + 8 * NT * kQStride * 2;
    static constexpr int kBarOff = kQloOff + (kQlo ? 8 * NT * kQStride * 2 : 0);
    static constexpr int kScanOff = (kBarOff + kWarps * kStages * 8 + 15) / 16 * 16;
    static constexpr int kMlOff = kScanOff + 512;           // (m, l) of the warps' rows
    static constexpr int kSmem = kMlOff + kWarps * ROWS * 8;
    static constexpr int kPad = KB == 0 ? 1024 : 128;       // to a boundary of as much
    static constexpr int kSmemAlloc = kSmem + kPad;
    // one-kernel form: the cluster's (m, l) pairs, the rows' log-sum-exp, the scores
    static constexpr int kPartOff = (kSmem + 15) / 16 * 16;
    static constexpr int kLseOff = kPartOff + kStepCluster * ROWS * 8;
    static constexpr int kScoreOff = kLseOff + ROWS * 4;
    static constexpr int kOneAlloc(int tokens) { return kScoreOff + tokens * ROWS * 4 + kPad; }

    __device__ static __forceinline__ int slot_row(int n, int e, int t) { return kPair ? t : 8 * n + 2 * t + e; }
};

// (m, l) += a part whose maximum is mb and sum lb.
__device__ __forceinline__ void join(float& m, float& l, float mb, float lb) {
    const float mn = fmaxf(m, mb);
    l = (m == -INFINITY ? l : l * fast_exp2(m - mn)) + (mb == -INFINITY ? lb : lb * fast_exp2(mb - mn));
    m = mn;
}

// Rows whose normaliser is NaN are NaN on every token that they see (the first query's last
// one: `last`), also where the score is -inf: NaN if there is one for this token, else 0.
template <int ROWS>
__device__ __noinline__ float nan_rows(const float* lse, int tok, int last, int group) {
    float w = 0.f;
#pragma unroll 1
    for (int r = 0; r < ROWS; ++r)
        if (lse[r] != lse[r] && tok <= last + r / group) w = lse[r];
    return w;
}

// ONE: the one-kernel form.
template <int KB, int ROWS, bool ONE>
__global__ void __launch_bounds__(128, ONE ? 2 : StepCfg<KB, ROWS>::kMinCtas)
    tq_step_scores_kernel(const __grid_constant__ StepParams p, const __grid_constant__ CUtensorMap kmap) {
    using C = StepCfg<KB, ROWS>;
    constexpr int NT = C::NT, NE = C::NE;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & (C::kPad - 1u));
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    uint8_t* wpipe = smem + warp * C::kStages * C::kStage;
    const uint32_t bar0 = smem_u32(smem + C::kBarOff) + warp * C::kStages * 8;
    if (lane == 0) {
        for (int s = 0; s < C::kStages; ++s) mbar_init(bar0 + 8 * s, 1);
        fence_barrier_init();
    }
    if (KB == 0 && threadIdx.x == 0) prefetch_tensormap(&kmap);
    __syncwarp();
    if constexpr (ONE) cluster_arrive();   // (met before the pairs are exchanged: all CTAs run)

    griddep_wait();
    BatchScan scan;
    int lo = 0, hi = 1;   // (ONE: a single share)
    if constexpr (!ONE) {
        scan.s = reinterpret_cast<int*>(smem + C::kScanOff);   // (the same for all warps)
        if (warp == 0) scan.init(scan.s, p.lengths, p.batch, p.hkv, p.max_len, lane);
        __syncthreads();
        const int all = __shfl_sync(0xffffffffu, scan.total(p.lengths, p.batch, p.hkv, p.max_len, lane), 0);
        const int P = static_cast<int>(gridDim.x), c_me = static_cast<int>(blockIdx.x);
        const int cq = all / P, cr = all - cq * P;
        lo = c_me * cq + (c_me * cr) / P;
        hi = (c_me + 1) * cq + ((c_me + 1) * cr) / P;
        if (lo >= hi) return;   // (uniform over the CTA)
    }
    __half* sQ = reinterpret_cast<__half*>(smem + C::kQOff);
    __half* sQlo = reinterpret_cast<__half*>(smem + C::kQloOff);
    const uint32_t q_lds = smem_u32(sQ) + ((lane & 7) * C::kQStride + 8 * (lane >> 3)) * 2;
    const uint32_t qlo_lds = smem_u32(sQlo) + ((lane & 7) * C::kQStride + 8 * (lane >> 3)) * 2;
    const Tables kt{p.ktab[0], p.ktab[1], p.ktab[2], p.ktab[3]};
    float2* sML = reinterpret_cast<float2*>(smem + C::kMlOff);

    int stage = 0;
    uint32_t phase = 0;
    int pos = lo;
    while (pos < hi) {
        int b, h, L, k0, k1;   // tokens of chunks [k0, k1) of unit (b, h)
        if constexpr (ONE) {
            const int u = static_cast<int>(blockIdx.x) / kStepCluster, rank = static_cast<int>(blockIdx.x) % kStepCluster;
            b = u / p.hkv;
            h = u - b * p.hkv;
            L = p.lengths[b];
            const int nch = unit_chunks(p.lengths, b, p.max_len);
            k0 = rank * nch / kStepCluster;
            k1 = (rank + 1) * nch / kStepCluster;
        } else {
            int before, nch;
            scan.locate(p.lengths, p.batch, p.hkv, p.max_len, pos, lane, b, before, L, nch);
            b = __shfl_sync(0xffffffffu, b, 0);
            before = __shfl_sync(0xffffffffu, before, 0);
            L = __shfl_sync(0xffffffffu, L, 0);
            nch = __shfl_sync(0xffffffffu, nch, 0);
            h = (pos - before) / nch;
            k0 = pos - before - h * nch;
            k1 = min(nch, k0 + (hi - pos));
        }
        const int unit = b * p.hkv + h;
        const int t_begin = k0 * kChunkTokens, t_end = min(k1 * kChunkTokens, min(L, p.max_len));
        const int nchunks = (t_end - t_begin + C::kTok - 1) / C::kTok;   // stages' worth of tokens
        const size_t row0 = static_cast<size_t>(unit) * p.cap;

        auto issue = [&](int c, int st) {   // lane 0 only
            const int tok0 = t_begin + c * C::kTok;
            const int nval = min(C::kTok, t_end - tok0);
            const uint32_t dst = smem_u32(wpipe + st * C::kStage), bar = bar0 + st * 8;
            if constexpr (KB == 0) {
                mbar_arrive_expect_tx(bar, 2 * 4096);
                tma_g2s_2d(dst, &kmap, 0, static_cast<int32_t>(row0 + tok0), bar);
                tma_g2s_2d(dst + 4096, &kmap, 64, static_cast<int32_t>(row0 + tok0), bar);
            } else {
                const uint32_t nb = static_cast<uint32_t>((nval + 7) & ~7) * 2;   // norms, 16-byte multiple
                mbar_arrive_expect_tx(bar, nval * C::kRbK + nb);
                bulk_g2s(dst, p.k_codes + (row0 + tok0) * C::kRbK, nval * C::kRbK, bar);
                bulk_g2s(dst + C::kKnOff, p.k_norm + row0 + tok0, nb, bar);
            }
        };
        if (lane == 0) {
            for (int s = 0; s < C::kStages; ++s) {
                const int c = warp + C::kWarps * s;
                int si = stage + s;
                if (si >= C::kStages) si -= C::kStages;
                if (c < nchunks) issue(c, si);
            }
        }
        __syncwarp();

        // ---- the query rows -> shared, as the decode kernel lays them out ----
        for (int r = warp; r < ROWS; r += C::kWarps) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (r < p.rows) {
                const int j = r / p.group, gl = r - j * p.group;
                const uint2 raw = *reinterpret_cast<const uint2*>(
                    p.q + ((static_cast<size_t>(b) * p.hq + h * p.group + gl) * p.tq + j) * kD + lane * 4);
                const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
                const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
                v[0] = f0.x; v[1] = f0.y; v[2] = f1.x; v[3] = f1.y;
                if constexpr (KB != 0) {
                    const uint32_t sn = sign_nibble(p.signs, lane);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = ((sn >> i) & 1u) ? -v[i] : v[i];
                    wht128_lane4(v, lane);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] *= 0.08838834764831845f;   // 1/sqrt(128)
                }
            }
            const uint32_t qh0 = pack_half2(v[0], v[1]), qh1 = pack_half2(v[2], v[3]);
            if constexpr (KB != 0) {
                // k-index 16 kc + 8 hi + 2 t + e holds dim 32 t + 4 kc + 2 hi + e
                const int kk = 16 * (lane & 7) + 2 * (lane >> 3);
                __half* qrow = sQ + (C::kPair ? 2 * r : r) * C::kQStride;
                *reinterpret_cast<uint32_t*>(qrow + kk) = qh0;
                *reinterpret_cast<uint32_t*>(qrow + kk + 8) = qh1;
                const float2 h0 = __half22float2(*reinterpret_cast<const __half2*>(&qh0));
                const float2 h1 = __half22float2(*reinterpret_cast<const __half2*>(&qh1));
                __half* lrow = C::kPair ? sQ + (2 * r + 1) * C::kQStride : sQlo + r * C::kQStride;
                *reinterpret_cast<uint32_t*>(lrow + kk) = pack_half2(v[0] - h0.x, v[1] - h0.y);
                *reinterpret_cast<uint32_t*>(lrow + kk + 8) = pack_half2(v[2] - h1.x, v[3] - h1.y);
            } else {
                *reinterpret_cast<uint2*>(sQ + r * C::kQStride + 4 * lane) = make_uint2(qh0, qh1);
            }
        }
        __syncthreads();

        auto load_qb = [&](uint32_t base, int n, int kc2, uint32_t (&bq)[4]) {
            ldsm_x4(base + (8 * n * C::kQStride + 32 * kc2) * 2, bq[0], bq[1], bq[2], bq[3]);
        };
        float m[NT][NE], l[NT][NE];
        int lim[NT][NE];   // last visible token of the thread's rows
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                m[n][e] = -INFINITY;
                l[n][e] = 0.f;
                lim[n][e] = min(L - p.tq + C::slot_row(n, e, t) / p.group, t_end - 1);
            }
        // this thread's first score of the share
        float* const out = (ONE ? reinterpret_cast<float*>(smem + C::kScoreOff)
                                : p.scores + (static_cast<size_t>(unit) * p.score_len + t_begin) * ROWS) +
                           g * ROWS + C::slot_row(0, 0, t);
        const int all_see = min(L - p.tq, t_end - 1);   // (padding rows see more; nobody reads them)

        // 32 tokens of a stage from its token `at`: scores to the workspace, maxima and sums
        // in registers.  A row's base m is the largest score that the thread first sees;
        // later scores may pass it, as long as the sums stay in range.
        auto process = [&](const uint8_t* st, int tok0, int at, auto full_tag) {
            constexpr bool FULL = decltype(full_tag)::value;
            float* const o = out + static_cast<size_t>(tok0 - t_begin) * ROWS;
            tok0 += at;
            float x[2][NT][4];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
                for (int n = 0; n < NT; ++n) x[tt][n][0] = x[tt][n][1] = x[tt][n][2] = x[tt][n][3] = 0.f;
                if constexpr (KB == 0) {
                    const int mi = lane >> 3;
                    const int row = at + tt * 16 + (mi & 1) * 8 + (lane & 7);
#pragma unroll
                    for (int kc2 = 0; kc2 < 4; ++kc2) {
                        uint32_t qb[NT][4];
#pragma unroll
                        for (int n = 0; n < NT; ++n) load_qb(q_lds, n, kc2, qb[n]);
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk) {
                            const int db = 4 * kc2 + 2 * kk + (mi >> 1);
                            uint32_t a0, a1, a2, a3;
                            ldsm_x4(smem_u32(st) + (db >> 3) * 4096 + row * 128 + (((db & 7) ^ (row & 7)) << 4), a0, a1,
                                    a2, a3);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_f16(x[tt][n], a0, a1, a2, a3, qb[n][2 * kk], qb[n][2 * kk + 1]);
                        }
                    }
                } else {
                    const QuarterWords wa = load_quarter<KB>(st + (at + tt * 16 + g) * C::kRbK + t * (C::kRbK / 4));
                    const QuarterWords wb = load_quarter<KB>(st + (at + tt * 16 + g + 8) * C::kRbK + t * (C::kRbK / 4));
                    auto kgroup = [&](auto jtag) {
                        constexpr int J = decltype(jtag)::value;
                        uint32_t ha[4], hb[4], unused[2];
                        dequant_group<KB, J, false>(wa, kt, 0u, 0u, ha, unused);
                        dequant_group<KB, J, false>(wb, kt, 0u, 0u, hb, unused);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint32_t qb[4];
                            if constexpr (C::kQlo) {
                                load_qb(qlo_lds, n, J, qb);
                                mma_f16(x[tt][n], ha[0], hb[0], ha[1], hb[1], qb[0], qb[1]);
                                mma_f16(x[tt][n], ha[2], hb[2], ha[3], hb[3], qb[2], qb[3]);
                            }
                            load_qb(q_lds, n, J, qb);
                            mma_f16(x[tt][n], ha[0], hb[0], ha[1], hb[1], qb[0], qb[1]);
                            mma_f16(x[tt][n], ha[2], hb[2], ha[3], hb[3], qb[2], qb[3]);
                        }
                    };
                    kgroup(std::integral_constant<int, 0>{});
                    kgroup(std::integral_constant<int, 1>{});
                    kgroup(std::integral_constant<int, 2>{});
                    kgroup(std::integral_constant<int, 3>{});
                    if constexpr (C::kPair) {   // q_lo's column into q_hi's
                        x[tt][0][0] += x[tt][0][1];
                        x[tt][0][2] += x[tt][0][3];
                    }
                }
            }
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                const int ta = tt * 16 + g, tb = ta + 8;
                float ka = p.scale_log2e, kb2 = p.scale_log2e;
                if constexpr (KB != 0) {
                    ka *= __half2float(*reinterpret_cast<const __half*>(st + C::kKnOff + 2 * (at + ta)));
                    kb2 *= __half2float(*reinterpret_cast<const __half*>(st + C::kKnOff + 2 * (at + tb)));
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int e = 0; e < NE; ++e) {
                        x[tt][n][e] *= ka;
                        x[tt][n][e + 2] *= kb2;
                        if (!FULL) {
                            if (tok0 + ta > lim[n][e]) x[tt][n][e] = -INFINITY;
                            if (tok0 + tb > lim[n][e]) x[tt][n][e + 2] = -INFINITY;
                        }
                    }
                    float* oa = o + (at + tt * 16) * ROWS + 8 * n;
                    float* ob = oa + 8 * ROWS;
                    if constexpr (NE == 2) {
                        if (FULL || tok0 + ta < t_end) *reinterpret_cast<float2*>(oa) = make_float2(x[tt][n][0], x[tt][n][1]);
                        if (FULL || tok0 + tb < t_end) *reinterpret_cast<float2*>(ob) = make_float2(x[tt][n][2], x[tt][n][3]);
                    } else {
                        if (FULL || tok0 + ta < t_end) *oa = x[tt][n][0];
                        if (FULL || tok0 + tb < t_end) *ob = x[tt][n][2];
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    auto sum = [&](float base) {
                        return (fast_exp2(x[0][n][e] - base) + fast_exp2(x[0][n][e + 2] - base)) +
                               (fast_exp2(x[1][n][e] - base) + fast_exp2(x[1][n][e + 2] - base));
                    };
                    float s = sum(m[n][e]);
                    if (!(s < 1.2676506e30f)) {   // 2^100 (m = -inf makes it inf or NaN)
                        const float mx = fmaxf(fmaxf(x[0][n][e], x[0][n][e + 2]), fmaxf(x[1][n][e], x[1][n][e + 2]));
                        if (mx > m[n][e]) {
                            l[n][e] *= m[n][e] == -INFINITY ? 1.f : fast_exp2(m[n][e] - mx);   // (l is 0 there, or NaN)
                            m[n][e] = mx;
                        }
                        s = sum(m[n][e] == -INFINITY ? 0.f : m[n][e]);
                    }
                    l[n][e] += s;
                }
        };

        bool stalled = false;
        int c = warp;
        for (; c < nchunks; c += C::kWarps) {
            const bool ok = mbar_wait_bounded(bar0 + 8 * stage, phase);
            if (__any_sync(0xffffffffu, !ok)) { stalled = true; break; }
            const uint8_t* st = wpipe + stage * C::kStage;
            const int tok0 = t_begin + c * C::kTok;
            if (tok0 + C::kTok - 1 <= all_see) {
#pragma unroll 1
                for (int at = 0; at < C::kTok; at += 32) process(st, tok0, at, std::true_type{});
            } else {
#pragma unroll 1
                for (int at = 0; at < C::kTok && tok0 + at < t_end; at += 32) process(st, tok0, at, std::false_type{});
            }
            __syncwarp();
            const int cn = c + C::kWarps * C::kStages;
            if (cn < nchunks && lane == 0) {
                fence_proxy_async();
                issue(cn, stage);
            }
            if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
        }
        if (ONE || pos + k1 - k0 >= hi) griddep_launch_dependents();
        if (stalled) {   // this warp's copies still in flight land (bounded)
            for (int k = 0; k < C::kStages; ++k) {
                if (c + C::kWarps * k >= nchunks) break;
                (void)mbar_wait_bounded(bar0 + 8 * stage, phase);
                if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
            }
            if (lane == 0) atomicOr(p.status, kStatusPipelineStall);
        }

        // ---- the share's (m, l) of each row ----
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < NE; ++e) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    join(m[n][e], l[n][e], __shfl_xor_sync(0xffffffffu, m[n][e], o),
                         __shfl_xor_sync(0xffffffffu, l[n][e], o));
                if (g == 0) sML[warp * ROWS + C::slot_row(n, e, t)] = make_float2(m[n][e], l[n][e]);
            }
        __syncthreads();
        if (threadIdx.x < ROWS) {
            float2 a = sML[threadIdx.x];
#pragma unroll
            for (int w = 1; w < C::kWarps; ++w) {
                const float2 o = sML[w * ROWS + threadIdx.x];
                join(a.x, a.y, o.x, o.y);
            }
            if constexpr (ONE) sML[threadIdx.x] = a;
            else p.part_ml[(static_cast<size_t>(blockIdx.x) + unit) * ROWS + threadIdx.x] = a;
        }
        if constexpr (ONE) {
            // every CTA of the cluster gets all shares' pairs, joins them and weighs its tokens
            cg::cluster_group cluster = cg::this_cluster();
            float2* parts = reinterpret_cast<float2*>(smem + C::kPartOff);
            float* lse = reinterpret_cast<float*>(smem + C::kLseOff);
            __syncthreads();   // (sML; and the warps are whole again)
            cluster_wait();
            for (int i = threadIdx.x; i < kStepCluster * ROWS; i += 128) {
                const int r = i % ROWS;
                *cluster.map_shared_rank(parts + cluster.block_rank() * ROWS + r, i / ROWS) = sML[r];
            }
            cluster.sync();
            if (threadIdx.x < ROWS) {
                float am = -INFINITY, al = 0.f;
#pragma unroll
                for (int c2 = 0; c2 < kStepCluster; ++c2) {
                    const float2 v = parts[c2 * ROWS + threadIdx.x];
                    join(am, al, v.x, v.y);
                }
                // (no token is seen, or all that are score -inf)
                const bool none = am == -INFINITY && al == 0.f;
                lse[threadIdx.x] = none || threadIdx.x >= p.rows ? INFINITY : am + log2f(al);
                if (none && threadIdx.x < p.rows && cluster.block_rank() == 0) atomicOr(p.status, kStatusShortContext);
            }
            __syncthreads();
            bool any_nan = false;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) any_nan = any_nan || lse[r] != lse[r];
            const int seen = p.seen != nullptr ? p.seen[b] : L - p.tq;
            float* w_out = p.weights + static_cast<size_t>(unit) * p.cap;
            for (int tok = t_begin + threadIdx.x; tok < t_end; tok += 128) {
                const float* x = reinterpret_cast<const float*>(smem + C::kScoreOff) + (tok - t_begin) * ROWS;
                float w = 0.f;
#pragma unroll
                for (int r = 0; r < ROWS; r += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(x + r), l4 = *reinterpret_cast<const float4*>(lse + r);
                    // (-inf: hidden, or of no weight; padding rows' lse is inf)
                    w += r < p.rows && v.x != -INFINITY ? fast_exp2(v.x - l4.x) : 0.f;
                    w += r + 1 < p.rows && v.y != -INFINITY ? fast_exp2(v.y - l4.y) : 0.f;
                    w += r + 2 < p.rows && v.z != -INFINITY ? fast_exp2(v.z - l4.z) : 0.f;
                    w += r + 3 < p.rows && v.w != -INFINITY ? fast_exp2(v.w - l4.w) : 0.f;
                }
                if (any_nan) w += nan_rows<ROWS>(lse, tok, L - p.tq, p.group);
                if (p.decay != 0.f && tok < seen) w = fmaf(p.decay, w_out[tok], w);
                w_out[tok] = w;
            }
            return;
        }
        if (__syncthreads_or(stalled)) break;
        pos += k1 - k0;
    }
}

// The tokens' weights from the scores; a CTA p.span tokens of a unit, TOK a thread and turn.
template <int ROWS, int TOK>
__global__ void __launch_bounds__(256) tq_step_sums_kernel(const __grid_constant__ StepParams p) {
    __shared__ float2 s_part[16][ROWS];
    __shared__ float s_lse[ROWS];
    const int tid = threadIdx.x;
    const int per = (p.max_len + p.span - 1) / p.span;
    const int unit = static_cast<int>(blockIdx.x) / per;
    const int t0 = (static_cast<int>(blockIdx.x) - unit * per) * p.span;
    const int b = unit / p.hkv, h = unit - b * p.hkv;
    // (lengths may be read before the wait: the scores kernel's CTAs waited for what wrote
    // them before any of them let this grid launch)
    const int L = p.lengths[b], lim = min(L, p.max_len);
    // chunks of all units, and of those before this sequence
    int before = 0, all = 0;
    for (int bb = tid & 31; bb < p.batch; bb += 32) {
        const int v = unit_chunks(p.lengths, bb, p.max_len) * p.hkv;
        all += v;
        if (bb < b) before += v;
    }
    all = __reduce_add_sync(0xffffffffu, all);
    before = __reduce_add_sync(0xffffffffu, before);
    const int nch = unit_chunks(p.lengths, b, p.max_len);
    // the shares c0 .. c1 that meet the unit's chunks
    const int P = p.ctas, k_first = before + h * nch;
    int c0 = 0, c1 = -1;
    if (nch > 0) {
        if (all < 0x7fffffff / P) {   // (32-bit divisions)
            c0 = ((k_first + 1) * P - 1) / all;
            c1 = ((k_first + nch) * P - 1) / all;
        } else {
            c0 = static_cast<int>((static_cast<long long>(k_first + 1) * P - 1) / all);
            c1 = static_cast<int>((static_cast<long long>(k_first + nch) * P - 1) / all);
        }
    }
    const int cq = all / P, cr = all - cq * P;
    const int seen = p.seen != nullptr ? p.seen[b] : L - p.tq;
    griddep_wait();
    griddep_launch_dependents();
    if (t0 >= lim && t0 > 0) return;   // (uniform over the CTA)

    float x[TOK][ROWS], old[TOK];
    float* out = p.weights + static_cast<size_t>(unit) * p.cap;
    const float4* sc = reinterpret_cast<const float4*>(p.scores + static_cast<size_t>(unit) * p.score_len * ROWS);
    const int end = min(lim, t0 + p.span);
    const bool fade = p.decay != 0.f;
    auto load = [&](int t1) {
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            const int t = t1 + tid + 256 * k;
            old[k] = 0.f;
            if (t < end) {
#pragma unroll
                for (int i = 0; i < ROWS / 4; ++i) {
                    const float4 v = __ldcg(sc + static_cast<size_t>(t) * (ROWS / 4) + i);
                    x[k][4 * i] = v.x, x[k][4 * i + 1] = v.y, x[k][4 * i + 2] = v.z, x[k][4 * i + 3] = v.w;
                }
                if (fade && t < seen) old[k] = out[t];
            }
        }
    };
    load(t0);   // (in flight while the shares are joined)
    {   // thread (i, r): every 16th share of row r
        const int i = tid / 16, r = tid % 16;
        float m = -INFINITY, l = 0.f;
        if (r < ROWS)
            for (int c = c0 + i; c <= c1; c += 16) {
                if (cq == 0 && (c * cr) / P == ((c + 1) * cr) / P) continue;   // (an empty share)
                const float2 v = __ldcg(p.part_ml + (static_cast<size_t>(c) + unit) * ROWS + r);
                join(m, l, v.x, v.y);
            }
        if (r < ROWS) s_part[i][r] = make_float2(m, l);
    }
    __syncthreads();
    if (tid < ROWS) {
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) join(m, l, s_part[i][tid].x, s_part[i][tid].y);
        const bool none = m == -INFINITY && l == 0.f;   // (no token is seen, or all that are score -inf)
        s_lse[tid] = none || tid >= p.rows ? INFINITY : m + log2f(l);
        if (none && tid < p.rows && t0 == 0) atomicOr(p.status, kStatusShortContext);
    }
    __syncthreads();
    float lse[ROWS];
    bool any_nan = false;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        lse[r] = s_lse[r];
        any_nan = any_nan || lse[r] != lse[r];
    }
    for (int t1 = t0; t1 < end; t1 += 256 * TOK) {
        float w[TOK];
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            w[k] = 0.f;
#pragma unroll
            for (int r = 0; r < ROWS; ++r)   // (-inf: hidden, or of no weight)
                w[k] += r < p.rows && x[k][r] != -INFINITY ? fast_exp2(x[k][r] - lse[r]) : 0.f;
            if (fade) w[k] = fmaf(p.decay, old[k], w[k]);
        }
        if (any_nan) {
#pragma unroll 1
            for (int k = 0; k < TOK; ++k) {
                const float x = nan_rows<ROWS>(s_lse, t1 + tid + 256 * k, L - p.tq, p.group);
#pragma unroll
                for (int i = 0; i < TOK; ++i) w[i] += i == k ? x : 0.f;
            }
        }
        if (t1 + 256 * TOK < end) load(t1 + 256 * TOK);   // (in flight while these are stored)
#pragma unroll
        for (int k = 0; k < TOK; ++k)
            if (t1 + tid + 256 * k < end) out[t1 + tid + 256 * k] = w[k];
    }
}

template <int KB, int ROWS>
static int launch_one(const StepParams& p, const CUtensorMap* kmap, int tokens, cudaStream_t stream) {
    using C = StepCfg<KB, ROWS>;
    auto* kernel = tq_step_scores_kernel<KB, ROWS, true>;
    static std::atomic<uint64_t> attr_done{0}, size_done{0};
    cudaError_t e = set_smem_attr_once(kernel, C::kOneAlloc(kStepOneTokens), size_done);
    if (e == cudaSuccess) e = allow_large_clusters_once(kernel, attr_done);
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(p.batch) * p.hkv * kStepCluster), dim3(128), kStepCluster,
                              C::kOneAlloc(tokens), stream, p, *kmap);
}

template <int KB, int ROWS>
static int launch_t(StepParams p, const CUtensorMap* kmap, cudaStream_t stream) {
    using C = StepCfg<KB, ROWS>;
    // The one-kernel form: up to 1024 tokens a CTA where each has an SM of its own, for
    // quantized K up to 512 where four share one.  (turbo3, 4 units of 8,000 tokens 7.2 us
    // and 11.6 with two kernels, of 16,000 10.3 and 13.5, of 32,000 16.4 and 15.6; 32 units
    // of 8,000 11.7 and 13.1; 16 of 16,000 14.4 and 13.0; fp16 K, 8 units of 16,000 11.3 and
    // 13.0, 16 of 8,000 13.0 and 13.2, 32 of 4,000 15.8 and 13.6.)
    const int tokens = ((p.max_len + 31) / 32 + kStepCluster - 1) / kStepCluster * 32;
    const long long ctas = 1ll * p.batch * p.hkv * kStepCluster;
    if (ctas <= host::kSMs ? tokens <= kStepOneTokens : KB != 0 && ctas <= 4 * host::kSMs && tokens <= kStepOneTokens / 2)
        return launch_one<KB, ROWS>(p, kmap, tokens, stream);
    static std::atomic<uint64_t> attr_done{0};
    cudaError_t e = set_smem_attr_once(tq_step_scores_kernel<KB, ROWS, false>, C::kSmemAlloc, attr_done);
    if (e != cudaSuccess) return e;
    e = launch_pdl(tq_step_scores_kernel<KB, ROWS, false>, dim3(p.ctas), dim3(128), C::kSmemAlloc, stream, p, *kmap);
    if (e != cudaSuccess) return e;
    // Few tokens: a token a thread, so that more SMs share them.  Many: up to 8 a thread,
    // four loads in flight, for as many CTAs as are resident at once.  (turbo3, 32 units of 4,000
    // tokens 13.5 us and 14.4, 8 of 20,000 both 19.6, 16 of 10,000 19.6 and 18.6, 64 of 10,000 33.9
    // and 29.8.)
    const long long units = 1ll * p.batch * p.hkv;
    constexpr int kMany = ROWS == 16 ? 1 : 4;
    if (units * ((p.max_len + 255) / 256) <= 4 * host::kSMs) {
        p.span = 256;
        return launch_pdl(tq_step_sums_kernel<ROWS, 1>, dim3(static_cast<unsigned>(units * ((p.max_len + 255) / 256))),
                          dim3(256), 0, stream, p);
    }
    p.span = 256 * kMany;
    while (p.span < 8192 && units * ((p.max_len + p.span - 1) / p.span) > 8 * host::kSMs) p.span *= 2;
    return launch_pdl(tq_step_sums_kernel<ROWS, kMany>, dim3(static_cast<unsigned>(units * ((p.max_len + p.span - 1) / p.span))),
                      dim3(256), 0, stream, p);
}

int launch_weights_step(int kbits, int rows, const StepParams& p, const CUtensorMap* kmap, cudaStream_t stream) {
    if (kbits == 16) return rows <= 8 ? launch_t<0, 8>(p, kmap, stream) : launch_t<0, 16>(p, kmap, stream);
    if (kbits == 3)
        return rows == 4   ? launch_t<3, 4>(p, kmap, stream)
               : rows == 8 ? launch_t<3, 8>(p, kmap, stream)
                           : launch_t<3, 16>(p, kmap, stream);
    if (kbits == 4)
        return rows == 4   ? launch_t<4, 4>(p, kmap, stream)
               : rows == 8 ? launch_t<4, 8>(p, kmap, stream)
                           : launch_t<4, 16>(p, kmap, stream);
    return cudaErrorInvalidValue;
}

// Resident CTAs per SM of the scores kernel.
template <int KB, int ROWS>
static int ctas_t() {
    using C = StepCfg<KB, ROWS>;
    return std::min(C::kMinCtas, (228 * 1024) / (C::kSmemAlloc + 1024));
}
int weights_step_ctas_per_sm(int kbits, int rows) {
    if (kbits == 16) return rows <= 8 ? ctas_t<0, 8>() : ctas_t<0, 16>();
    if (kbits == 3) return rows == 4 ? ctas_t<3, 4>() : rows == 8 ? ctas_t<3, 8>() : ctas_t<3, 16>();
    return rows == 4 ? ctas_t<4, 4>() : rows == 8 ? ctas_t<4, 8>() : ctas_t<4, 16>();
}

}  // namespace tq
