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
// term is rounded once.  The base of a row may trail its scores by 10 (log2), or
// by as much less as keeps p n_v of the tile's largest norm in fp16: with a slack
// of 4 every third tile had a row that moved its base, with 10 hardly any has.
//
// What bounds it: the tensor core needs 24 MMAs of 64 cycles for a tile (0.74
// us), the exponentials 1024 cycles of MUFU (0.5 us), dequantisation and
// softmax some 1000 issue slots per scheduler (0.5 us); but one group of four
// warps runs them in turn.  So a CTA has two groups, each with its own token
// tiles (group g takes every second one), its own K and V tiles, S and O, and
// nothing to wait for from the other one until they merge at the end: one
// group's MMAs and waits are filled by the other's dequantisation and softmax.
// Within a group S(n) runs under the V dequantisation and P.V(n) under the next
// K dequantisation.
//
// Split: the (batch, kv head, row tile) units lie end to end as 128-token
// chunks, and CTA c of P takes [c C / P, (c + 1) C / P) of the C chunks, from
// the actual lengths; it writes one partial (m, l, O) per unit that it touches,
// which tq_tree_combine_kernel merges, normalises and rotates back.
#include <float.h>

#include <algorithm>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kTok = 128;            // tokens per tile (chunk)
constexpr int kTreeRows = 128;       // query rows per unit
constexpr float kSlack = 10.f;         // log2 by which a score may pass its row's base

template <int KB, int VB>
struct TreeCfg {
    static constexpr int kRbK = (KB == 0) ? 256 : KB * 16;
    static constexpr int kRbV = VB * 16;
    static constexpr int kQOff = 0;                                   // fp16 Q' (q_hi), 32 KB
    static constexpr int kQloOff = (KB == 0) ? 0 : 32768;             // q_lo (quantized K), 32 KB
    static constexpr int kVtOff = (KB == 0) ? 32768 : 65536;          // per group V^T [dim][token], 32 KB
    // quantized K: per group K [token][dim] (32 KB) and its records; fp16 K:
    // the MMA tiles as they are copied, three that the groups' tiles take in turn
    static constexpr int kKOff = kVtOff + 65536;
    static constexpr int kKTiles = (KB == 0) ? 3 : 2;
    static constexpr int kSKOff = kKOff + kKTiles * 32768;
    static constexpr int kSK = (KB == 0) ? 0 : kTok * kRbK;
    static constexpr int kSVOff = kSKOff + 2 * kSK;                   // per group V records
    static constexpr int kSV = kTok * kRbV;
    static constexpr int kColOff = kSVOff + 2 * kSV;                  // per group n_k scale log2 e [128]
    static constexpr int kNvOff = kColOff + 2 * kTok * 4;             // per group n_v [128]
    // mbarriers: K copied [3], V copied [2], K stored [2], V stored [2] (fp16
    // K), softmax done [2], S done [2], P.V done [2], V records free [2], Q'
    // stored, K tile read [3] (fp16 K); TMEM slot
    static constexpr int kBarOff = kNvOff + 2 * kTok * 4;
    static constexpr int kBars = 21;   // (odd: 16-byte alignment behind the TMEM slot)
    static constexpr int kNmOff = kBarOff + 8 * kBars + 8;             // per group the largest n_v of each warp's tokens
    static constexpr int kSmem = kNmOff + 32;
    static constexpr int kSmemAlloc = kSmem + 768;   // to a 1024-byte boundary from a 256-byte one
    static_assert(kSmemAlloc <= 232448, "227 KB per CTA");
    static constexpr uint32_t kIdesc = umma_idesc_f16_f32(128, 128);
};

// Warp groups of four warps: 0 and 1 the softmax groups, 2 dequantises, 3 has
// the issuing warps.  Registers per thread after the split (sum times 128 is
// the launch's 512 x 128).
constexpr int kTreeThreads = 512;
constexpr int kRegsSoftmax = 200, kRegsDequant = 72, kRegsIssue = 40;
static_assert(2 * kRegsSoftmax + kRegsDequant + kRegsIssue <= 4 * 128, "within the launch's registers");

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// V^T of 128 tokens from their records, by four warps (w = 0..3): lane 4v + t
// dequantises quarter t of tokens 16 vw + v and + 8, stored transposed in rows
// pi(d) = d ^ 2(d >> 5), whose 8 rows per stored matrix lie in different banks.
template <int VB>
__device__ __forceinline__ void store_vt(const uint8_t* rec, uint8_t* sVt, const Tables& vt, int w, int lane) {
    constexpr int rb = VB * 16;
    const int sj = lane >> 3, sc = lane & 7;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int vw = w + 4 * i;
        const int ta = 16 * vw + (lane >> 2);
        uint32_t ha[16], hb[16];
        dequant_q32<VB>(rec + ta * rb + (lane & 3) * (rb / 4), vt, ha);
        dequant_q32<VB>(rec + (ta + 8) * rb + (lane & 3) * (rb / 4), vt, hb);
        const int tokc = 2 * (vw & 3) + (sj & 1);
        uint32_t va[2];
#pragma unroll
        for (int par = 0; par < 2; ++par) {
            const int row = 32 * (sc >> 1) + 2 * ((((par << 1) | (sj >> 1)) ^ (sc >> 1)) & 3) + (sc & 1);
            va[par] = smem_u32(sVt) + (vw >> 2) * 16384 + row * 128 + ((tokc ^ (row & 7)) << 4);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            stsm_x4_trans(va[k & 1] + 1024 * (k >> 1), ha[2 * k], hb[2 * k], ha[2 * k + 1], hb[2 * k + 1]);
    }
}

// Where token t's scale and norm lie: the four of lane t's columns (2t, 2t + 1,
// 8 + 2t, 9 + 2t of 16) together.
__device__ __forceinline__ int frag_place(int t) {
    return (t & ~15) | ((t & 6) << 1) | ((t & 8) >> 2) | (t & 1);
}

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

// All chunks of the call (whole warp).
__device__ __forceinline__ int tree_total(const TreeParams& p, int lane) {
    int v = 0;
    for (int b = lane; b < p.batch; b += 32) v += tree_chunks(p.lengths[b], p.max_len) * p.per_b;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sequence that holds chunk pos, and the chunks of all before it (whole warp).
__device__ __forceinline__ void tree_locate(const TreeParams& p, int pos, int lane, int& b, int& before) {
    int cum = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const int v = b0 + lane < p.batch ? tree_chunks(p.lengths[b0 + lane], p.max_len) * p.per_b : 0;
        const int inc = lane_prefix(v, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, cum + inc > pos);
        if (hit) {
            const int l = __ffs(hit) - 1;
            b = b0 + l;
            before = cum + __shfl_sync(0xffffffffu, inc - v, l);
            return;
        }
        cum += __shfl_sync(0xffffffffu, inc, 31);
    }
    b = 0;   // pos past the end (not reached by the callers)
    before = 0;
}

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

    griddep_wait();   // cache, lengths, mask and q come from earlier work on the stream
    const int P = static_cast<int>(gridDim.x), c_me = static_cast<int>(blockIdx.x);
    const int total = __shfl_sync(0xffffffffu, tree_total(p, lane), 0);
    const int lo = static_cast<int>(static_cast<long long>(c_me) * total / P);
    const int hi = static_cast<int>(static_cast<long long>(c_me + 1) * total / P);
    if (lo >= hi) return;   // (uniform over the CTA)

    const uint32_t bars = smem_u32(smem + C::kBarOff);
    const uint32_t bar_k = bars, bar_v = bars + 24, bar_kr = bars + 40, bar_vr = bars + 56, bar_p = bars + 72,
                   bar_s = bars + 88, bar_o = bars + 104, bar_vf = bars + 120, bar_q = bars + 136, bar_kf = bars + 144;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 8 * C::kBars);
    if (tid == 0) {
        for (int i = 0; i < 5; ++i) mbar_init(bar_k + 8 * i, 1);      // K copied, V copied
        for (int i = 0; i < 6; ++i) mbar_init(bar_kr + 8 * i, 128);   // K stored, V stored, softmax done
        for (int i = 0; i < 4; ++i) mbar_init(bar_s + 8 * i, 1);      // S done, P.V done
        for (int i = 0; i < 2; ++i) mbar_init(bar_vf + 8 * i, 4);     // V records free: a warp each
        mbar_init(bar_q, 256);
        for (int i = 0; i < 3; ++i) mbar_init(bar_kf + 8 * i, 1);     // K tile read
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(smem_u32(tslot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem0 = *tslot;   // group g: columns 256 g: S (its first 64 take P), then O

    bool stalled = false;   // once set, waits return at once and nothing more is issued
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!stalled && !mbar_wait_bounded(bar, parity)) stalled = true;
    };
    // Tiles of the earlier segments: all of them (the K ring of fp16 K), and of
    // each group (every other barrier completes one phase per tile of its group)
    int tbase = 0;
    uint32_t used[2] = {0, 0};
    uint32_t segs = 0;
    int pos = lo;

    // The segment at pos: chunks [k0, k0 + ntiles) of unit (b, h, rt).
    struct Segment {
        int b, h, rt, ui, k0, ntiles, L, t_lim;
        size_t row0;
    };
    auto segment = [&]() {
        Segment s;
        int before;
        tree_locate(p, pos, lane, s.b, before);
        s.b = __shfl_sync(0xffffffffu, s.b, 0);
        before = __shfl_sync(0xffffffffu, before, 0);
        s.L = p.lengths[s.b];
        const int nch = tree_chunks(s.L, p.max_len);
        s.ui = (pos - before) / nch;   // h * row_tiles + rt
        s.k0 = (pos - before) - s.ui * nch;
        s.ntiles = min(nch - s.k0, hi - pos);
        s.h = s.ui / p.row_tiles;
        s.rt = s.ui - s.h * p.row_tiles;
        s.t_lim = min(s.L, p.max_len);
        s.row0 = (static_cast<size_t>(s.b) * p.hkv + s.h) * p.cap;
        return s;
    };
    // all warps: the end of a segment; true when some wait timed out
    auto end_segment = [&](const Segment& s) {
        tc_fence_before();
        const bool bad = __syncthreads_or(stalled) != 0;
        tc_fence_after();
        tbase += s.ntiles;
        used[0] += (s.ntiles + 1) >> 1;
        used[1] += s.ntiles >> 1;
        ++segs;
        pos += s.ntiles;
        return bad;
    };

    if (wg == 3) {
        // ---- issuing warps: one thread each for the MMAs, the K copies and the V copies ----
        regs_dec<kRegsIssue>();
        const int role = warp & 3;
        bool bad = false;
        uint32_t sent_s[2] = {0, 0}, sent_o[2] = {0, 0}, sent = 0;
        while (pos < hi && !bad) {
            const Segment s = segment();
            if (role == 0 && lane == 0) {
                // S(n) of a group once K(n) is there and its last P.V has read P;
                // P.V(n) once its softmax is done: whichever group is ready
                wait(bar_q, segs & 1);
                tc_fence_after();
                int ns[2] = {0, 1}, no[2] = {0, 1};   // each group's next S and P.V tile
                uint64_t t0 = global_timer_ns();
                for (uint32_t spin = 1; !stalled && (no[0] < s.ntiles || no[1] < s.ntiles); ++spin) {
                    bool moved = false;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const uint32_t tm = tmem0 + 256 * g;
                        const uint32_t iu = used[g] + (no[g] >> 1);   // index of the group's next P.V (and S before it)
                        if (no[g] < s.ntiles && ns[g] > no[g]) {
                            if (mbar_test_wait(bar_p + 8 * g, iu & 1) &&
                                (KB != 0 || mbar_test_wait(bar_vr + 8 * g, iu & 1))) {
                                tc_fence_after();
                                const uint32_t vt = smem_u32(smem + C::kVtOff + g * 32768);
#pragma unroll
                                for (int kk = 0; kk < 8; ++kk)
                                    umma_f16_ts(tm + 128, tm + 8 * kk,
                                                umma_desc_sw128(vt + (kk >> 2) * 16384 + (kk & 3) * 32), C::kIdesc,
                                                (no[g] != g || kk > 0) ? 1u : 0u);
                                umma_commit(bar_o + 8 * g);
                                ++sent_o[g];
                                no[g] += 2;
                                moved = true;
                            }
                        } else if (ns[g] < s.ntiles && ns[g] == no[g]) {
                            const int t = tbase + ns[g];
                            const bool k_in = KB == 0 ? mbar_test_wait(bar_k + 8 * (t % 3), (t / 3) & 1)
                                                      : mbar_test_wait(bar_kr + 8 * g, iu & 1);
                            if (k_in && (iu == 0 || mbar_test_wait(bar_o + 8 * g, (iu - 1) & 1))) {
                                tc_fence_after();
                                const uint32_t kbase = smem_u32(smem + C::kKOff + (KB == 0 ? t % 3 : g) * 32768);
#pragma unroll
                                for (int kk = 0; kk < 8; ++kk) {
                                    const uint32_t koff = (kk >> 2) * 16384 + (kk & 3) * 32;
                                    umma_f16(tm, umma_desc_sw128(smem_u32(smem + C::kQOff) + koff),
                                             umma_desc_sw128(kbase + koff), C::kIdesc, kk > 0 ? 1u : 0u);
                                    if constexpr (KB != 0)
                                        umma_f16(tm, umma_desc_sw128(smem_u32(smem + C::kQloOff) + koff),
                                                 umma_desc_sw128(kbase + koff), C::kIdesc, 1u);
                                }
                                umma_commit(bar_s + 8 * g);
                                if constexpr (KB == 0) umma_commit(bar_kf + 8 * (t % 3));
                                ++sent_s[g];
                                ns[g] += 2;
                                moved = true;
                            }
                        }
                    }
                    if (moved) t0 = global_timer_ns();
                    else if ((spin & 255u) == 0 && global_timer_ns() - t0 > 2000000000ull) stalled = true;
                }
            } else if (role == 1 && lane == 0) {
                for (int n = 0; n < s.ntiles && !stalled; ++n) {   // K records (fp16 K: MMA tiles)
                    const int g = n & 1, t = tbase + n;
                    const uint32_t iu = used[g] + (n >> 1);
                    const int tok0 = (s.k0 + n) * kTok;
                    if constexpr (KB == 0) {
                        if (t >= 3) wait(bar_kf + 8 * (t % 3), (t / 3 - 1) & 1);   // S has read the ring's tile t - 3
                        if (stalled) break;
                        const uint32_t bar = bar_k + 8 * (t % 3), dst = smem_u32(smem + C::kKOff + (t % 3) * 32768);
                        mbar_arrive_expect_tx(bar, 32768);
                        for (int half = 0; half < 2; ++half)
                            for (int q = 0; q < 4; ++q)
                                tma_g2s_2d(dst + half * 16384 + q * 4096, &kmap, half * 64,
                                           static_cast<int32_t>(s.row0 + tok0 + q * 32), bar);
                    } else {
                        if (n >= 2) wait(bar_kr + 8 * g, (iu - 1) & 1);   // the last tile's records are read
                        if (stalled) break;
                        const uint32_t bytes = min(kTok, s.t_lim - tok0) * C::kRbK;
                        fence_proxy_async();
                        mbar_arrive_expect_tx(bar_k + 8 * g, bytes);
                        bulk_g2s(smem_u32(smem + C::kSKOff + g * C::kSK), p.k_codes + (s.row0 + tok0) * C::kRbK, bytes,
                                 bar_k + 8 * g);
                    }
                    ++sent;
                }
            } else if (role == 2 && lane == 0) {
                for (int n = 0; n < s.ntiles && !stalled; ++n) {   // V records
                    const int g = n & 1;
                    const uint32_t iu = used[g] + (n >> 1);
                    const int tok0 = (s.k0 + n) * kTok;
                    if (n >= 2) wait(bar_vf + 8 * g, (iu - 1) & 1);
                    if (stalled) break;
                    const uint32_t bytes = min(kTok, s.t_lim - tok0) * C::kRbV;
                    fence_proxy_async();
                    mbar_arrive_expect_tx(bar_v + 8 * g, bytes);
                    bulk_g2s(smem_u32(smem + C::kSVOff + g * C::kSV), p.v_codes + (s.row0 + tok0) * C::kRbV, bytes,
                             bar_v + 8 * g);
                    ++sent;
                }
            }
            __syncwarp();
            // (on a time-out, what is in flight ends before the memory goes
            // away; a copy's barrier completes when its bytes have landed)
            const Segment cur = s;
            const int tb = tbase;
            const uint32_t u0 = used[0], u1 = used[1];
            bad = end_segment(cur);
            if (bad && lane == 0) {
                if (role == 0) {
                    atomicOr(p.status, kStatusPipelineStall);
                    for (int g = 0; g < 2; ++g) {
                        if (sent_s[g] > 0) (void)mbar_wait_bounded(bar_s + 8 * g, (sent_s[g] - 1) & 1);
                        if (sent_o[g] > 0) (void)mbar_wait_bounded(bar_o + 8 * g, (sent_o[g] - 1) & 1);
                    }
                } else if (role <= 2 && sent > 0) {
                    const int done = static_cast<int>(sent) - tb;   // tiles of this segment that were sent
                    for (int n = max(0, done - 3); n < done; ++n) {
                        const uint32_t iu = ((n & 1) ? u1 : u0) + (n >> 1);
                        if (role == 2) (void)mbar_wait_bounded(bar_v + 8 * (n & 1), iu & 1);
                        else if (KB == 0) (void)mbar_wait_bounded(bar_k + 8 * ((tb + n) % 3), ((tb + n) / 3) & 1);
                        else (void)mbar_wait_bounded(bar_k + 8 * (n & 1), iu & 1);
                    }
                }
            }
        }
    } else if (wg == 2) {
        // ---- dequantising warps: K(n) of both groups, or with fp16 K V(n)^T ----
        regs_dec<kRegsDequant>();
        const int r = tid & 127;
        bool bad = false;
        while (pos < hi && !bad) {
            const Segment s = segment();
            if constexpr (KB != 0) {
                auto norm = [&](int n) {
                    const int t = (s.k0 + n) * kTok + r;
                    return n < s.ntiles && t < s.t_lim ? __half2float(p.k_norm[s.row0 + t]) : 0.f;
                };
                float nk = norm(0), nk1 = norm(1);
                for (int n = 0; n < s.ntiles; ++n) {
                    const int g = n & 1;
                    const uint32_t iu = used[g] + (n >> 1);
                    const float nk2 = norm(n + 2);
                    wait(bar_k + 8 * g, iu & 1);
                    if (iu > 0) wait(bar_s + 8 * g, (iu - 1) & 1);   // the group's last S has read its K tile
                    // a token per thread; the quarters are taken in an order that
                    // differs between lanes whose records start in the same banks
                    const Tables kt{p.ktab[0], p.ktab[1], p.ktab[2], p.ktab[3]};
                    const uint8_t* rec = smem + C::kSKOff + g * C::kSK + r * C::kRbK;
                    uint8_t* sK = smem + C::kKOff + g * 32768;
                    const int turn = KB == 4 ? r >> 1 : r >> 3;
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
                    if (iu > 0) wait(bar_p + 8 * g, (iu - 1) & 1);   // the group's last softmax has read the scales
                    (reinterpret_cast<float*>(smem + C::kColOff) + g * kTok)[frag_place(r)] = nk * p.scale_log2e;
                    mbar_arrive(bar_kr + 8 * g);
                    nk = nk1;
                    nk1 = nk2;
                }
            } else {
                const Tables vt{p.vtab[0], p.vtab[1], p.vtab[2], p.vtab[3]};
                for (int n = 0; n < s.ntiles; ++n) {
                    const int g = n & 1;
                    const uint32_t iu = used[g] + (n >> 1);
                    wait(bar_v + 8 * g, iu & 1);
                    if (iu > 0) wait(bar_o + 8 * g, (iu - 1) & 1);   // the group's last P.V has read its V tile
                    store_vt<VB>(smem + C::kSVOff + g * C::kSV, smem + C::kVtOff + g * 32768, vt, warp & 3, lane);
                    fence_proxy_async();
                    mbar_arrive(bar_vr + 8 * g);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_vf + 8 * g);
                }
            }
            bad = end_segment(s);
        }
    } else {
        // ---- softmax groups ----
        regs_inc<kRegsSoftmax>();
        const int g = wg, r = tid & 127;   // group; row (tensor-memory lane), and token of its tiles
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem0 + 256 * g + lane_off, t_o = t_s + 128;
        uint8_t* sVt = smem + C::kVtOff + g * 32768;
        const float* col = reinterpret_cast<const float*>(smem + C::kColOff) + g * kTok;
        float* nvs = reinterpret_cast<float*>(smem + C::kNvOff) + g * kTok;
        float* nvm = reinterpret_cast<float*>(smem + C::kNmOff) + 4 * g;
        bool bad = false;
        while (pos < hi && !bad) {
            const Segment s = segment();
            const int base = s.L - p.tq;                   // first drafted token
            const int full_below = min(base, s.t_lim);     // tokens below this are seen by every row
            const bool row_ok = s.rt * kTreeRows + r < p.rows;               // (row r of the tile)
            const int row32 = s.rt * kTreeRows + 32 * (warp & 3);
            const bool live = row32 < p.rows;                                // some row of the warp's 32 exists
            const uint32_t* mask = p.tree + static_cast<size_t>(s.b) * p.tree_per_seq;
            auto norm = [&](int n) {
                const int t = (s.k0 + n) * kTok + r;
                return n < s.ntiles && t < s.t_lim ? __half2float(p.v_norm[s.row0 + t]) : 0.f;
            };
            float nv = norm(g);

            // ---- Q' of the unit's rows: two threads per row, 64 dims each ----
            {
            const int qr = tid >> 1, half = tid & 1;
                const int qrr = s.rt * kTreeRows + qr;
                float x[64];
                if (qrr < p.rows) {
                    const int j = qrr / p.group, hl = qrr - j * p.group;
                    const __half* qp = p.q + ((static_cast<size_t>(s.b) * p.hq + s.h * p.group + hl) * p.tq + j) * kD + 64 * half;
#pragma unroll
                    for (int k = 0; k < 64; k += 8) {
                        const uint4 w = *reinterpret_cast<const uint4*>(qp + k);
                        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ww[e]));
                            x[k + 2 * e] = f.x;
                            x[k + 2 * e + 1] = f.y;
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 64; ++k) x[k] = 0.f;
                }
                if constexpr (KB != 0) {
                    const uint32_t s0 = half ? p.signs[2] : p.signs[0], s1 = half ? p.signs[3] : p.signs[1];
#pragma unroll
                    for (int k = 0; k < 64; ++k) x[k] = (((k < 32 ? s0 : s1) >> (k & 31)) & 1u) ? -x[k] : x[k];
#pragma unroll
                    for (int m = 1; m < 64; m <<= 1)
#pragma unroll
                        for (int k = 0; k < 64; ++k)
                            if (!(k & m)) {
                                const float a = x[k], c = x[k + m];
                                x[k] = a + c;
                                x[k + m] = a - c;
                            }
                    // the last stage pairs dim k with dim 64 + k, the other thread's
#pragma unroll
                    for (int k = 0; k < 64; ++k) {
                        const float o = __shfl_xor_sync(0xffffffffu, x[k], 1);
                        x[k] = (half ? o - x[k] : x[k] + o) * 0.08838834764831845f;   // 1/sqrt(128)
                    }
                }
#pragma unroll
                for (int k = 0; k < 64; k += 8) {
                    uint32_t hv[4], lv[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        hv[e] = pack_half2(x[k + 2 * e], x[k + 2 * e + 1]);
                        if constexpr (KB != 0) {   // q_lo = Rot(q) - q_hi (exact in fp32), rounded once more
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hv[e]));
                            lv[e] = pack_half2(x[k + 2 * e] - f.x, x[k + 2 * e + 1] - f.y);
                        }
                    }
                    const uint32_t off = sw128_offset(qr, 64 * half + k);
                    *reinterpret_cast<uint4*>(smem + C::kQOff + off) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
                    if constexpr (KB != 0)
                        *reinterpret_cast<uint4*>(smem + C::kQloOff + off) = make_uint4(lv[0], lv[1], lv[2], lv[3]);
                }
            }
            fence_proxy_async();   // the MMAs read Q' through the async proxy
            mbar_arrive(bar_q);

            // The softmax holds its scores as MMA fragments: lane 4v + t has rows
            // v + 8q (q = 0..3) of the warp's 32 and columns 2t, 2t + 1 of every
            // eight, so a thread reads a quarter of the tile's scales and norms
            // (with a row per thread, their broadcast reads took a third of the
            // shared-memory bandwidth that the MMAs' operands need).
            float m_base[4], l_sum[4];   // base (log2) and this thread's part of the sum of rows v + 8q
#pragma unroll
            for (int q = 0; q < 4; ++q) m_base[q] = -INFINITY, l_sum[q] = 0.f;
            for (int n = g; n < s.ntiles; n += 2) {
                const int tok0 = (s.k0 + n) * kTok;
                const uint32_t iu = used[g] + (n >> 1);
                // (an overflowed norm counts as 65504: 0 * inf would be NaN in the
                // rows that do not see the token)
                nv = fminf(nv, 65504.f);
                nvs[frag_place(r)] = nv;
                // the largest norm of each warp's tokens (non-negative floats order
                // like their bits)
                const uint32_t nmax = __reduce_max_sync(0xffffffffu, __float_as_uint(nv));
                if (lane == 0) nvm[warp & 3] = __uint_as_float(nmax);
                nv = norm(n + 2);
                if constexpr (KB != 0) {   // V(n)^T, under the S product
                    wait(bar_v + 8 * g, iu & 1);
                    if (n != g) wait(bar_o + 8 * g, (iu - 1) & 1);   // the last P.V has read V^T
                    const Tables vt{p.vtab[0], p.vtab[1], p.vtab[2], p.vtab[3]};
                    store_vt<VB>(smem + C::kSVOff + g * C::kSV, sVt, vt, warp & 3, lane);
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_vf + 8 * g);
                } else {
                    if (n != g) wait(bar_o + 8 * g, (iu - 1) & 1);   // (O may be rescaled)
                }
                named_bar_sync(1 + g, 128);   // the norms are stored
                wait(bar_s + 8 * g, iu & 1);
                if constexpr (KB != 0) wait(bar_kr + 8 * g, iu & 1);   // the scales of tile n are stored
                tc_fence_after();
                if (live) {   // (warp-uniform) softmax
                    // how far a score may pass its row's base: p n_v stays below 2^15.99
                    const float4 nm = *reinterpret_cast<const float4*>(nvm);
                    const float slack = fminf(kSlack, 15.99f - __log2f(fmaxf(fmaxf(nm.x, nm.y), fmaxf(nm.z, nm.w))));
                    // Most tiles are seen whole by every row and raise no base: one
                    // pass over S, 32 columns at a time with the next ones in
                    // flight, P held in registers and stored at the end unless some
                    // score passed its row's base by more than the slack.  Then, on a row's
                    // first tile and where the mask comes in, the tile is taken
                    // from S by the two rolled passes below.
                    const bool partial = tok0 + kTok > full_below;   // some row sees the tile in part
                    const uint32_t t_hi = t_s + (16u << 16);         // rows 16-31
                    bool fresh_row = false;
#pragma unroll
                    for (int q = 0; q < 4; ++q) fresh_row |= m_base[q] == -INFINITY;
                    bool slow = partial || __any_sync(0xffffffffu, fresh_row);
                    if (!slow) {
                        uint32_t pk[2][4][8];   // [rows 0-15, 16-31][32 tokens]
                        uint32_t v[2][2][16];   // [buffer][rows 0-15, 16-31]
                        float2 sum[4], nb[4];
                        float mq[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            sum[q] = make_float2(0.f, 0.f);
                            nb[q] = make_float2(-m_base[q], -m_base[q]);
                            mq[q] = -INFINITY;
                        }
                        tmem_ld_frag_issue(t_s, v[0][0]);
                        tmem_ld_frag_issue(t_hi, v[0][1]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            tmem_ld_wait(v[c & 1][0], v[c & 1][1]);
                            if (c < 3) {
                                tmem_ld_frag_issue(t_s + 32 * (c + 1), v[(c + 1) & 1][0]);
                                tmem_ld_frag_issue(t_hi + 32 * (c + 1), v[(c + 1) & 1][1]);
                            }
#pragma unroll
                            for (int h2 = 0; h2 < 2; ++h2) {
                                const int place = 32 * c + 16 * h2 + 4 * (lane & 3);
                                float4 s4 = make_float4(p.scale_log2e, p.scale_log2e, p.scale_log2e, p.scale_log2e);
                                if constexpr (KB != 0) s4 = *reinterpret_cast<const float4*>(col + place);
                                const float4 w4 = *reinterpret_cast<const float4*>(nvs + place);
#pragma unroll
                                for (int i = 0; i < 2; ++i)
#pragma unroll
                                    for (int q = 0; q < 4; ++q) {
                                        const uint32_t* e = v[c & 1][q >> 1] + 8 * h2 + 4 * i + 2 * (q & 1);
                                        const float2 x =
                                            __ffma2_rn(make_float2(__uint_as_float(e[0]), __uint_as_float(e[1])),
                                                       i ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y), nb[q]);
                                        mq[q] = fmaxf(mq[q], fmaxf(x.x, x.y));
                                        const float2 pe = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                                        sum[q] = __fadd2_rn(sum[q], pe);
                                        const float2 w = __fmul2_rn(pe, i ? make_float2(w4.z, w4.w) : make_float2(w4.x, w4.y));
                                        pk[q >> 1][c][2 * (2 * h2 + i) + (q & 1)] = pack_half2(w.x, w.y);
                                    }
                            }
                        }
                        const float top = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
                        slow = __any_sync(0xffffffffu, top > slack);
                        if (!slow) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) l_sum[q] += sum[q].x + sum[q].y;
#pragma unroll
                            for (int c = 0; c < 4; ++c) {   // P over S columns 0..63
                                tmem_st_frag_issue(t_s + 16 * c, pk[0][c]);
                                tmem_st_frag_issue(t_hi + 16 * c, pk[1][c]);
                            }
                            tmem_st_wait();
                        }
                    }
                    if (slow) {
                    // Two passes, 32 columns a turn in two halves, one half in
                    // flight while the other is worked on: the rows' largest
                    // scores, which may move their bases, then P over S (the 16
                    // columns that a turn stores it has read before).
                    float2 nb[4];
                    auto set_base = [&]() {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float b0 = m_base[q] == -INFINITY ? 0.f : -m_base[q];
                            nb[q] = make_float2(b0, b0);
                        }
                    };
                    // x of columns 16c .. 16c + 15 from their S values: f(q, i, x)
                    auto scores = [&](int c, const uint32_t (&lo16)[8], const uint32_t (&hi16)[8], auto f) {
                        float4 s4 = make_float4(p.scale_log2e, p.scale_log2e, p.scale_log2e, p.scale_log2e);
                        if constexpr (KB != 0) s4 = *reinterpret_cast<const float4*>(col + 16 * c + 4 * (lane & 3));
                        uint32_t vis[4] = {0x303u, 0x303u, 0x303u, 0x303u};   // bits 0, 1, 8, 9: this thread's columns
                        if (partial) {
                            const int t0 = tok0 + 16 * c;
#pragma unroll 1
                            for (int q = 0; q < 4; ++q) {
                                const int rr = row32 + (lane >> 2) + 8 * q;
                                uint32_t w = rr < p.rows ? tree_window(mask + (rr / p.group) * p.tree_words,
                                                                       p.tree_words, t0 - base)
                                                         : 0u;
                                if (t0 + 32 > s.t_lim) w &= t0 < s.t_lim ? (1u << (s.t_lim - t0)) - 1u : 0u;
                                w >>= 2 * (lane & 3);
                                vis[0] = q == 0 ? w : vis[0];
                                vis[1] = q == 1 ? w : vis[1];
                                vis[2] = q == 2 ? w : vis[2];
                                vis[3] = q == 3 ? w : vis[3];
                            }
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t* e = (q < 2 ? lo16 : hi16) + 4 * i + 2 * (q & 1);
                                float2 x = __ffma2_rn(make_float2(__uint_as_float(e[0]), __uint_as_float(e[1])),
                                                      i ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y), nb[q]);
                                if (partial) {
                                    if (!((vis[q] >> (8 * i)) & 1u)) x.x = -INFINITY;
                                    if (!((vis[q] >> (8 * i + 1)) & 1u)) x.y = -INFINITY;
                                }
                                f(q, i, x);
                            }
                    };
                    uint32_t a0[8], a1[8], b0[8], b1[8];
                    // ---- the largest score of each row over its base ----
                    set_base();
                    float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    auto take_max = [&](int q, int, float2 x) { mq[q] = fmaxf(mq[q], fmaxf(x.x, x.y)); };
                    tmem_ld_frag_issue(t_s, a0);
                    tmem_ld_frag_issue(t_hi, a1);
#pragma unroll 1
                    for (int c = 0; c < 8; c += 2) {
                        tmem_ld_wait(a0, a1);
                        tmem_ld_frag_issue(t_s + 16 * c + 16, b0);
                        tmem_ld_frag_issue(t_hi + 16 * c + 16, b1);
                        scores(c, a0, a1, take_max);
                        tmem_ld_wait(b0, b1);
                        // (the last turn fetches the first columns again, for the pass below)
                        const int next = (16 * c + 32) & 127;
                        tmem_ld_frag_issue(t_s + next, a0);
                        tmem_ld_frag_issue(t_hi + next, a1);
                        scores(c + 1, b0, b1, take_max);
                    }
                    bool grow = false;
#pragma unroll
                    for (int q = 0; q < 4; ++q) grow |= mq[q] > (m_base[q] == -INFINITY ? -INFINITY : slack);
                    if (__any_sync(0xffffffffu, grow)) {
                        float alpha[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {   // the row's maximum is spread over its four lanes
                            float mx = fmaxf(mq[q], __shfl_xor_sync(0xffffffffu, mq[q], 1));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                            const bool fresh = m_base[q] == -INFINITY;
                            const bool up = mx > (fresh ? -INFINITY : slack);
                            alpha[q] = up ? (fresh ? 0.f : fast_exp2(-mx)) : 1.f;
                            l_sum[q] *= alpha[q];
                            if (up) m_base[q] = (fresh ? 0.f : m_base[q]) + mx;
                        }
                        set_base();
                        if (n != g) {   // rescale the rows of O (P.V of the last tile is done); there lane = row
                            float al = 1.f;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float o = __shfl_sync(0xffffffffu, alpha[q], 4 * (lane & 7));
                                if ((lane >> 3) == q) al = o;
                            }
                            tmem_ld_wait(a0, a1);
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                uint32_t o[32];
                                tmem_ld32(t_o + 32 * c, o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                                tmem_st32(t_o + 32 * c, o);
                            }
                        }
                    }
                    // ---- P ----
                    float2 sum[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) sum[q] = make_float2(0.f, 0.f);
#pragma unroll 1
                    for (int c = 0; c < 8; c += 2) {
                        uint32_t pk[2][8];   // 32 tokens as 16 columns, rows 0-15 and 16-31
                        float4 w4 = make_float4(0.f, 0.f, 0.f, 0.f);
                        int half = 0;
                        auto weigh = [&](int q, int i, float2 x) {
                            const float2 pe = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                            sum[q] = __fadd2_rn(sum[q], pe);
                            const float2 w = __fmul2_rn(pe, i ? make_float2(w4.z, w4.w) : make_float2(w4.x, w4.y));
                            pk[q >> 1][2 * (2 * half + i) + (q & 1)] = pack_half2(w.x, w.y);
                        };
                        tmem_ld_wait(a0, a1);
                        tmem_ld_frag_issue(t_s + 16 * c + 16, b0);
                        tmem_ld_frag_issue(t_hi + 16 * c + 16, b1);
                        w4 = *reinterpret_cast<const float4*>(nvs + 16 * c + 4 * (lane & 3));
                        scores(c, a0, a1, weigh);
                        tmem_ld_wait(b0, b1);
                        if (c < 6) {
                            tmem_ld_frag_issue(t_s + 16 * c + 32, a0);
                            tmem_ld_frag_issue(t_hi + 16 * c + 32, a1);
                        }
                        w4 = *reinterpret_cast<const float4*>(nvs + 16 * c + 16 + 4 * (lane & 3));
                        half = 1;
                        scores(c + 1, b0, b1, weigh);
                        tmem_st_frag_issue(t_s + 8 * c, pk[0]);
                        tmem_st_frag_issue(t_hi + 8 * c, pk[1]);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) l_sum[q] += sum[q].x + sum[q].y;
                    tmem_st_wait();
                    }
                }
                tc_fence_before();
                mbar_arrive(bar_p + 8 * g);   // P(n) (and V(n)^T) are stored, the scales and norms read
                named_bar_sync(1 + g, 128);   // (before any thread of the group overwrites the norms)
            }

            // ---- merge the two groups, write the unit's partial ----
            // Group g keeps dims 64 g .. 64 g + 63 of every row and hands the
            // others over through its own V^T tile, 16-byte pieces XORed with the
            // row; the (m, l) pairs go through Q'.
            const bool had = g < s.ntiles;
            if (had) wait(bar_o + 8 * g, (used[g] + ((s.ntiles - 1 - g) >> 1)) & 1);
            const bool late = named_bar_or(3, 256, stalled);
            tc_fence_after();
            if (late) stalled = true;
            if (s.ntiles + pos >= hi || late) griddep_launch_dependents();   // last segment: let the merge launch
            if (!late) {
                float* xch = reinterpret_cast<float*>(sVt);
                float2* sml = reinterpret_cast<float2*>(smem + C::kQOff);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float l = l_sum[q] + __shfl_xor_sync(0xffffffffu, l_sum[q], 1);
                    l += __shfl_xor_sync(0xffffffffu, l, 2);
                    if ((lane & 3) == 0) sml[g * kTok + 32 * (warp & 3) + (lane >> 2) + 8 * q] = make_float2(m_base[q], l);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t v[32];
                    if (had) {
                        tmem_ld32(t_o + 64 * (1 - g) + 32 * c, v);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = 0u;
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4*>(xch + r * 64 + 4 * ((8 * c + e / 4) ^ (r & 15))) =
                            make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
                named_bar_sync(3, 256);
                const float* ox = reinterpret_cast<const float*>(smem + C::kVtOff + (1 - g) * 32768);
                const float2 ml = sml[g * kTok + r], oml = sml[(1 - g) * kTok + r];
                const float M = fmaxf(ml.x, oml.x);
                const float a = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - M);
                const float c2 = oml.x == -INFINITY ? 0.f : fast_exp2(oml.x - M);
                const int unit = s.b * p.per_b + s.ui;
                const size_t slot_row = (static_cast<size_t>(c_me) + unit) * kTreeRows + r;
                float* po = p.part_o + slot_row * kD + 64 * g;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t v[32];
                    if (had) {
                        tmem_ld32(t_o + 64 * g + 32 * c, v);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = 0u;
                    }
                    // (a row that saw no token has weight 0, whatever its columns
                    // hold.)  Column pi(d) holds dim d; pi flips bits 1 and 2 by the
                    // 32-dim block 2g + c, so pairs move as a whole.
                    const int flip = 2 * (2 * g + c);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 o = *reinterpret_cast<const float4*>(ox + r * 64 + 4 * ((8 * c + e / 4) ^ (r & 15)));
                        const float2 y0 = make_float2((a != 0.f ? a * __uint_as_float(v[e]) : 0.f) + (c2 != 0.f ? c2 * o.x : 0.f),
                                                      (a != 0.f ? a * __uint_as_float(v[e + 1]) : 0.f) + (c2 != 0.f ? c2 * o.y : 0.f));
                        const float2 y1 = make_float2((a != 0.f ? a * __uint_as_float(v[e + 2]) : 0.f) + (c2 != 0.f ? c2 * o.z : 0.f),
                                                      (a != 0.f ? a * __uint_as_float(v[e + 3]) : 0.f) + (c2 != 0.f ? c2 * o.w : 0.f));
                        if (row_ok) {
                            *reinterpret_cast<float2*>(po + 32 * c + (e ^ flip)) = y0;
                            *reinterpret_cast<float2*>(po + 32 * c + ((e + 2) ^ flip)) = y1;
                        }
                    }
                }
                if (g == 0 && row_ok)
                    reinterpret_cast<float2*>(p.part_ml)[slot_row] = make_float2(M, a * ml.y + c2 * oml.y);
            }
            bad = end_segment(s);   // Q', the exchange and the tensor memory are free for the next segment
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem0, 512);
}

// A warp per output row: merge the partials of the CTAs over the row's unit by
// their log-sum-exp weights, four at a time, apply v_rescale / l, leave the
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
    auto has = [&](int i) {   // whether CTA c0 + i had chunks at all
        const long long c = c0 + i;
        return i < n && c * all / P < (c + 1) * all / P;
    };
    const size_t row0 = (static_cast<size_t>(c0) + unit) * kTreeRows + r;
    griddep_wait();
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += 4) {
        float2 ml[4];
        float4 o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool u = has(i0 + k);
            const size_t at = row0 + static_cast<size_t>(i0 + k) * kTreeRows;
            ml[k] = u ? __ldcg(reinterpret_cast<const float2*>(p.part_ml) + at) : make_float2(-INFINITY, 0.f);
            o[k] = u ? __ldcg(reinterpret_cast<const float4*>(p.part_o + at * kD) + lane)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float Mn = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
        if (Mn == -INFINITY) continue;
        const float sc = M == -INFINITY ? 0.f : fast_exp2(M - Mn);
        acc.x *= sc; acc.y *= sc; acc.z *= sc; acc.w *= sc;
        den *= sc;
        M = Mn;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (ml[k].x == -INFINITY) continue;
            const float w = fast_exp2(ml[k].x - M);
            den += w * ml[k].y;
            acc.x += w * o[k].x; acc.y += w * o[k].y;
            acc.z += w * o[k].z; acc.w += w * o[k].w;
        }
    }
    float inv = 0.f;
    if (den > 0.f) inv = p.v_rescale / den;
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
    cudaError_t e = set_smem_attr_once(tq_tree_kernel<KB, VB>, C::kSmemAlloc, attr_done);
    if (e != cudaSuccess) return e;
    if (ev0) cudaEventRecord(ev0, stream);
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
