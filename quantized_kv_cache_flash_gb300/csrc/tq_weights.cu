// The softmax weights that cached tokens get from a block of queries
// (tq_attention_weights), on the 5th-generation tensor cores.
//
// Per (batch, KV head) unit the rows are head of the group * tq + query position (as q lies
// in memory), a pair of 128-row query tiles at a time.  A token's sum needs every row's normaliser, so
// the scores are taken twice:
//   stats  S[128 rows x 128 tok] = Q' . K^T     a thread a row: its sum of exp2 (of a base)
//   sum    S[128 tok x 128 rows] = K . Q'^T     a thread a token: sum of exp2(s - lse[row])
// Both orientations read the same tiles (Q' and K are K-major either way), and neither
// needs a value of another lane.  Q' = Rot(q) as q_hi + q_lo (quantized K, whose tile
// holds the fp16 centroids, exact) or q (fp16 K); it is laid out once by a kernel before.
//
// The tiles of all (sequence, pair, KV head) units, laid end to end, are split evenly
// over one CTA per SM; a CTA's run may end one unit and begin the next.  With several
// pairs a token's sums are written per pair and added up by a last kernel, in the
// pairs' order.
//
// Roles of a CTA's warps (hand-overs through mbarriers, every wait bounded):
//   0-3, 4-7  a query tile each: its rows' sums (stats), its part of the tokens' (sum)
//   8-11      dequantise K (n) (quantized K); with a single query tile 4-7 take every second one
//   12, 14    issue the MMAs of every second K tile: the thread that issues stands still while
//             the tensor core works, and the other one's waits are over when it is done
//   13        copies Q' and the records (fp16 K: the tiles)
// Tensor memory: two buffers of 256 columns, S(n) of both query tiles; four of 128 with one.
//
// 8 sequences of 4,000 to 16,384 tokens, 64 queries, 32/8 heads, turbo4 (256 rows a unit): 139 us;
// rows kernel 6.5, stats 68, sums 61.  The products with q_lo and both passes are 190 GFLOP,
// 100 us at the measured rate; what bounds stats is shared memory (an MMA of 128 x 128 x 16
// reads 8 KB, 87 cycles for 64 of the tensor core, beside 32 KB of K stored and its records read
// a tile), what bounds the sums two exponentials a thread and column beside them.  With fp16 K the
// window takes 95 us (K's 167 MB twice).  Two prompts of 2,047 tokens behind up to 511, 28/4 heads,
// fp16 K: 116 us; stats 59, sums 57, the pairs' sum 7, with tensor core 0.41, exponentials 0.38 and
// issue 0.44 active: none is full, each of the roles waits for another; turbo4: 184 us.  8
// sequences of 10,000, 8 KV heads, with 20 to 128 rows (one query tile): 74 to 79 us, 91 to 100 with
// both groups for S; 24 for one sequence of 8,000, of which 18 are launches and the first tile's way
// through the roles.
#include <algorithm>
#include <type_traits>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

constexpr int kWtTile = 128;
constexpr int kWtThreads = 512;

template <int KB>
struct WtCfg {
    static constexpr int kRbK = (KB == 0) ? 256 : KB * 16;
    static constexpr int kSlots = (KB == 0) ? 4 : 2;            // K tiles
    // Q' of the pair: q_hi, q_lo, each 256 rows in the layout of sw128_offset but with
    // halves of 32 KB (dims 0-63, 64-127)
    static constexpr int kParts = (KB == 0) ? 1 : 2;
    static constexpr int kQOff = 0;
    static constexpr int kKOff = kParts * 65536;
    // Records and norms.  With twice as many barriers as stages (an even number) each barrier
    // belongs to one group of dequantising warps, which waits for all of its phases in order;
    // a group that saw every second phase alone could take one for the one two later.
    static constexpr int kStages = (KB == 0) ? 0 : 3, kStgBars = 2 * kStages;
    static constexpr int kStgOff = kKOff + kSlots * 32768;
    static constexpr int kStg = (KB == 0) ? 0 : kWtTile * kRbK + 256;
    static constexpr int kColOff = kStgOff + kStages * kStg;          // fp32 n_k * scale * log2(e) [4][128]
    static constexpr int kLseOff = kColOff + 2048;              // fp32 -log2(sum) of a row [256]
    static constexpr int kPosOff = kLseOff + 1024;              // query position of a row [256]
    static constexpr int kHalfOff = kPosOff + 1024;             // fp32 the second query tile's sums [4][128]
    static constexpr int kSpanOff = kHalfOff + 2048;            // int2 least and largest position of 32 rows [8]
    // S done [4], S read [4], Q' copied, Q' read, K stored [4], K read [4], records copied
    // [kStgBars], records read [kStgBars], the other issuing warp's turn [2]; the TMEM slot
    static constexpr int kGo = 18 + 2 * kStgBars;
    static constexpr int kBarOff = kSpanOff + 64;
    static constexpr int kSmem = kBarOff + (kGo + 2) * 8 + 8;
    static constexpr int kSmemAlloc = kSmem + 768;              // to a 1024-byte boundary from a 256-byte one
    static_assert(kSmemAlloc <= 232448, "227 KB per CTA");
};

// A unit's part of a CTA's run: K tiles [k0, k1) of (sequence b, KV head h, pair).
struct WtSeg {
    int b, h, pair, k0, k1, L;
    int nt, base;   // the unit's tiles, and those of the units before it
};

// x / p.tq and x / p.pairs for 0 <= x < 2^31 (see div_magic)
__device__ __forceinline__ int over_tq(const WeightsParams& p, int x) {
    return static_cast<int>((static_cast<uint64_t>(x) * p.div_tq_m) >> p.div_tq_s);
}
__device__ __forceinline__ int over_pairs(const WeightsParams& p, int x) {
    return static_cast<int>((static_cast<uint64_t>(x) * p.div_pairs_m) >> p.div_pairs_s);
}
// Smallest and largest query position of rows r0 .. r1.
__device__ __forceinline__ int2 wt_span(const WeightsParams& p, int r0, int r1) {
    if (r1 - r0 >= p.tq - 1) return make_int2(0, p.tq - 1);   // (every position)
    const int g0 = over_tq(p, r0), g1 = over_tq(p, r1);
    return g0 == g1 ? make_int2(r0 - g0 * p.tq, r1 - g1 * p.tq) : make_int2(0, p.tq - 1);
}
// K tiles that the rows of a pair see.
__device__ __forceinline__ int wt_tiles(const WeightsParams& p, int L, int pair) {
    const int j_hi = wt_span(p, 256 * pair, min(p.rows, 256 * (pair + 1)) - 1).y;
    const int last = min(min(L, p.max_len) - 1, L - p.tq + j_hi);
    return last < 0 ? 0 : last / kWtTile + 1;
}

// The tiles of all (sequence, pair) groups over the KV heads, by a warp.
__device__ __forceinline__ void wt_total(const WeightsParams& p, int lane, int& all) {
    const int groups = p.batch * p.pairs;
    all = 0;
    for (int g = lane; g < groups; g += 32) {
        const int b = over_pairs(p, g);
        all += p.hkv * wt_tiles(p, p.lengths[b], p.pair0 + g - b * p.pairs);
    }
    all = __reduce_add_sync(0xffffffffu, all);
}

// A CTA's run [pos, hi) of the tiles, unit after unit; each warp keeps its own.
struct WtRun {
    int pos, hi, all;
    int b, pair, h, tile, L, nt;

    __device__ __forceinline__ void enter(const WeightsParams& p) {   // L and nt of (b, pair), past empty ones
        for (; b < p.batch; pair = 0, ++b) {
            L = p.lengths[b];
            for (; pair < p.pairs; ++pair)
                if ((nt = wt_tiles(p, L, p.pair0 + pair)) > 0) return;
        }
    }
    __device__ __forceinline__ void start(const WeightsParams& p, int lane) {
        wt_total(p, lane, all);
        // floor(c * all / P) in 32 bits: c * (all mod P) < P^2
        const int c = static_cast<int>(blockIdx.x), P = static_cast<int>(gridDim.x);
        const int q = all / P, r = all - q * P;
        pos = c * q + c * r / P;
        hi = (c + 1) * q + (c + 1) * r / P;
        b = pair = h = tile = L = nt = 0;
        if (pos >= hi) return;
        // the group that holds pos
        const int groups = p.batch * p.pairs;
        int cum = 0;
        for (int g0 = 0; g0 < groups; g0 += 32) {
            const int g = g0 + lane, bb = min(over_pairs(p, g), p.batch - 1);
            const int n = g < groups ? p.hkv * wt_tiles(p, p.lengths[bb], p.pair0 + g - bb * p.pairs) : 0;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, cum + inc > pos);
            if (hit) {
                const int l = __ffs(hit) - 1;
                const int local = pos - cum - __shfl_sync(0xffffffffu, inc - n, l);
                b = over_pairs(p, g0 + l);
                pair = g0 + l - b * p.pairs;
                enter(p);
                h = local / nt;
                tile = local - h * nt;
                return;
            }
            cum += __shfl_sync(0xffffffffu, inc, 31);
        }
    }
    __device__ __forceinline__ bool next(const WeightsParams& p, WtSeg& s) {
        if (pos >= hi) return false;
        s = WtSeg{b, h, pair, tile, min(nt, tile + hi - pos), L, nt, pos - tile};
        pos += s.k1 - s.k0;
        tile = 0;
        if (++h == p.hkv) {
            h = 0;
            ++pair;
            enter(p);
        }
        return true;
    }
};

// Rot(q) as q_hi and q_lo in the MMA layout (quantized K); a warp a row.
__global__ void __launch_bounds__(256) tq_weights_rows_kernel(const __grid_constant__ WeightsParams p) {
    const int lane = threadIdx.x & 31;
    const int per = p.pairs * 256;
    const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    griddep_wait();
    griddep_launch_dependents();
    const int unit = static_cast<int>(row / per), rl = static_cast<int>(row - static_cast<long long>(unit) * per);
    const int b = unit / p.hkv, h = unit - b * p.hkv, r = p.pair0 * 256 + rl;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < p.rows) {
        const uint2 w = *reinterpret_cast<const uint2*>(
            p.q + ((static_cast<size_t>(b) * p.hq + h * p.group) * p.tq + r) * kD + 4 * lane);
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
        v[0] = f0.x, v[1] = f0.y, v[2] = f1.x, v[3] = f1.y;
        const uint32_t sn = sign_nibble(p.signs, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = ((sn >> i) & 1u) ? -v[i] : v[i];
        wht128_lane4(v, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= 0.08838834764831845f;   // 1/sqrt(128)
    }
    uint8_t* at = p.q_tiles + (static_cast<size_t>(unit) * p.pairs + rl / 256) * 131072 + (lane >> 4) * 32768 +
                  sw128_offset(rl & 255, (4 * lane) & 63);
    const uint2 hi = make_uint2(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]));
    *reinterpret_cast<uint2*>(at) = hi;
    // q_lo = Rot(q) - q_hi (exact in fp32), rounded once more
    const float2 h0 = __half22float2(*reinterpret_cast<const __half2*>(&hi.x));
    const float2 h1 = __half22float2(*reinterpret_cast<const __half2*>(&hi.y));
    *reinterpret_cast<uint2*>(at + 65536) =
        make_uint2(pack_half2(v[0] - h0.x, v[1] - h0.y), pack_half2(v[2] - h1.x, v[3] - h1.y));
}

// SINGLE: one query tile in all (quantized K); its second group of warps dequantises every
// second K tile instead, and two more K tiles lie in its part of Q'.  (fp16 K needs neither:
// 64 units of 10,000 tokens take 31 us a pass, 0.77 of the copy bandwidth.)
template <int KB, bool SUM, bool SINGLE>
__global__ void __launch_bounds__(kWtThreads, 1)
    tq_weights_kernel(const __grid_constant__ WeightsParams p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap qmap) {
    using C = WtCfg<KB>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    float* s_col = reinterpret_cast<float*>(smem + C::kColOff);
    float* s_lse = reinterpret_cast<float*>(smem + C::kLseOff);
    int* s_pos = reinterpret_cast<int*>(smem + C::kPosOff);
    float* s_half = reinterpret_cast<float*>(smem + C::kHalfOff);
    int2* s_span = reinterpret_cast<int2*>(smem + C::kSpanOff);
    const uint32_t bar_s = smem_u32(smem + C::kBarOff), bar_sf = bar_s + 32, bar_q = bar_s + 64, bar_qf = bar_s + 72,
                   bar_k = bar_s + 80, bar_kf = bar_s + 112, bar_stg = bar_s + 144, bar_stgf = bar_stg + 8 * C::kStgBars,
                   bar_go = bar_s + 8 * C::kGo;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + (C::kGo + 2) * 8);
    constexpr bool single = SINGLE;
    constexpr int readers = single ? 128 : 256;   // threads that read S
    constexpr int NS = KB == 0 || single ? 4 : 2, slot_bits = NS == 4 ? 2 : 1;   // K tiles
    constexpr int NB = single ? 4 : 2, buf_bits = single ? 2 : 1;   // buffers of S, 128 columns a query tile
    auto k_half = [&](int slot, int half) {   // dims 0-63 or 64-127 of a K tile
        return KB != 0 && slot >= 2 ? C::kQOff + 16384 + (slot - 2) * 65536 + half * 32768
                                    : C::kKOff + slot * 32768 + half * 16384;
    };
    if (tid == 0) {
        for (int i = 0; i < C::kStgBars; ++i) {
            mbar_init(bar_stg + 8 * i, 1);
            mbar_init(bar_stgf + 8 * i, 128);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar_s + 8 * i, 1);
            mbar_init(bar_sf + 8 * i, readers);
        }
        for (int i = 0; i < 2; ++i) mbar_init(bar_go + 8 * i, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar_k + 8 * i, KB == 0 ? 1 : 128);
            mbar_init(bar_kf + 8 * i, 1);
        }
        mbar_init(bar_q, 1);
        mbar_init(bar_qf, 2);
        fence_barrier_init();
    }
    if (KB == 0 && tid == 0) {
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&qmap);
    }
    // What each kernel reads of the ones before: stats Q' (quantized K), the sums part_ml; the warps
    // that do so wait there, the others begin at once.  (The caller's data may be read before:
    // the first kernel waited for what wrote them before any of its CTAs let the next grid
    // launch, and so did stats for Q'.)
    constexpr bool kWaitFirst = KB == 0 && !SUM;
    if constexpr (kWaitFirst) {
        griddep_wait();
        griddep_launch_dependents();
    }
    if (!SUM && p.pair0 == 0 && blockIdx.x == 0 && warp == 15) {   // rows that see no token
        bool none = false;
        for (int b = lane; b < p.batch; b += 32) none = none || p.lengths[b] < p.tq;
        if (none) atomicOr(p.status, kStatusShortContext);
    }
    WtRun run;
    run.start(p, lane);
    if (run.pos >= run.hi) {   // (uniform over the CTA; nothing allocated yet)
        if (!kWaitFirst) griddep_wait();
        return;
    }
    if (warp == 0) tmem_alloc(smem_u32(tslot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    int ring = 0;           // n % kStgBars, and n / kStgBars
    uint32_t round = 0;
    auto next_stage = [&] {
        if (++ring == C::kStgBars) ring = 0, ++round;
    };
    auto stage_at = [&] { return C::kStgOff + (ring < C::kStages ? ring : ring - C::kStages) * C::kStg; };

    bool stalled = false;  // once set, waits return at once and no MMA or copy is issued
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!stalled && !mbar_wait_bounded(bar, parity)) stalled = true;
    };
    int n = 0;             // K tiles so far, over the units
    WtSeg s;
    if (warp < 4 || (warp < 8 && !single)) {
        const int wg = warp >> 2, r = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        if constexpr (SUM) {
            griddep_wait();
            griddep_launch_dependents();
        }
        while (run.next(p, s)) {
            const int lim = min(s.L, p.max_len);
            const int row0 = (p.pair0 + s.pair) * 256;            // the pair's first row
            const int unit = (s.b * p.pairs + s.pair) * p.hkv + s.h;
            if constexpr (SUM) {
                const int nrows = min(256, p.rows - row0);
                named_bar_sync(1, readers);   // (the unit before is done with its values)
                // the row's partial sums joined
                {
                    const int P = static_cast<int>(gridDim.x), q = run.all / P, rest = run.all - q * P;
                    const uint64_t all = run.all;
                    const int c0 = static_cast<int>(((s.base + 1ull) * P - 1) / all);
                    const int c1 = static_cast<int>(((s.base + 0ull + s.nt) * P - 1) / all);
                    const float2* ml = p.part_ml + static_cast<size_t>(unit) * 256 + tid;
                    float M = -INFINITY, sum = 0.f;
                    for (int c = c0; c <= c1; c += 8) {   // (eight loads in flight)
                        float2 x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            x[i] = make_float2(-INFINITY, 0.f);
                            // (an empty run wrote nothing)
                            if (c + i <= c1 && !(q == 0 && (c + i) * rest / P == (c + i + 1) * rest / P))
                                x[i] = __ldcg(ml + static_cast<size_t>(c + i) * 256);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float mn = fmaxf(M, x[i].x);
                            sum = (M == -INFINITY ? sum : sum * fast_exp2(M - mn)) +
                                  (x[i].x == -INFINITY ? x[i].y : x[i].y * fast_exp2(x[i].x - mn));
                            M = mn;
                        }
                    }
                    float neg = -(M + log2f(sum));
                    if (neg == INFINITY) {   // all its scores are -inf: it adds nothing, as one that sees no token
                        neg = -INFINITY;
                        if (tid < nrows) atomicOr(p.status, kStatusShortContext);
                    }
                    s_lse[tid] = neg;
                    // (a row without any token is behind every token's first position)
                    const int at = tid < nrows ? row0 + tid - over_tq(p, row0 + tid) * p.tq : -0x7fffffff - 1;
                    s_pos[tid] = at;
                    const int least = __reduce_min_sync(0xffffffffu, at), most = __reduce_max_sync(0xffffffffu, at);
                    if (lane == 0) s_span[tid >> 5] = make_int2(least, most);
                }
                named_bar_sync(1, readers);
                // tokens that every row of the pair sees
                const int all_see = s.L - p.tq + wt_span(p, row0, row0 + nrows - 1).x;
                const int seen = p.seen != nullptr ? p.seen[s.b] : s.L - p.tq;
                const int here = min(128, nrows - 128 * wg);   // rows of this query tile (or below 1)
                float* const out = p.part_w != nullptr
                                       ? p.part_w + (static_cast<size_t>(s.b * p.hkv + s.h) * p.pairs + s.pair) * p.part_len
                                       : p.weights + static_cast<size_t>(s.b * p.hkv + s.h) * p.cap;
                float before = 0.f, old = 0.f;   // the tile before's sum and weight so far
                auto put = [&](int m, int t, float w) {   // token t's sum, of tile number m
                    if (!single) {
                        named_bar_sync(2 + (m & 3), 256);
                        w += s_half[128 * (m & 3) + r];
                    }
                    if (t >= lim || stalled) return;
                    out[t] = w + p.decay * old;
                };
                const float* lse = s_lse + 128 * wg;
                const int* pos = s_pos + 128 * wg;
                for (int k = s.k0; k < s.k1; ++k, ++n) {
                    const int buf = n & (NB - 1), t = k * kWtTile + r;
                    // (in flight while S is waited for)
                    const bool more = wg == 0 && p.part_w == nullptr && t < min(seen, lim) && p.decay != 0.f;
                    const float now = more ? out[t] : 0.f;
                    wait(bar_s + 8 * buf, (n >> buf_bits) & 1);
                    tc_fence_after();
                    const float c = KB == 0 ? p.scale_log2e : s_col[128 * buf + r];
                    const uint32_t d = tmem + 512 / NB * buf + 128 * wg + lane_off;
                    const int from = t - (s.L - p.tq);   // the first query position that sees the token
                    const float2 cc = make_float2(c, c);
                    float2 a[4] = {};
                    auto add = [&](const uint32_t* f, int x, auto masked) {   // rows x .. x + 31
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 l = *reinterpret_cast<const float4*>(lse + x + e);
                            const float2 y0 = __ffma2_rn(make_float2(__uint_as_float(f[e]), __uint_as_float(f[e + 1])), cc,
                                                         make_float2(l.x, l.y));
                            const float2 y1 = __ffma2_rn(make_float2(__uint_as_float(f[e + 2]), __uint_as_float(f[e + 3])),
                                                         cc, make_float2(l.z, l.w));
                            float2 z0 = make_float2(fast_exp2(y0.x), fast_exp2(y0.y));
                            float2 z1 = make_float2(fast_exp2(y1.x), fast_exp2(y1.y));
                            if constexpr (decltype(masked)::value) {
                                const int4 j = *reinterpret_cast<const int4*>(pos + x + e);
                                if (j.x < from) z0.x = 0.f;
                                if (j.y < from) z0.y = 0.f;
                                if (j.z < from) z1.x = 0.f;
                                if (j.w < from) z1.y = 0.f;
                            }
                            a[(e >> 1) & 3] = __fadd2_rn(a[(e >> 1) & 3], z0);
                            a[((e >> 1) & 3) + 1] = __fadd2_rn(a[((e >> 1) & 3) + 1], z1);
                        }
                    };
                    if (k * kWtTile + kWtTile - 1 <= all_see && here == 128) {
                        uint32_t v[2][32];   // the next 32 rows in flight
                        tmem_ld32_issue(d, v[0]);
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            tmem_ld_wait(v[x & 1]);
                            if (x < 3) tmem_ld32_issue(d + 32 * (x + 1), v[(x + 1) & 1]);
                            add(v[x & 1], 32 * x, std::false_type{});
                        }
                    } else {   // all of the warp's tokens are seen by 32 rows, none is, or each row says which
#pragma unroll 1
                        for (int x = 0; x < here; x += 32) {
                            const int2 span = s_span[4 * wg + x / 32];   // (padding rows: -2^31)
                            if (span.y < from - lane) continue;
                            uint32_t v[32];
                            tmem_ld32(d + x, v);
                            if (span.x >= 0 && span.x >= from - lane + 31) add(v, x, std::false_type{});
                            else add(v, x, std::true_type{});
                        }
                    }
                    const float2 t2 = __fadd2_rn(__fadd2_rn(a[0], a[1]), __fadd2_rn(a[2], a[3]));
                    const float w = t2.x + t2.y;
                    tc_fence_before();
                    mbar_arrive(bar_sf + 8 * buf);
                    // the second query tile's part goes to the first one's thread, which looks for
                    // it a tile later (four slots: S(n + 4) waits for what the first group does
                    // after it has read this one)
                    if (wg == 1) {
                        s_half[128 * (n & 3) + r] = w;
                        __threadfence_block();
                        named_bar_arrive(2 + (n & 3), 256);
                    } else {
                        if (k > s.k0) put(n - 1, t - kWtTile, before);
                        before = w;
                        old = now;
                    }
                }
                if (wg == 0) put(n - 1, (s.k1 - 1) * kWtTile + r, before);
            } else {
                // rows of query tile wg: last visible token of this row, and of all of them
                const int first = row0 + 128 * wg, row = first + r;
                const int mine = row < p.rows ? min(s.L - p.tq + row - over_tq(p, row) * p.tq, lim - 1) : -1;
                const bool live = row < p.rows;
                // over the warp's rows: the last token that all see, and that one sees
                const int lo = __reduce_min_sync(0xffffffffu, live ? mine : 0x7fffffff);
                const int hi = __reduce_max_sync(0xffffffffu, mine);
                // A row's base m is the largest score of the tile that it first sees; later
                // scores may pass it, as long as the sums stay in range.
                float m = -INFINITY, l = 0.f;
                for (int k = s.k0; k < s.k1; ++k, ++n) {
                    const int buf = n & (NB - 1);
                    wait(bar_s + 8 * buf, (n >> buf_bits) & 1);
                    tc_fence_after();
                    const uint32_t d = tmem + 512 / NB * buf + 128 * wg + lane_off;
                    const float* col = s_col + 128 * buf;
                    const int tok0 = k * kWtTile;
                    const int visible = hi < tok0 ? 0 : min(4, (hi - tok0) / 32 + 1);   // pieces of 32 tokens
                    bool slow = __any_sync(0xffffffffu, live && m == -INFINITY && mine >= tok0);
                    if (visible > 0 && !slow) {
                        const float base = m == -INFINITY ? 0.f : m;
                        const float2 nb = make_float2(-base, -base);
                        float2 a[4] = {};
                        auto add = [&](const uint32_t* f, int x, auto masked) {   // tokens x .. x + 31 of the tile
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 c = KB == 0 ? make_float4(p.scale_log2e, p.scale_log2e, p.scale_log2e,
                                                                       p.scale_log2e)
                                                         : *reinterpret_cast<const float4*>(col + x + e);
                                float2 y0 = __ffma2_rn(make_float2(__uint_as_float(f[e]), __uint_as_float(f[e + 1])),
                                                       make_float2(c.x, c.y), nb);
                                float2 y1 = __ffma2_rn(make_float2(__uint_as_float(f[e + 2]), __uint_as_float(f[e + 3])),
                                                       make_float2(c.z, c.w), nb);
                                if constexpr (decltype(masked)::value) {
                                    const int left = mine - (tok0 + x + e);
                                    if (left < 0) y0.x = -INFINITY;
                                    if (left < 1) y0.y = -INFINITY;
                                    if (left < 2) y1.x = -INFINITY;
                                    if (left < 3) y1.y = -INFINITY;
                                }
                                a[(e >> 1) & 3] = __fadd2_rn(a[(e >> 1) & 3], make_float2(fast_exp2(y0.x), fast_exp2(y0.y)));
                                a[((e >> 1) & 3) + 1] =
                                    __fadd2_rn(a[((e >> 1) & 3) + 1], make_float2(fast_exp2(y1.x), fast_exp2(y1.y)));
                            }
                        };
                        if (tok0 + kWtTile - 1 <= lo) {
                            uint32_t v[2][32];   // the next 32 tokens in flight
                            tmem_ld32_issue(d, v[0]);
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                tmem_ld_wait(v[x & 1]);
                                if (x < 3) tmem_ld32_issue(d + 32 * (x + 1), v[(x + 1) & 1]);
                                add(v[x & 1], 32 * x, std::false_type{});
                            }
                        } else {
#pragma unroll 1
                            for (int x = 0; x < 32 * visible; x += 32) {
                                uint32_t v[32];
                                tmem_ld32(d + x, v);
                                if (tok0 + x + 31 <= lo) add(v, x, std::false_type{});
                                else add(v, x, std::true_type{});
                            }
                        }
                        const float2 t2 = __fadd2_rn(__fadd2_rn(a[0], a[1]), __fadd2_rn(a[2], a[3]));
                        const float sum = t2.x + t2.y;
                        slow = __any_sync(0xffffffffu, live && !(sum < 1.2676506e30f));   // 2^100 (or NaN)
                        if (!slow) l += sum;
                    }
                    if (slow) {
#pragma unroll 1
                        for (int x = 0; x < 128; x += 32) {
                            uint32_t v[32];
                            tmem_ld32(d + x, v);
                            float mx = -INFINITY;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                float y = __uint_as_float(v[e]) * (KB == 0 ? p.scale_log2e : col[x + e]);
                                if (tok0 + x + e > mine) y = -INFINITY;
                                mx = fmaxf(mx, y);
                                v[e] = __float_as_uint(y);
                            }
                            if (mx > m) {
                                l *= m == -INFINITY ? 1.f : fast_exp2(m - mx);   // (l is 0 there, or NaN)
                                m = mx;
                            }
                            const float base = m == -INFINITY ? 0.f : m;
                            float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int e = 0; e < 32; ++e) a[e & 3] += fast_exp2(__uint_as_float(v[e]) - base);
                            l += (a[0] + a[1]) + (a[2] + a[3]);
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(bar_sf + 8 * buf);
                }
                p.part_ml[(static_cast<size_t>(blockIdx.x) + unit) * 256 + 128 * wg + r] = make_float2(m, l);
            }
        }
    } else if (warp < 12) {
        if constexpr (KB != 0) {   // a token a thread
            const int r = tid & 127, other = warp < 8 ? 0 : 1;   // (single: the tiles of the other group)
            const Tables kt{p.ktab[0], p.ktab[1], p.ktab[2], p.ktab[3]};
            while (run.next(p, s)) {
                const int lim = min(s.L, p.max_len);
                for (int k = s.k0; k < s.k1; ++k, ++n, next_stage()) {
                    const int buf = n & (NB - 1);
                    if (single && (n & 1) == other) continue;
                    const uint8_t* stg = smem + stage_at();
                    const int slot = n & (NS - 1);
                    wait(bar_stg + 8 * ring, round & 1);
                    if (n >= NS) wait(bar_kf + 8 * slot, ((n >> slot_bits) - 1) & 1);
                    // the quarters in an order that differs between lanes whose records
                    // start in the same banks
                    const int turn = KB == 4 ? r >> 1 : r >> 3;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        const int side = (q + turn) & 3;
                        uint8_t* sK = smem + k_half(slot, side >> 1);
                        uint32_t hh[16];
                        dequant_q32<KB>(stg + r * C::kRbK + side * (C::kRbK / 4), kt, hh);
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            *reinterpret_cast<uint4*>(sK + sw128_offset(r, 32 * (side & 1) + 8 * m)) =
                                make_uint4(hh[4 * m], hh[4 * m + 1], hh[4 * m + 2], hh[4 * m + 3]);
                    }
                    const float nk = __half2float(reinterpret_cast<const __half*>(stg + kWtTile * C::kRbK)[r]);
                    mbar_arrive(bar_stgf + 8 * ring);
                    if (n >= NB) wait(bar_sf + 8 * buf, ((n >> buf_bits) - 1) & 1);   // the scales of n - NB are read
                    s_col[128 * buf + r] = k * kWtTile + r < lim ? nk * p.scale_log2e : 0.f;
                    fence_proxy_async();
                    mbar_arrive(bar_k + 8 * slot);
                }
            }
        }
    } else if (warp == 12 || warp == 14) {
        const bool one = lane == 0;
        const int odd = warp == 14;
        int seg = 0, last = -1;   // units so far; the last tile issued
        while (run.next(p, s)) {
            if (!one) continue;
            const int tiles = (p.pair0 + s.pair) * 256 + 128 < p.rows ? 2 : 1;   // query tiles with rows
            wait(bar_q, seg++ & 1);
            for (int k = s.k0; k < s.k1; ++k, ++n) {
                const int buf = n & (NB - 1), slot = n & (NS - 1);
                if ((n & 1) != odd) continue;
                wait(bar_k + 8 * slot, (n >> slot_bits) & 1);
                if (n >= NB) wait(bar_sf + 8 * buf, ((n >> buf_bits) - 1) & 1);
                // in turns, so that tile n is done while n + 1 is worked on; the other warp's
                // begins a little before the end of this one's
                if (n > 0) wait(bar_go + 8 * odd, ((n - 1) >> 1) & 1);
                if (stalled) break;
                tc_fence_after();
                const uint32_t k0 = smem_u32(smem) + k_half(slot, 0), k1 = smem_u32(smem) + k_half(slot, 1);
                const uint32_t qbase = smem_u32(smem + C::kQOff), d = tmem + 512 / NB * buf;
                // q_lo first: the sums are cut at every step, the less the smaller they are
                if constexpr (SUM) {   // both query tiles at once
                    const uint32_t idesc = umma_idesc_f16_f32(128, single ? (p.rows + 15) / 16 * 16 : tiles == 2 ? 256 : 128);
#pragma unroll
                    for (int part = C::kParts - 1; part >= 0; --part)
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            if (part == 0 && kk == 6) mbar_arrive(bar_go + 8 * (odd ^ 1));
                            umma_f16(d, umma_desc_sw128((kk < 4 ? k0 : k1) + (kk & 3) * 32),
                                     umma_desc_sw128(qbase + part * 65536 + (kk >> 2) * 32768 + (kk & 3) * 32), idesc,
                                     kk > 0 || part + 1 < C::kParts ? 1u : 0u);
                        }
                } else {
#pragma unroll 1
                    for (int t = 0; t < tiles; ++t)
#pragma unroll
                        for (int part = C::kParts - 1; part >= 0; --part)
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {
                                if (part == 0 && kk == 4 && t == tiles - 1) mbar_arrive(bar_go + 8 * (odd ^ 1));
                                umma_f16(d + 128 * t,
                                         umma_desc_sw128(qbase + part * 65536 + (kk >> 2) * 32768 + t * 16384 + (kk & 3) * 32),
                                         umma_desc_sw128((kk < 4 ? k0 : k1) + (kk & 3) * 32),
                                         umma_idesc_f16_f32(128, 128), kk > 0 || part + 1 < C::kParts ? 1u : 0u);
                            }
                }
                umma_commit(bar_s + 8 * buf);
                umma_commit(bar_kf + 8 * slot);
                last = n;
            }
            if (stalled) break;
            umma_commit(bar_qf);
        }
        // after a time-out: the MMAs in flight end before tensor memory is freed
        if (one && stalled && last >= 0) (void)mbar_wait_bounded(bar_kf + 8 * (last & (NS - 1)), (last >> slot_bits) & 1);
        __syncwarp();
    } else if (warp == 13) {
        const bool one = lane == 0;
        int seg = 0, begun = 0;   // tiles whose copies were issued
        bool q_open = false;
        if constexpr (!SUM && !kWaitFirst) {
            griddep_wait();
            griddep_launch_dependents();
        }
        while (run.next(p, s)) {
            if (!one) continue;
            const int lim = min(s.L, p.max_len);
            const size_t row0 = static_cast<size_t>(s.b * p.hkv + s.h) * p.cap;
            const int unit_q = s.b * p.hkv + s.h;
            const int tiles = (p.pair0 + s.pair) * 256 + 128 < p.rows ? 2 : 1;
            // Q' once the MMAs of the unit before, of both issuing warps, have read theirs
            if (seg > 0) wait(bar_qf, (seg - 1) & 1);
            if (stalled) break;
            mbar_arrive_expect_tx(bar_q, tiles * C::kParts * 32768);
            if constexpr (KB == 0) {
                // q itself (rows past the unit's are other heads', or zeros; masked later)
                const int at = (s.b * p.hq + s.h * p.group) * p.tq + (p.pair0 + s.pair) * 256;
                for (int t = 0; t < tiles; ++t)
                    for (int half = 0; half < 2; ++half)
                        tma_g2s_2d(smem_u32(smem + C::kQOff) + half * 32768 + t * 16384, &qmap, half * 64, at + 128 * t,
                                   bar_q);
            } else {
                for (int x = 0; x < 4; ++x)   // parts and halves
                    bulk_g2s(smem_u32(smem + C::kQOff) + x * 32768,
                             p.q_tiles + (static_cast<size_t>(unit_q) * p.pairs + s.pair) * 131072 + x * 32768,
                             tiles * 16384, bar_q);
            }
            ++seg;
            q_open = true;
            for (int k = s.k0; k < s.k1; ++k, ++n) {
                const int tok0 = k * kWtTile;
                if constexpr (KB == 0) {
                    const int slot = n & (NS - 1);
                    if (n >= NS) wait(bar_kf + 8 * slot, ((n >> slot_bits) - 1) & 1);
                    if (stalled) break;
                    mbar_arrive_expect_tx(bar_k + 8 * slot, 32768);
                    // (rows past the tensor's end are zero-filled; masked later)
                    for (int half = 0; half < 2; ++half)
                        for (int rb = 0; rb < 4; ++rb)
                            tma_g2s_2d(smem_u32(smem) + k_half(slot, half) + rb * 4096, &kmap,
                                       half * 64, static_cast<int32_t>(row0 + tok0 + rb * 32), bar_k + 8 * slot);
                } else {
                    // tile n - kStages, in the same stage, is read
                    if (ring >= C::kStages) wait(bar_stgf + 8 * (ring - C::kStages), round & 1);
                    else if (round > 0) wait(bar_stgf + 8 * (ring + C::kStages), (round - 1) & 1);
                    if (stalled) break;
                    const int nval = min(kWtTile, lim - tok0);
                    const uint32_t nb = static_cast<uint32_t>((nval + 7) & ~7) * 2;
                    const uint32_t dst = smem_u32(smem) + stage_at(), bar = bar_stg + 8 * ring;
                    mbar_arrive_expect_tx(bar, nval * C::kRbK + nb);
                    bulk_g2s(dst, p.k_codes + (row0 + tok0) * C::kRbK, nval * C::kRbK, bar);
                    bulk_g2s(dst + kWtTile * C::kRbK, p.k_norm + row0 + tok0, nb, bar);
                    next_stage();
                }
                ++begun;
            }
            if (stalled) break;
        }
        // (after a time-out: the copies in flight land before shared memory goes away)
        if (one && stalled) {
            if (q_open) (void)mbar_wait_bounded(bar_q, (seg - 1) & 1);
            constexpr int flight = KB == 0 ? NS : C::kStages, bars = KB == 0 ? NS : C::kStgBars;
            for (int x = max(begun - flight, 0); x < begun; ++x)
                (void)mbar_wait_bounded((KB == 0 ? bar_k : bar_stg) + 8 * (x % bars), (x / bars) & 1);
        }
        // (the last commits have arrived before shared memory goes away)
        if (one && !stalled) wait(bar_qf, (seg - 1) & 1);
        __syncwarp();
    }
    tc_fence_before();
    if (__syncthreads_or(stalled) && tid == 0) atomicOr(p.status, kStatusPipelineStall);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// A token's sums over the pairs that see it, added to its weight: 32 tokens a CTA, its
// warps taking every eighth pair.
__global__ void __launch_bounds__(256) tq_weights_add_kernel(const __grid_constant__ WeightsParams p) {
    __shared__ float s_sum[8][32];
    const int per = p.part_len / 32;
    const int unit = static_cast<int>(blockIdx.x) / per, t0 = (static_cast<int>(blockIdx.x) - unit * per) * 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = t0 + lane;
    griddep_wait();
    griddep_launch_dependents();
    const int b = unit / p.hkv, L = p.lengths[b], lim = min(L, p.max_len);
    if (t0 >= lim) return;
    const float* part = p.part_w + static_cast<size_t>(unit) * p.pairs * p.part_len + t;
    float sum = 0.f;
#pragma unroll 4
    for (int q = warp; q < p.pairs; q += 8)
        if (t0 / kWtTile < wt_tiles(p, L, p.pair0 + q)) sum += __ldcg(part + static_cast<size_t>(q) * p.part_len);
    s_sum[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || t >= lim) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += s_sum[i][lane];
    const int seen = p.seen != nullptr ? p.seen[b] : L - p.tq;
    float* out = p.weights + static_cast<size_t>(unit) * p.cap + t;
    float old = 0.f;
    if (p.pair0 > 0) old = *out;   // (a call in several blocks of pairs)
    else if (t < seen && p.decay != 0.f) old = p.decay * *out;
    *out = old + sum;
}

template <int KB, bool SINGLE>
static int launch_t(const WeightsParams& p, const CUtensorMap* kmap, const CUtensorMap* qmap, cudaStream_t stream) {
    using C = WtCfg<KB>;
    static std::atomic<uint64_t> done0{0}, done1{0};
    cudaError_t e = set_smem_attr_once(tq_weights_kernel<KB, false, SINGLE>, C::kSmemAlloc, done0);
    if (e == cudaSuccess) e = set_smem_attr_once(tq_weights_kernel<KB, true, SINGLE>, C::kSmemAlloc, done1);
    if (e != cudaSuccess) return e;
    const unsigned units = static_cast<unsigned>(p.batch) * p.hkv;
    if (KB != 0) e = launch_pdl(tq_weights_rows_kernel, dim3(units * p.pairs * 32), dim3(256), 0, stream, p);
    if (e == cudaSuccess)
        e = launch_pdl(tq_weights_kernel<KB, false, SINGLE>, dim3(p.ctas), dim3(kWtThreads), C::kSmemAlloc, stream, p, *kmap, *qmap);
    if (e == cudaSuccess)
        e = launch_pdl(tq_weights_kernel<KB, true, SINGLE>, dim3(p.ctas), dim3(kWtThreads), C::kSmemAlloc, stream, p, *kmap, *qmap);
    if (e == cudaSuccess && p.part_w != nullptr)
        e = launch_pdl(tq_weights_add_kernel, dim3(units * (p.part_len / 32)), dim3(256), 0, stream, p);
    return e;
}

int launch_weights(int kbits, const WeightsParams& p, const CUtensorMap* kmap, const CUtensorMap* qmap,
                   cudaStream_t stream) {
    const bool single = p.rows <= 128;
    if (kbits == 16) return launch_t<0, false>(p, kmap, qmap, stream);
    if (kbits == 3) return single ? launch_t<3, true>(p, kmap, qmap, stream) : launch_t<3, false>(p, kmap, qmap, stream);
    if (kbits == 4) return single ? launch_t<4, true>(p, kmap, qmap, stream) : launch_t<4, false>(p, kmap, qmap, stream);
    return cudaErrorInvalidValue;
}

}  // namespace tq
