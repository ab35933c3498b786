// Prefill attention over packed sequences on the 5th-generation tensor cores
// (tcgen05, accumulators in tensor memory): the prompts of a batch, each of its own
// length, laid end to end in q and out without padding.
//
// Query j of a sequence's n attends to its tokens [0, L - n + j]; scores and P.V are
// taken in the rotated basis and only the output is rotated back:
//   S[128 rows x 128 tok]  = Q'[128 x 128] . K^T     (8 or 16 MMAs of K = 16, fp32 in TMEM)
//   O[128 rows x 128 dim] += P[128 x 128 tok] . V    (8 MMAs, fp32 in TMEM)
// Q' = Rot(q) as q_hi + q_lo (quantized K, whose tile holds the fp16 centroids,
// exact) or q itself (fp16 K); the softmax scale and the K norm are applied to the
// fp32 scores.  P takes the V norm and is rounded to fp16 once; the V tile holds
// the exact centroids.
//
// A CTA takes two 128-row query tiles of one sequence and KV head, so a K/V tile is
// dequantised once for 256 rows.  Its warps have roles and hand over through
// mbarriers (every wait bounded):
//   0-3, 4-7   the query tiles' rows: Q', the softmax of tile n, the output
//   8-11       dequantise: K(n) once both S(n - 1) have read K(n - 1), the norms once
//              both softmaxes(n - 1) are done, V(n)^T once both P.V(n - 1) are
//   12, 13     issue S_0, S_1 and P.V_0, P.V_1: each waits for its operands alone, and
//              the tensor core takes what is ready
//   14         copies the records of tile n + 2 into the slot of tile n (bulk copies;
//              fp16 K by tensor map straight into the MMA layout)
// Tensor memory: per query tile S (128 columns, whose first 64 take P back as fp16
// pairs) and O (128 columns), all 512.
//
// What bounds it: per tile, the chain of a query tile's S, softmax and P.V (they take
// turns on one S / P buffer; tensor memory is full) and the tensor core.  Quantized K:
// 48 MMAs and the chain 1750 + 1700 + 900 cycles, with 250 of hand-overs between, in a
// period of 4850; fp16 K: 32 MMAs, 1150 + 1700 + 900 in 3900.  Around the loop a CTA
// takes some 18000 cycles for its item, Q' and the output.  Measured: 12 prompts of 64 to
// 4096 tokens, turbo4, 32 / 8 heads, 439 us (608 TFLOP/s, q_lo's products not counted);
// three chunks of 2047 to 8192 tokens behind up to 8191, fp16 K, 28 / 4 heads, 1604 us
// (1.15 PFLOP/s); three prompts of 17 to 300 tokens 21 us.  With two groups of warps that
// dequantise and issue for themselves the same calls took 541, 2255 and 25 us: the
// thread that issues stands still while the tensor core works (600 to 1500 cycles a
// product), as does the one that starts the copies (1000 a tile).
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

template <int KB, int VB>
struct PackCfg {
    static constexpr int kTile = 128;                           // tokens per tile, rows per query tile
    static constexpr int kRbK = (KB == 0) ? 256 : KB * 16;
    static constexpr int kRbV = VB * 16;
    static constexpr int kQOff = 0;                             // fp16 Q' (q_hi) of the two query tiles (64 KB)
    static constexpr int kVtOff = 65536;                        // fp16 V^T [dim][token] (32 KB)
    static constexpr int kKOff = 98304;                         // fp16 K [token][dim] (quantized K)
    static constexpr int kQloOff = kKOff + 32768;               // fp16 q_lo of the two tiles (quantized K, 64 KB)
    static constexpr int kStgOff = (KB == 0) ? kKOff : kQloOff + 65536;
    // staging slot: K (fp16 K: the MMA tile itself, 32 KB; else records), K norms, V records, V norms
    static constexpr int kSK = (KB == 0) ? 32768 : kTile * kRbK;
    static constexpr int kSKn = (KB == 0) ? 0 : kTile * 2;
    static constexpr int kSV = kTile * kRbV;
    static constexpr int kSVn = kTile * 2;
    static constexpr int kSlotRaw = kSK + kSKn + kSV + kSVn;
    // (fp16 K is read by the MMA straight from the slot: 1024-byte aligned)
    static constexpr int kSlotAlign = (KB == 0) ? 1024 : 128;
    static constexpr int kSlot = (kSlotRaw + kSlotAlign - 1) / kSlotAlign * kSlotAlign;
    static constexpr int kColOff = kStgOff + 2 * kSlot;         // fp32 n_k * scale * log2(e) [128]
    static constexpr int kNvOff = kColOff + kTile * 4;          // fp32 n_v [128], fp16 largest n_v of 32 [4]
    // mbarriers: records copied [2], slot free [2], S done [2], P.V done [2], P stored
    // [2], K stored (dims 0-63, 64-127), scales stored, V stored, Q' stored, K's dims
    // 0-63 read; the TMEM slot
    static constexpr int kBarOff = kNvOff + kTile * 4 + 8;
    static constexpr int kSmem = kBarOff + 16 * 8 + 4;
    static constexpr int kSmemAlloc = kSmem + 768;              // to a 1024-byte boundary from a 256-byte one
    static_assert(kSmemAlloc <= 232448, "227 KB per CTA");
    static constexpr uint32_t kIdesc = umma_idesc_f16_f32(128, 128);
};

constexpr int kPackThreads = 512;
constexpr int kRegsLaunch = 128, kRegsSoftmax = 184, kRegsOther = 72;
static_assert(2 * kRegsSoftmax + 2 * kRegsOther <= 4 * kRegsLaunch, "within the launch's registers");

// Which query tile pair a CTA takes.  All pairs of all sequences are ranked by the
// K/V tiles they read, most first (the grid then ends on the shortest ones), and
// rank k of every KV head goes to the CTAs k hkv .. k hkv + hkv - 1, so CTAs that
// start together read different KV heads of the same tokens.  A pair's tile count
// grows with its place in the sequence, so the pairs of a sequence that read more
// than c tiles are its last ones, and their number is one division; the smallest c
// that leaves at most k pairs above it is found by bisection, one warp adding the
// sequences up.
struct PackedSeq {
    int n, ctx, lim;   // query rows, tokens before them, tokens read at most
    int first, all;    // first row, pairs
};

// x / p.span for 0 <= x: the product with 2^32 / span rounded up is at most one off
__device__ __forceinline__ int over_span(const PrefillParams& p, int x) {
    const int q = static_cast<int>(__umulhi(static_cast<uint32_t>(x), p.span_inv));
    return q * static_cast<int64_t>(p.span) > x ? q - 1 : q;
}

__device__ __forceinline__ PackedSeq packed_seq(const PrefillParams& p, int b) {
    PackedSeq s{0, 0, 0, 0, 0};
    if (b >= p.batch) return s;
    const int first = p.cu[b], next = p.cu[b + 1], L = p.lengths[b];
    if (first < 0 || next < first || next > p.total) return s;   // no rows (flagged by the first CTA)
    s.first = first;
    s.n = next - first;
    s.ctx = L - s.n;
    s.lim = min(L, p.max_len);
    s.all = s.n > 0 ? over_span(p, s.n - 1) + 1 : 0;
    return s;
}

// Pairs of a sequence that read more than c >= 0 tiles.
__device__ __forceinline__ int pairs_above(const PrefillParams& p, const PackedSeq& s, int c) {
    // pair q reads past tile c where its last row does: its last token, the
    // smaller of ctx + min(n, (q + 1) span) - 1 and lim - 1, is at 128 c or after
    const int need = 128 * c + 1 - s.ctx;   // positions up to that row
    if (128 * c >= s.lim || need > s.n) return 0;
    return s.all - (need <= p.span ? 0 : over_span(p, need - 1));
}

// The item of rank k, by one warp: sequence (-1 past the last rank), pair, and the
// sequence's first row, rows and length.
__device__ __forceinline__ void packed_find(const PrefillParams& p, int k, int lane, int* item) {
    const PackedSeq mine = packed_seq(p, lane);
    auto total = [&](auto&& f) {
        int v = f(mine);
        for (int bb = 32 + lane; bb < p.batch; bb += 32) v += f(packed_seq(p, bb));
        return __reduce_add_sync(0xffffffffu, v);
    };
    if (lane == 0) item[0] = -1;
    __syncwarp();
    if (k >= total([](const PackedSeq& s) { return s.all; })) return;
    int longest = max(mine.lim, 0);
    for (int bb = 32 + lane; bb < p.batch; bb += 32) longest = max(longest, packed_seq(p, bb).lim);
    // pairs above lo > k >= pairs above hi = 0
    int lo = -1, hi = (__reduce_max_sync(0xffffffffu, longest) + 127) / 128;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (total([&](const PackedSeq& s) { return pairs_above(p, s, mid); }) > k) lo = mid;
        else hi = mid;
    }
    // the pairs of hi tiles, sequence after sequence
    int left = k - total([&](const PackedSeq& s) { return pairs_above(p, s, hi); });
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const PackedSeq s = b0 == 0 ? mine : packed_seq(p, b0 + lane);
        const int skip = pairs_above(p, s, hi);
        const int here = (hi == 0 ? s.all : pairs_above(p, s, hi - 1)) - skip;
        int inc = here;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, inc > left);
        if (hit) {
            if (lane == __ffs(hit) - 1) {
                item[0] = b0 + lane;
                item[1] = s.all - skip - here + (left - (inc - here));
                item[2] = s.first;
                item[3] = s.n;
                item[4] = s.ctx + s.n;
            }
            return;
        }
        left -= __shfl_sync(0xffffffffu, inc, 31);
    }
}

template <int KB, int VB>
__global__ void __launch_bounds__(kPackThreads, 1)
    tq_packed_prefill_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap kmap) {
    using C = PackCfg<KB, VB>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

    uint8_t* sQ = smem + C::kQOff;       // [2][128 x 128] fp16
    uint8_t* sVt = smem + C::kVtOff;
    // n_k * scale * log2(e) per token (quantized K), in frag_place order
    float* colK = reinterpret_cast<float*>(smem + C::kColOff);
    const uint32_t bar_stg = smem_u32(smem + C::kBarOff), bar_free = bar_stg + 16, bar_s = bar_stg + 32,
                   bar_o = bar_stg + 48, bar_p = bar_stg + 64, bar_k = bar_stg + 80, bar_sc = bar_stg + 96,
                   bar_v = bar_stg + 104, bar_q = bar_stg + 112, bar_kr = bar_stg + 120;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 128);
    int* s_item = reinterpret_cast<int*>(smem + C::kColOff);   // until the first scales
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_stg + 8 * i, 1);
            mbar_init(bar_free + 8 * i, 128 + (KB == 0 ? 2 : 0));   // the dequantising threads (and both S)
            mbar_init(bar_s + 8 * i, 1);
            mbar_init(bar_o + 8 * i, 1);
            mbar_init(bar_p + 8 * i, 128);
            mbar_init(bar_k + 8 * i, 128);
        }
        mbar_init(bar_kr, 1);
        mbar_init(bar_sc, 128);
        mbar_init(bar_v, 128);
        mbar_init(bar_q, 256);
        fence_barrier_init();
    }
    griddep_wait();  // cache, lengths, bounds and q come from earlier work on the stream
    // query tile t at columns 256 t: S, its first 64 reused for P as fp16 pairs, then O
    // (behind the wait: an append before may have let this grid start ahead of its own
    // allocations)
    if (warp == 1) tmem_alloc(smem_u32(tslot), 512);
    if (warp == 0) {
        packed_find(p, static_cast<int>(blockIdx.x) / p.hkv, tid, s_item);
    } else if (warp == 2 && blockIdx.x == 0) {
        bool bad = false;
        for (int bb = tid - 64; bb < p.batch; bb += 32)
            bad = bad || p.cu[bb] < 0 || p.cu[bb + 1] < p.cu[bb] || p.cu[bb + 1] > p.total;
        if (bad) atomicOr(p.status, kStatusBadIndex);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    // sequence, query tile pair, the sequence's first row in q and out, rows, length
    const int b = s_item[0], pair = s_item[1], qrow0 = s_item[2], tqn = s_item[3], L = s_item[4];
    __syncthreads();   // (read: the scales may be written)
    if (b < 0) {   // past the last pair (uniform over the CTA)
        if (warp == 1) tmem_dealloc(tmem, 512);
        return;
    }
    const int h = static_cast<int>(blockIdx.x) % p.hkv;
    const int mtiles = (tqn + p.pos_per_tile - 1) / p.pos_per_tile;
    const int t_lim = min(L, p.max_len);
    const int j_hi = min(tqn - 1, (2 * pair + 2) * p.pos_per_tile - 1);
    const int last = min(L - tqn + j_hi, t_lim - 1);   // the last token that a row of the CTA sees
    const int ntiles = last >= 0 ? last / C::kTile + 1 : 0;
    const size_t row0 = static_cast<size_t>(b * p.hkv + h) * p.cap;

    bool stalled = false;  // once set, waits return at once and no MMA or copy is issued
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!stalled && !mbar_wait_bounded(bar, parity)) stalled = true;
    };
    // One decision for the CTA, by all its threads at the end of their roles.
    auto any_stalled = [&]() { return named_bar_or(1, kPackThreads, stalled) != 0; };

    if (warp < 8) {
        regs_inc<kRegsSoftmax>();
        // ---- a query tile's rows: thread = row r = TMEM lane of tile tl ----
        const int tl = warp >> 2, r = tid & 127, lane = tid & 31;
        const int mt = 2 * pair + tl;
        const int jl = r / p.group, hl = r - jl * p.group;   // query position, head of the group
        const int j = mt * p.pos_per_tile + jl;
        const bool row_ok = mt < mtiles && jl < p.pos_per_tile && j < tqn;
        // the row in q and out; none for padding rows
        constexpr unsigned long long kNone = ~0ull;
        const unsigned long long io =
            row_ok ? ((static_cast<unsigned long long>(qrow0) + j) * p.hq + h * p.group + hl) * kD : kNone;
        // this tile's rows see every token up to lim_lo
        const int lim_lo = mt < mtiles ? min(L - tqn + mt * p.pos_per_tile, t_lim - 1) : -1;
        uint8_t* sQt = sQ + tl * 32768;
        uint8_t* sQlt = smem + C::kQloOff + tl * 32768;

        // q, a warp's 32 rows 16 bytes a lane and two rows at a time (a thread that walks
        // its own row touches 32 rows an instruction), all loads in flight together
        {
            uint4 w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const unsigned long long at = __shfl_sync(0xffffffffu, io, 2 * i + (lane >> 4));
                w[i] = make_uint4(0u, 0u, 0u, 0u);
                if (at != kNone) w[i] = __ldg(reinterpret_cast<const uint4*>(p.q + at) + (lane & 15));
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                *reinterpret_cast<uint4*>(
                    sQt + sw128_offset(32 * (warp & 3) + 2 * i + (lane >> 4), 8 * (lane & 15))) = w[i];
            __syncwarp();
        }
        if constexpr (KB != 0) {   // Rot(q) of the thread's row as q_hi + q_lo
            float x[128];
#pragma unroll
            for (int k = 0; k < 128; k += 8) {
                const uint4 w = *reinterpret_cast<const uint4*>(sQt + sw128_offset(r, k));
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ww[e]));
                    x[k + 2 * e] = ((p.signs[k >> 5] >> ((k + 2 * e) & 31)) & 1u) ? -f.x : f.x;
                    x[k + 2 * e + 1] = ((p.signs[k >> 5] >> ((k + 2 * e + 1) & 31)) & 1u) ? -f.y : f.y;
                }
            }
            wht128_thread(x);
#pragma unroll
            for (int k = 0; k < 128; k += 8) {
                uint32_t hv[4], lv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 v = __fmul2_rn(make_float2(x[k + 2 * e], x[k + 2 * e + 1]),   // 1/sqrt(128)
                                                make_float2(0.08838834764831845f, 0.08838834764831845f));
                    hv[e] = pack_half2(v.x, v.y);
                    // q_lo = Rot(q) - q_hi (exact in fp32), rounded once more
                    const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hv[e]));
                    lv[e] = pack_half2(v.x - hf.x, v.y - hf.y);
                }
                *reinterpret_cast<uint4*>(sQt + sw128_offset(r, k)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
                *reinterpret_cast<uint4*>(sQlt + sw128_offset(r, k)) = make_uint4(lv[0], lv[1], lv[2], lv[3]);
            }
        }
        fence_proxy_async();  // the MMAs read Q' through the async proxy
        mbar_arrive(bar_q);

        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + 256 * tl + lane_off;         // the warp's rows of S (and of P)
        const uint32_t t_o = tmem + 256 * tl + 128 + lane_off;   // and of O

        // The softmax works on MMA fragments.  Lane 4v + c of a warp has rows v + 8q (q =
        // 0..3) of its 32 and columns 2c, 2c + 1 of every eight, so a thread reads a
        // quarter of the tile's scales and norms.  A tile that every row sees takes one
        // pass, P in registers until it is known that no score passes its row's base by
        // more than the slack (which shows in the thread's sums); then, with the mask,
        // and on a row's first tile, the rows' maxima are taken first.
        float fm[4], fl[4];   // base (log2) and this thread's part of the sum
        int flim[4];          // last visible token
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int rq = 32 * (warp & 3) + (lane >> 2) + 8 * q, jq = rq / p.group;
            fm[q] = -INFINITY;
            fl[q] = 0.f;
            flim[q] = mt < mtiles && jq < p.pos_per_tile && mt * p.pos_per_tile + jq < tqn
                          ? min(L - tqn + mt * p.pos_per_tile + jq, t_lim - 1)
                          : -1;
        }
        auto softmax = [&](int n) {
            const int tok0 = n * C::kTile;
            const float* col = colK + 4 * (lane & 3);
            const uint8_t* nv_base = smem + C::kNvOff;
            const float* nvs = reinterpret_cast<const float*>(nv_base) + 4 * (lane & 3);
            // how far a score may pass its row's base: p n_v stays below 2^15 (from the
            // largest norm's exponent; subnormal norms count as 2^-15), and how far the
            // largest one does where the base moves (a term then starts at 2^4 or above
            // whatever the norms' size, and loses bits below 2^-18)
            const uint2 top = *reinterpret_cast<const uint2*>(nv_base + C::kTile * 4);
            const uint32_t top2 = __vmaxu2(top.x, top.y), top1 = max(top2 & 0xffffu, top2 >> 16);
            const int slack_i = max(0, 14 + 15 - static_cast<int>(top1 >> 10));
            const float slack = static_cast<float>(slack_i), most = __int_as_float((slack_i + 127) << 23);
            const bool masked = tok0 + C::kTile - 1 > lim_lo;
            const uint32_t t_hi = t_s + (16u << 16);   // rows 16-31
            float2 nb[4], sum[4];
            auto scale4 = [&](int c) {
                if constexpr (KB != 0) return *reinterpret_cast<const float4*>(col + 16 * c);
                return make_float4(p.scale_log2e, p.scale_log2e, p.scale_log2e, p.scale_log2e);
            };
            // x of columns 16c .. 16c + 15 (x[4i + q]) from the S values of rows 0-15 and 16-31
            auto scores = [&](int c, const uint32_t* v0, const uint32_t* v1, float2 (&x)[8]) {
                const float4 s4 = scale4(c);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = e >> 2, q = e & 3;
                    const uint32_t* f = (q < 2 ? v0 : v1) + 4 * i + 2 * (q & 1);
                    x[e] = __ffma2_rn(make_float2(__uint_as_float(f[0]), __uint_as_float(f[1])),
                                      i ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y), nb[q]);
                }
            };
            auto hide = [&](int c, float2 (&x)[8]) {   // tokens past a row's last visible one
                const int t0 = tok0 + 16 * c + 2 * (lane & 3);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int left = flim[e & 3] - t0 - 8 * (e >> 2);
                    if (left < 0) x[e].x = -INFINITY;
                    if (left < 1) x[e].y = -INFINITY;
                }
            };
            // P of the columns, as the fragments of a store of 16 packed columns (j = 0..3:
            // eight tokens each; the pair j0, j0 + 1 here)
            auto weigh = [&](int c, int j0, const float2 (&x)[8], uint32_t (&pk)[2][8]) {
                const float4 w4 = *reinterpret_cast<const float4*>(nvs + 16 * c);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = e >> 2, q = e & 3;
                    const float2 pe = make_float2(fast_exp2(x[e].x), fast_exp2(x[e].y));
                    sum[q] = __fadd2_rn(sum[q], pe);
                    const float2 w = __fmul2_rn(pe, i ? make_float2(w4.z, w4.w) : make_float2(w4.x, w4.y));
                    pk[q >> 1][2 * (j0 + i) + (q & 1)] = pack_half2(w.x, w.y);
                }
            };
            auto set_base = [&]() {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float b0 = fm[q] == -INFINITY ? 0.f : -fm[q];
                    nb[q] = make_float2(b0, b0);
                    sum[q] = make_float2(0.f, 0.f);
                }
            };
            bool fresh_row = false;
#pragma unroll
            for (int q = 0; q < 4; ++q) fresh_row = fresh_row || fm[q] == -INFINITY;
            bool move = masked || __any_sync(0xffffffffu, fresh_row);
#pragma unroll 1
            for (;;) {
                set_base();
                if (move) {   // the rows' maxima, which may move their bases
                    float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        uint32_t v0[8], v1[8];
                        tmem_ld_frag_issue(t_s + 16 * c, v0);
                        tmem_ld_frag_issue(t_hi + 16 * c, v1);
                        tmem_ld_wait(v0, v1);
                        float2 x[8];
                        scores(c, v0, v1, x);
                        if (masked) hide(c, x);
#pragma unroll
                        for (int e = 0; e < 8; ++e) mq[e & 3] = fmaxf(mq[e & 3], fmaxf(x[e].x, x[e].y));
                    }
                    float alpha[4];
                    bool grow = false;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {   // a row's maximum is spread over its four lanes
                        float mx = fmaxf(mq[q], __shfl_xor_sync(0xffffffffu, mq[q], 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        const bool fresh = fm[q] == -INFINITY;
                        const bool up = mx > (fresh ? -INFINITY : slack);
                        mx -= fmaxf(0.f, slack - 10.f);   // (what the base moves by)
                        alpha[q] = up ? (fresh ? 0.f : fast_exp2(-mx)) : 1.f;
                        fl[q] *= alpha[q];
                        if (up) fm[q] = (fresh ? 0.f : fm[q]) + mx;
                        grow = grow || up;
                    }
                    if (n > 0 && __any_sync(0xffffffffu, grow)) {   // rescale O (P.V(n-1) is done)
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            uint32_t o0[8], o1[8];
                            tmem_ld_frag_issue(t_o + 16 * c, o0);
                            tmem_ld_frag_issue(t_o + (16u << 16) + 16 * c, o1);
                            tmem_ld_wait(o0, o1);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                o0[e] = __float_as_uint(__uint_as_float(o0[e]) * alpha[(e >> 1) & 1]);
                                o1[e] = __float_as_uint(__uint_as_float(o1[e]) * alpha[2 + ((e >> 1) & 1)]);
                            }
                            tmem_st_frag256(t_o + 16 * c, o0);
                            tmem_st_frag256(t_o + (16u << 16) + 16 * c, o1);
                        }
                        tmem_st_wait();
                    }
                    set_base();
                }
                if (masked) {
                    // 32 tokens a turn, P over columns of S that have been read
#pragma unroll 1
                    for (int c = 0; c < 8; c += 2) {
                        uint32_t pk[2][8];
#pragma unroll
                        for (int h2 = 0; h2 < 2; ++h2) {
                            uint32_t v0[8], v1[8];
                            tmem_ld_frag_issue(t_s + 16 * (c + h2), v0);
                            tmem_ld_frag_issue(t_hi + 16 * (c + h2), v1);
                            tmem_ld_wait(v0, v1);
                            float2 x[8];
                            scores(c + h2, v0, v1, x);
                            hide(c + h2, x);
                            weigh(c + h2, 2 * h2, x, pk);
                        }
                        tmem_st_frag_issue(t_s + 8 * c, pk[0]);
                        tmem_st_frag_issue(t_hi + 8 * c, pk[1]);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) fl[q] += sum[q].x + sum[q].y;
                    break;
                }
                uint32_t pk[4][2][8];
                uint32_t v[2][2][8];   // 16 columns at a time, the next ones in flight
                tmem_ld_frag_issue(t_s, v[0][0]);
                tmem_ld_frag_issue(t_hi, v[0][1]);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    tmem_ld_wait(v[c & 1][0], v[c & 1][1]);
                    if (c < 7) {
                        tmem_ld_frag_issue(t_s + 16 * (c + 1), v[(c + 1) & 1][0]);
                        tmem_ld_frag_issue(t_hi + 16 * (c + 1), v[(c + 1) & 1][1]);
                    }
                    float2 x[8];
                    scores(c, v[c & 1][0], v[c & 1][1], x);
                    weigh(c, 2 * (c & 1), x, pk[c >> 1]);
                }
                float s4[4], top = 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    s4[q] = sum[q].x + sum[q].y;
                    top = fmaxf(top, s4[q]);
                }
                if (move || !__any_sync(0xffffffffu, top > most)) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) fl[q] += s4[q];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tmem_st_frag_issue(t_s + 16 * c, pk[c][0]);
                        tmem_st_frag_issue(t_hi + 16 * c, pk[c][1]);
                    }
                    break;
                }
                move = true;
            }
            tmem_st_wait();
        };
        for (int n = 0; n < ntiles; ++n) {
            wait(bar_sc, n & 1);
            wait(bar_s + 8 * tl, n & 1);
            tc_fence_after();
            softmax(n);
            tc_fence_before();
            mbar_arrive(bar_p + 8 * tl);
        }
        if (ntiles > 0) wait(bar_o + 8 * tl, (ntiles - 1) & 1);
        tc_fence_after();
        if (any_stalled()) {
            if (tid == 0) atomicOr(p.status, kStatusPipelineStall);
        } else {
            // ---- O / l, v_rescale, inverse rotation, fp16 ----
            // the sums, a row per thread from here on (the scales and norms are read)
            float* rows = colK + 128 * tl;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float l = fl[q] + __shfl_xor_sync(0xffffffffu, fl[q], 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                if ((lane & 3) == 0) rows[32 * (warp & 3) + (lane >> 2) + 8 * q] = l;
            }
            __syncwarp();
            const float l_sum = rows[r];
            float o[128];
            if (ntiles > 0) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {  // every lane: the loads are warp-collective
                    uint32_t v[32];
                    tmem_ld32(t_o + 32 * c, v);
                    // O's column pi(d) holds dim d (V^T rows are stored in that order)
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[32 * c + e] = __uint_as_float(v[e ^ (2 * c)]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 128; ++e) o[e] = 0.f;
            }
            // (a NaN sum is a row of NaN scores, not one that sees no token)
            if (row_ok && l_sum == 0.f) atomicOr(p.status, kStatusShortContext);
            // 1/l, v_rescale and the rotation's 1/sqrt(128), applied after the
            // (linear) transform in one packed multiply
            const float g = l_sum == 0.f ? 0.f : p.v_rescale / l_sum * 0.08838834764831845f;
            wht128_thread(o);
            // over this row of Q', which the MMAs have read
#pragma unroll
            for (int k = 0; k < 128; k += 8) {
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 v = __fmul2_rn(make_float2(o[k + e], o[k + e + 1]), make_float2(g, g));
                    y[e >> 1] = pack_half2(((p.signs[k >> 5] >> ((k + e) & 31)) & 1u) ? -v.x : v.x,
                                           ((p.signs[k >> 5] >> ((k + e + 1) & 31)) & 1u) ? -v.y : v.y);
                }
                *reinterpret_cast<uint4*>(sQt + sw128_offset(r, k)) = make_uint4(y[0], y[1], y[2], y[3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) {   // padding rows write nothing
                const unsigned long long at = __shfl_sync(0xffffffffu, io, 2 * i + (lane >> 4));
                const uint4 y = *reinterpret_cast<const uint4*>(
                    sQt + sw128_offset(32 * (warp & 3) + 2 * i + (lane >> 4), 8 * (lane & 15)));
                if (at != kNone) *(reinterpret_cast<uint4*>(p.out + at) + (lane & 15)) = y;
            }
        }
    } else if (warp < 12) {
        regs_dec<kRegsOther>();
        // ---- dequantise: thread r of 128 ----
        const int r = tid - 256;
        // K's dims 64 half .. 64 half + 63, one token a thread
        // (in halves, so that one is stored while S reads the other: 12 prompts of 64 to
        // 4096 tokens 436 us, whole tiles 442)
        [[maybe_unused]] auto k_dequant = [&](int n, int half) {
            if constexpr (KB != 0) {
                const Tables kt{p.ktab[0], p.ktab[1], p.ktab[2], p.ktab[3]};
                const uint8_t* rec = smem + C::kStgOff + (n & 1) * C::kSlot + r * C::kRbK;
                uint8_t* sK = smem + C::kKOff + half * 16384;
                // the quarters in an order that differs between lanes whose records
                // start in the same banks
                const int turn = KB == 4 ? r >> 1 : r >> 3;
#pragma unroll 1
                for (int q = 0; q < 2; ++q) {
                    const int side = (q + turn) & 1;
                    uint32_t hh[16];
                    dequant_q32<KB>(rec + (2 * half + side) * (C::kRbK / 4), kt, hh);
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        *reinterpret_cast<uint4*>(sK + sw128_offset(r, 32 * side + 8 * m)) =
                            make_uint4(hh[4 * m], hh[4 * m + 1], hh[4 * m + 2], hh[4 * m + 3]);
                }
                fence_proxy_async();
                mbar_arrive(bar_k + 8 * half);
            }
        };
        for (int n = 0; n < ntiles; ++n) {
            const uint8_t* slot = smem + C::kStgOff + (n & 1) * C::kSlot;
            wait(bar_stg + 8 * (n & 1), (n >> 1) & 1);
            if constexpr (KB != 0) {
                // each half of K once S_0(n - 1) and S_1(n - 1) have read the one before
                if (n > 0) wait(bar_kr, (n - 1) & 1);
                k_dequant(n, 0);
                if (n > 0) wait(bar_s + 8, (n - 1) & 1);
                k_dequant(n, 1);
            }
            if (n > 0) {   // the scales and norms of n - 1 are read
                wait(bar_p, (n - 1) & 1);
                wait(bar_p + 8, (n - 1) & 1);
            }
            const bool in = n * C::kTile + r < t_lim;
            if constexpr (KB != 0) {
                const float nk = __half2float(reinterpret_cast<const __half*>(slot + C::kSK)[r]);
                colK[frag_place(r)] = in ? nk * p.scale_log2e : 0.f;
            }
            const float nv =
                in ? __half2float(reinterpret_cast<const __half*>(slot + C::kSK + C::kSKn + C::kSV)[r]) : 0.f;
            float* nvs = reinterpret_cast<float*>(smem + C::kNvOff);
            nvs[frag_place(r)] = fmaxf(fminf(nv, 65504.f), -65504.f);
            // the largest finite one (non-negative floats order like their bits)
            const uint32_t top = __reduce_max_sync(0xffffffffu, fabsf(nv) < 65536.f ? __float_as_uint(fabsf(nv)) : 0u);
            if ((r & 31) == 0)
                reinterpret_cast<__half*>(nvs + C::kTile)[r >> 5] = __float2half_rn(__uint_as_float(top));
            mbar_arrive(bar_sc);
            if (n > 0) {   // V(n - 1)^T is read
                wait(bar_o, (n - 1) & 1);
                wait(bar_o + 8, (n - 1) & 1);
            }
            store_vt<VB>(slot + C::kSK + C::kSKn, sVt, Tables{p.vtab[0], p.vtab[1], p.vtab[2], p.vtab[3]}, warp - 8,
                         tid & 31);
            fence_proxy_async();
            mbar_arrive(bar_v);
            mbar_arrive(bar_free + 8 * (n & 1));
        }
        any_stalled();
    } else {
        regs_dec<kRegsOther>();
        // ---- issue: one thread a warp ----
        const bool one = (tid & 31) == 0;
        if (warp == 12 && one && ntiles > 0) {   // S_t(n) = Q'_t . K(n)^T into tile t's S columns
            int done = 0;
            wait(bar_q, 0);
            for (int n = 0; n < ntiles && !stalled; ++n) {
                if constexpr (KB == 0) wait(bar_stg + 8 * (n & 1), (n >> 1) & 1);
                const uint32_t kbase =
                    (KB == 0) ? smem_u32(smem + C::kStgOff + (n & 1) * C::kSlot) : smem_u32(smem + C::kKOff);
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    if (n > 0) wait(bar_o + 8 * t, (n - 1) & 1);   // P.V_t(n - 1) has read the P there
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (KB != 0 && t == 0) wait(bar_k + 8 * half, n & 1);
                        if (!stalled) {
                            tc_fence_after();
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                const uint32_t koff = half * 16384 + kk * 32;
                                umma_f16(tmem + 256 * t, umma_desc_sw128(smem_u32(sQ) + t * 32768 + koff),
                                         umma_desc_sw128(kbase + koff), C::kIdesc, half + kk > 0 ? 1u : 0u);
                                if constexpr (KB != 0)  // + q_lo . K^T
                                    umma_f16(tmem + 256 * t,
                                             umma_desc_sw128(smem_u32(smem + C::kQloOff) + t * 32768 + koff),
                                             umma_desc_sw128(kbase + koff), C::kIdesc, 1u);
                            }
                            if (KB != 0 && t == 1 && half == 0) umma_commit(bar_kr);
                        }
                    }
                    if (stalled) break;   // (the MMAs in flight are waited for below)
                    umma_commit(bar_s + 8 * t);
                    if constexpr (KB == 0) umma_commit(bar_free + 8 * (n & 1));
                    ++done;
                }
            }
            // after a time-out: the MMAs in flight, half a tile's among them, end before
            // tensor memory is freed (the commit of the S that comes next)
            if (stalled) {
                umma_commit(bar_s + 8 * (done & 1));
                (void)mbar_wait_bounded(bar_s + 8 * (done & 1), (done >> 1) & 1);
            }
        } else if (warp == 13 && one) {   // O_t += P_t(n) . V(n), P from tensor memory over S_t
            int done = 0;
            for (int n = 0; n < ntiles && !stalled; ++n) {
                wait(bar_v, n & 1);
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    wait(bar_p + 8 * t, n & 1);
                    if (stalled) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t koff = (kk >> 2) * 16384 + (kk & 3) * 32;
                        umma_f16_ts(tmem + 256 * t + 128, tmem + 256 * t + 8 * kk,
                                    umma_desc_sw128(smem_u32(sVt) + koff), C::kIdesc, (n > 0 || kk > 0) ? 1u : 0u);
                    }
                    umma_commit(bar_o + 8 * t);
                    ++done;
                }
            }
            if (stalled) {
                umma_commit(bar_o + 8 * (done & 1));
                (void)mbar_wait_bounded(bar_o + 8 * (done & 1), (done >> 1) & 1);
            }
        } else if (warp == 14 && one) {   // tile n into staging slot n & 1
            auto issue = [&](int n) {
                const int tok0 = n * C::kTile;
                const int nval = min(C::kTile, t_lim - tok0);
                uint8_t* slot = smem + C::kStgOff + (n & 1) * C::kSlot;
                const uint32_t bar = bar_stg + 8 * (n & 1);
                const uint32_t nb = static_cast<uint32_t>((nval + 7) & ~7) * 2;
                uint32_t bytes = nval * C::kRbV + nb;
                bytes += (KB == 0) ? 32768u : nval * C::kRbK + nb;
                mbar_arrive_expect_tx(bar, bytes);
                if constexpr (KB == 0) {
                    // 128 rows x 128 dims in four 32-row boxes per 64-dim half (rows past
                    // the tensor's end are zero-filled; masked below)
                    for (int half = 0; half < 2; ++half)
                        for (int rb = 0; rb < 4; ++rb)
                            tma_g2s_2d(smem_u32(slot) + half * 16384 + rb * 4096, &kmap, half * 64,
                                       static_cast<int32_t>(row0 + tok0 + rb * 32), bar);
                } else {
                    bulk_g2s(smem_u32(slot), p.k_codes + (row0 + tok0) * C::kRbK, nval * C::kRbK, bar);
                    bulk_g2s(smem_u32(slot + C::kSK), p.k_norm + row0 + tok0, nb, bar);
                }
                bulk_g2s(smem_u32(slot + C::kSK + C::kSKn), p.v_codes + (row0 + tok0) * C::kRbV,
                         nval * C::kRbV, bar);
                bulk_g2s(smem_u32(slot + C::kSK + C::kSKn + C::kSV), p.v_norm + row0 + tok0, nb, bar);
            };
            int done = 0;
            for (; done < ntiles; ++done) {
                if (done >= 2) wait(bar_free + 8 * (done & 1), ((done >> 1) - 1) & 1);
                if (stalled) break;
                issue(done);
            }
            // (after a time-out: the copies in flight land before shared memory goes away)
            if (stalled)
                for (int m = max(done - 2, 0); m < done; ++m)
                    (void)mbar_wait_bounded(bar_stg + 8 * (m & 1), (m >> 1) & 1);
        }
        __syncwarp();
        any_stalled();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int KB, int VB>
static int launch_t(const PrefillParams& p, const CUtensorMap* kmap, cudaStream_t stream) {
    using C = PackCfg<KB, VB>;
    static std::atomic<uint64_t> attr_done{0};
    const cudaError_t e = set_smem_attr_once(tq_packed_prefill_kernel<KB, VB>, C::kSmemAlloc, attr_done, -1, kRegsLaunch);
    if (e != cudaSuccess) return e;
    return launch_pdl(tq_packed_prefill_kernel<KB, VB>, dim3(p.slots * p.hkv), dim3(kPackThreads), C::kSmemAlloc,
                      stream, p, *kmap);
}

int launch_packed_prefill(int kbits, int vbits, const PrefillParams& p, const CUtensorMap* kmap,
                          cudaStream_t stream) {
    if (kbits == 16 && vbits == 4) return launch_t<0, 4>(p, kmap, stream);
    if (kbits == 16 && vbits == 3) return launch_t<0, 3>(p, kmap, stream);
    if (kbits == 3 && vbits == 3) return launch_t<3, 3>(p, kmap, stream);
    if (kbits == 4 && vbits == 4) return launch_t<4, 4>(p, kmap, stream);
    if (kbits == 4 && vbits == 3) return launch_t<4, 3>(p, kmap, stream);
    return cudaErrorInvalidValue;
}

}  // namespace tq
