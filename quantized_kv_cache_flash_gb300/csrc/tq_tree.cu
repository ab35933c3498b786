// Attention of a drafted tree over the packed cache on the 5th-generation
// tensor cores: split over the context, for blocks of more than 16 query rows
// per KV head (fewer run on the decode kernel, whose warp MMAs hold 16).
//
// Per 128 query rows (drafted nodes x heads of the group) and 128 tokens:
//   S[128 x 128] = Q' . K^T          (8 or 16 MMAs of K = 16, fp32 in tensor memory)
//   P[r][t]      = 2^(S n_k scale log2 e - base_r) n_v / 16   (rounded to fp16)
//   O[128 x 128] += P . C_v          (8 MMAs, fp32 in tensor memory)
// with Q' = Rot(q) as two fp16 halves (quantized K: K's tile holds the fp16
// centroids, the norm goes to the fp32 scores) or q (fp16 K).  V's tile holds
// the centroids themselves, exact in fp16, and the V norm goes into P, so a
// term is rounded once.  The base of a row trails its maximum by at most 4
// (log2), so p <= 16 and p n_v / 16 stays in fp16 for every norm; the factor 16
// comes back in the merge.
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
constexpr float kPScale = 1.0f / 16.0f;

template <int KB, int VB>
struct TreeCfg {
    static constexpr int kRbK = (KB == 0) ? 256 : KB * 16;
    static constexpr int kRbV = VB * 16;
    static constexpr int kQOff = 0;                                   // fp16 Q' (q_hi), 32 KB
    static constexpr int kQloOff = 32768;                             // q_lo (quantized K), 32 KB
    static constexpr int kVtOff = (KB == 0) ? 32768 : 65536;          // per group V^T [dim][token], 32 KB
    static constexpr int kKOff = kVtOff + 65536;                      // per group K [token][dim] (quantized K)
    static constexpr int kStgOff = (KB == 0) ? kKOff : kKOff + 65536;
    // staged records of a tile (fp16 K: the MMA tile itself, three stages that
    // the two groups' tiles take in turn; else one per group)
    static constexpr int kStages = (KB == 0) ? 3 : 2;
    static constexpr int kSK = (KB == 0) ? 32768 : kTok * kRbK;
    static constexpr int kSV = kTok * kRbV;
    static constexpr int kAlign = (KB == 0) ? 1024 : 128;
    static constexpr int kSlot = (kSK + kSV + kAlign - 1) / kAlign * kAlign;
    static constexpr int kColOff = kStgOff + kStages * kSlot;         // per group n_k scale log2 e [128]
    static constexpr int kNvOff = kColOff + 2 * kTok * 4;             // per group n_v / 16 [128]
    // mbarriers full[3], S[2], O[2]; TMEM slot
    static constexpr int kBarOff = kNvOff + 2 * kTok * 4;
    static constexpr int kSmem = kBarOff + 64;
    static constexpr int kSmemAlloc = kSmem + 896;   // to a 1024-byte boundary from a 128-byte one
    static_assert(kSmemAlloc <= 232448, "227 KB per CTA");
    static constexpr uint32_t kIdesc = umma_idesc_f16_f32(128, 128);
};

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
__global__ void __launch_bounds__(256, 1)
    tq_tree_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap kmap) {
    using C = TreeCfg<KB, VB>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int lane = tid & 31;
    const int g = warp >> 2, r = tid & 127;   // group; row (tensor-memory lane) and token of its tiles

    griddep_wait();   // cache, lengths, mask and q come from earlier work on the stream
    const int P = static_cast<int>(gridDim.x), c_me = static_cast<int>(blockIdx.x);
    const int total = __shfl_sync(0xffffffffu, tree_total(p, lane), 0);
    const int lo = static_cast<int>(static_cast<long long>(c_me) * total / P);
    const int hi = static_cast<int>(static_cast<long long>(c_me + 1) * total / P);
    if (lo >= hi) return;   // (uniform over the CTA)

    const uint32_t bar_full = smem_u32(smem + C::kBarOff);   // + 8 stage
    const uint32_t bar_s = bar_full + 24 + 8 * g, bar_o = bar_full + 40 + 8 * g;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 56);
    if (tid == 0) {
        for (int i = 0; i < 7; ++i) mbar_init(bar_full + 8 * i, 1);
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(smem_u32(tslot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot + 256 * g;                  // this group's S (its first 64 columns take P), then O
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off, t_o = tmem + 128 + lane_off;

    uint8_t* sVt = smem + C::kVtOff + g * 32768;
    uint8_t* sK = smem + C::kKOff + g * 32768;
    float* col = reinterpret_cast<float*>(smem + C::kColOff) + g * kTok;
    float* nvs = reinterpret_cast<float*>(smem + C::kNvOff) + g * kTok;

    bool stalled = false;   // once set, waits return at once and nothing more is issued
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!stalled && !mbar_wait_bounded(bar, parity)) stalled = true;
    };
    uint32_t used = 0;      // this group's S (and P.V) products so far
    uint32_t sent_s = 0, sent_o = 0;   // those that this thread has issued
    int tbase = 0;          // tiles of the earlier segments: stage and phase of tile n are those of tbase + n
    int pos = lo;
    while (pos < hi) {
        // ---- the segment: chunks [k0, k0 + ntiles) of unit (b, h, rt) ----
        int b, before;
        tree_locate(p, pos, lane, b, before);
        b = __shfl_sync(0xffffffffu, b, 0);
        before = __shfl_sync(0xffffffffu, before, 0);
        const int L = p.lengths[b];
        const int nch = tree_chunks(L, p.max_len);
        const int ui = (pos - before) / nch;   // h * row_tiles + rt
        const int k0 = (pos - before) - ui * nch;
        const int ntiles = min(nch - k0, hi - pos);
        const int h = ui / p.row_tiles, rt = ui - h * p.row_tiles;
        const int t_lim = min(L, p.max_len);
        const int base = L - p.tq;             // first drafted token
        const int full_below = min(base, t_lim);   // tokens below this are seen by every row
        const size_t row0 = (static_cast<size_t>(b) * p.hkv + h) * p.cap;
        // this thread's query row: node j, head hl of the group
        const int rr = rt * kTreeRows + r;
        const bool row_ok = rr < p.rows;
        const bool live = rt * kTreeRows + 32 * (warp & 3) < p.rows;   // some lane of the warp has a row
        const uint32_t* mrow = p.tree + static_cast<size_t>(b) * p.tree_per_seq +
                               (row_ok ? rr / p.group : 0) * p.tree_words;

        auto issue = [&](int n) {   // one thread: the records of tile n
            const int tok0 = (k0 + n) * kTok;
            const int nval = min(kTok, t_lim - tok0);
            const int st = (tbase + n) % C::kStages;
            uint8_t* slot = smem + C::kStgOff + st * C::kSlot;
            const uint32_t bar = bar_full + 8 * st;
            mbar_arrive_expect_tx(bar, ((KB == 0) ? 32768u : nval * C::kRbK) + nval * C::kRbV);
            if constexpr (KB == 0) {
                for (int half = 0; half < 2; ++half)
                    for (int q = 0; q < 4; ++q)
                        tma_g2s_2d(smem_u32(slot) + half * 16384 + q * 4096, &kmap, half * 64,
                                   static_cast<int32_t>(row0 + tok0 + q * 32), bar);
            } else {
                bulk_g2s(smem_u32(slot), p.k_codes + (row0 + tok0) * C::kRbK, nval * C::kRbK, bar);
            }
            bulk_g2s(smem_u32(slot + C::kSK), p.v_codes + (row0 + tok0) * C::kRbV, nval * C::kRbV, bar);
        };
        if (tid == 0 && !stalled)
            for (int n = 0; n < C::kStages && n < ntiles; ++n) issue(n);

        // norms of this thread's token of its group's next tile
        auto norm_k = [&](int n) {
            const int t = (k0 + n) * kTok + r;
            return (KB != 0 && n < ntiles && t < t_lim) ? __half2float(p.k_norm[row0 + t]) : 0.f;
        };
        auto norm_v = [&](int n) {
            const int t = (k0 + n) * kTok + r;
            return (n < ntiles && t < t_lim) ? __half2float(p.v_norm[row0 + t]) : 0.f;
        };
        float nk = norm_k(g), nv = norm_v(g);

        // ---- Q' of the unit's rows: two threads per row, 64 dims each ----
        {
            const int qr = tid >> 1, half = tid & 1;
            const int qrr = rt * kTreeRows + qr;
            float x[64];
            if (qrr < p.rows) {
                const int j = qrr / p.group, hl = qrr - j * p.group;
                const __half* qp = p.q + ((static_cast<size_t>(b) * p.hq + h * p.group + hl) * p.tq + j) * kD + 64 * half;
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
        tc_fence_before();
        __syncthreads();
        tc_fence_after();

        float m_base = -INFINITY, l_sum = 0.f;
        const uint32_t used0 = used;
        for (int n = g; n < ntiles; n += 2) {
            const int tok0 = (k0 + n) * kTok;
            const int st = (tbase + n) % C::kStages;
            const uint8_t* slot = smem + C::kStgOff + st * C::kSlot;
            wait(bar_full + 8 * st, ((tbase + n) / C::kStages) & 1);

            // K(n): a token per thread; the quarters are taken in an order that
            // differs between lanes whose records start in the same banks
            if constexpr (KB != 0) {
                const Tables kt{p.ktab[0], p.ktab[1], p.ktab[2], p.ktab[3]};
                const uint8_t* rec = slot + r * C::kRbK;
                const int turn = KB == 4 ? r >> 1 : r >> 3;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    const int quarter = (q + turn) & 3;
                    uint32_t hh[16];
                    dequant_q32<KB>(rec + quarter * (C::kRbK / 4), kt, hh);
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        *reinterpret_cast<uint4*>(sK + sw128_offset(r, 32 * quarter + 8 * m)) =
                            make_uint4(hh[4 * m], hh[4 * m + 1], hh[4 * m + 2], hh[4 * m + 3]);
                }
                fence_proxy_async();
            }
            col[r] = (KB == 0) ? p.scale_log2e : nk * p.scale_log2e;
            // (an overflowed norm counts as 65504: 0 * inf would be NaN in the
            // rows that do not see the token)
            nvs[r] = fminf(nv, 65504.f) * kPScale;
            nk = norm_k(n + 2);
            nv = norm_v(n + 2);
            tc_fence_before();
            named_bar_sync(1 + g, 128);   // K(n) and the norms are stored
            if (n != g) wait(bar_o, (used - 1) & 1);   // P.V of the group's last tile: P, V^T and O are free
            tc_fence_after();
            if (r == 0 && !stalled) {
                const uint32_t kbase = smem_u32((KB == 0) ? slot : sK);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t koff = (kk >> 2) * 16384 + (kk & 3) * 32;
                    umma_f16(tmem, umma_desc_sw128(smem_u32(smem + C::kQOff) + koff), umma_desc_sw128(kbase + koff),
                             C::kIdesc, kk > 0 ? 1u : 0u);
                    if constexpr (KB != 0)
                        umma_f16(tmem, umma_desc_sw128(smem_u32(smem + C::kQloOff) + koff),
                                 umma_desc_sw128(kbase + koff), C::kIdesc, 1u);
                }
                umma_commit(bar_s);
                ++sent_s;
            }
            __syncwarp();

            // V(n)^T under the S product: lane 4v + t dequantises quarter t of
            // tokens 16 vw + v and + 8, stored transposed in rows pi(d) = d ^ 2(d >> 5),
            // whose 8 rows per stored matrix lie in different banks
            {
                const Tables vt{p.vtab[0], p.vtab[1], p.vtab[2], p.vtab[3]};
                const uint8_t* vrec = slot + C::kSK;
                const int sj = lane >> 3, sc = lane & 7;
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    const int vw = (warp & 3) + 4 * i;
                    const int ta = 16 * vw + (lane >> 2);
                    uint32_t ha[16], hb[16];
                    dequant_q32<VB>(vrec + ta * C::kRbV + (lane & 3) * (C::kRbV / 4), vt, ha);
                    dequant_q32<VB>(vrec + (ta + 8) * C::kRbV + (lane & 3) * (C::kRbV / 4), vt, hb);
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
                fence_proxy_async();
            }

            wait(bar_s, used & 1);
            tc_fence_after();
            if (live) {   // (warp-uniform) softmax of this thread's row, as in the prefill kernel
                float x[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32];
                    tmem_ld32(t_s + 32 * c, v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[32 * c + e] = __uint_as_float(v[e]);
                }
                const bool fresh = (m_base == -INFINITY);
                const float base0 = fresh ? 0.f : m_base;
                const float2 nb2 = make_float2(-base0, -base0);
#pragma unroll
                for (int e = 0; e < 128; e += 4) {
                    const float4 s4 = *reinterpret_cast<const float4*>(col + e);
                    const float2 a = __ffma2_rn(make_float2(x[e], x[e + 1]), make_float2(s4.x, s4.y), nb2);
                    const float2 c = __ffma2_rn(make_float2(x[e + 2], x[e + 3]), make_float2(s4.z, s4.w), nb2);
                    x[e] = a.x;
                    x[e + 1] = a.y;
                    x[e + 2] = c.x;
                    x[e + 3] = c.y;
                }
                if (tok0 + kTok > full_below) {   // a tile that some row sees in part
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int t0 = tok0 + 32 * c;
                        uint32_t vis = row_ok ? tree_window(mrow, p.tree_words, t0 - base) : 0u;
                        if (t0 + 32 > t_lim) vis &= t0 < t_lim ? (1u << (t_lim - t0)) - 1u : 0u;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((vis >> e) & 1u)) x[32 * c + e] = -INFINITY;
                    }
                }
                float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 128; e += 8)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mq[j] = fmaxf(mq[j], fmaxf(x[e + 2 * j], x[e + 2 * j + 1]));
                const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
                const bool grow = fresh ? (mx > -INFINITY) : (mx > 4.f);
                if (__any_sync(0xffffffffu, grow)) {
                    const float shift = grow ? mx : 0.f;
                    const float alpha = grow ? (fresh ? 0.f : fast_exp2(-mx)) : 1.f;
                    l_sum *= alpha;
                    if (grow) m_base = base0 + mx;
#pragma unroll
                    for (int e = 0; e < 128; ++e) x[e] -= shift;
                    if (n != g) {   // rescale this row of O (P.V of the last tile is done)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t v[32];
                            tmem_ld32(t_o + 32 * c, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
                            tmem_st32(t_o + 32 * c, v);
                        }
                    }
                }
                float2 s2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const int k = 64 * c + 2 * e;
                        const float4 w = *reinterpret_cast<const float4*>(nvs + k);
                        const float2 pa = make_float2(fast_exp2(x[k]), fast_exp2(x[k + 1]));
                        const float2 pb = make_float2(fast_exp2(x[k + 2]), fast_exp2(x[k + 3]));
                        s2[e & 3] = __fadd2_rn(s2[e & 3], pa);
                        s2[(e & 3) + 1] = __fadd2_rn(s2[(e & 3) + 1], pb);
                        const float2 wa = __fmul2_rn(pa, make_float2(w.x, w.y));
                        const float2 wb = __fmul2_rn(pb, make_float2(w.z, w.w));
                        pk[e] = pack_half2(wa.x, wa.y);
                        pk[e + 1] = pack_half2(wb.x, wb.y);
                    }
                    tmem_st32(t_s + 32 * c, pk);   // P over S columns 0..63
                }
                const float2 sa = __fadd2_rn(s2[0], s2[1]), sb = __fadd2_rn(s2[2], s2[3]);
                const float2 sm = __fadd2_rn(sa, sb);
                l_sum += sm.x + sm.y;
            }
            tc_fence_before();
            if (named_bar_or(1 + g, 128, stalled)) stalled = true;   // V(n)^T and P(n) are stored
            tc_fence_after();
            if (r == 0 && !stalled) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    umma_f16_ts(tmem + 128, tmem + 8 * kk,
                                umma_desc_sw128(smem_u32(sVt) + (kk >> 2) * 16384 + (kk & 3) * 32), C::kIdesc,
                                (n != g || kk > 0) ? 1u : 0u);
                umma_commit(bar_o);
                ++sent_o;
                if (n + C::kStages < ntiles) {   // tile n's stage is consumed by everybody
                    fence_proxy_async();
                    issue(n + C::kStages);
                }
            }
            __syncwarp();
            ++used;
        }

        // ---- merge the two groups, write the unit's partial ----
        // Group g keeps dims 64 g .. 64 g + 63 of every row and hands the
        // others over through its own V^T tile, 16-byte pieces XORed with the row.
        const bool had = used != used0;
        if (had) wait(bar_o, (used - 1) & 1);
        const bool bad = __syncthreads_or(stalled) != 0;
        tc_fence_after();
        if (pos + ntiles >= hi || bad) griddep_launch_dependents();   // last segment: let the merge launch
        if (bad) {
            stalled = true;
            // the products and copies still in flight end before the shared and
            // tensor memory go away
            if (sent_s > 0) (void)mbar_wait_bounded(bar_s, (sent_s - 1) & 1);
            if (sent_o > 0) (void)mbar_wait_bounded(bar_o, (sent_o - 1) & 1);
            if (tid == 0) {
                atomicOr(p.status, kStatusPipelineStall);
                for (int n = max(0, ntiles - C::kStages); n < ntiles; ++n)
                    (void)mbar_wait_bounded(bar_full + 8 * ((tbase + n) % C::kStages), ((tbase + n) / C::kStages) & 1,
                                            100000000ull);
            }
            break;
        }
        float* xch = reinterpret_cast<float*>(sVt);
        col[r] = m_base;
        nvs[r] = l_sum;
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
        __syncthreads();
        {
            const float* ox = reinterpret_cast<const float*>(smem + C::kVtOff + (1 - g) * 32768);
            const float om = (reinterpret_cast<const float*>(smem + C::kColOff) + (1 - g) * kTok)[r];
            const float ol = (reinterpret_cast<const float*>(smem + C::kNvOff) + (1 - g) * kTok)[r];
            const float M = fmaxf(m_base, om);
            const float a = m_base == -INFINITY ? 0.f : fast_exp2(m_base - M);
            const float c2 = om == -INFINITY ? 0.f : fast_exp2(om - M);
            const int unit = b * p.per_b + ui;
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
                float y[32];
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 o = *reinterpret_cast<const float4*>(ox + r * 64 + 4 * ((8 * c + e / 4) ^ (r & 15)));
                    // (a row that saw no token has weight 0, whatever its columns hold)
                    y[e] = (a != 0.f ? a * __uint_as_float(v[e]) : 0.f) + (c2 != 0.f ? c2 * o.x : 0.f);
                    y[e + 1] = (a != 0.f ? a * __uint_as_float(v[e + 1]) : 0.f) + (c2 != 0.f ? c2 * o.y : 0.f);
                    y[e + 2] = (a != 0.f ? a * __uint_as_float(v[e + 2]) : 0.f) + (c2 != 0.f ? c2 * o.z : 0.f);
                    y[e + 3] = (a != 0.f ? a * __uint_as_float(v[e + 3]) : 0.f) + (c2 != 0.f ? c2 * o.w : 0.f);
                }
                if (row_ok) {
                    // column pi(d) holds dim d; pi flips bits 1 and 2 by the 32-dim
                    // block 2g + c
                    const int flip = 2 * (2 * g + c);
#pragma unroll
                    for (int d = 0; d < 32; d += 4) {
                        float4 w;
                        // (flip is 0, 2, 4 or 6: whole pairs move, so a float4 is two pairs)
                        w = make_float4(y[d], y[d + 1], y[d + 2], y[d + 3]);
                        const float2 first = make_float2(w.x, w.y), second = make_float2(w.z, w.w);
                        *reinterpret_cast<float2*>(po + 32 * c + (d ^ flip)) = first;
                        *reinterpret_cast<float2*>(po + 32 * c + ((d + 2) ^ flip)) = second;
                    }
                }
            }
            if (g == 0 && row_ok)
                reinterpret_cast<float2*>(p.part_ml)[slot_row] = make_float2(M, a * l_sum + c2 * ol);
        }
        tc_fence_before();
        __syncthreads();   // Q', the exchange and the tensor memory are free for the next segment
        tc_fence_after();
        tbase += ntiles;
        pos += ntiles;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(*tslot, 512);
}

// A warp per output row: merge the partials of the CTAs over the row's unit by
// their log-sum-exp weights, four at a time, apply 16 v_rescale / l, leave the
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
    if (den > 0.f) inv = p.v_rescale / (kPScale * den);
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
    e = launch_pdl(tq_tree_kernel<KB, VB>, dim3(p.num_ctas), dim3(256), C::kSmemAlloc, stream, p, *kmap);
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
