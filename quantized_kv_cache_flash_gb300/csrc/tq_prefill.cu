// Chunked-prefill attention over the packed KV cache on the 5th-generation
// tensor cores (tcgen05, accumulators in tensor memory).
//
// Same result as the decode kernels -- query j of a Tq block attends to
// tokens [0, L - Tq + j] of its sequence, scores and P.V in the rotated basis,
// only the output inverse-rotated (mlxcel pull request #369, Change) -- for
// blocks of many queries (a prefill chunk), where every K/V tile serves 128
// query rows and the two products are dense GEMMs:
//   S[128 rows x 128 tok]  = Q'[128 x 128] . K^T     (8 or 16 MMAs of K = 16, fp32 in TMEM)
//   O[128 rows x 128 dim] += P[128 x 128 tok] . V    (8 MMAs, fp32 in TMEM)
// Q' = Rot(q) (quantized K) or q (fp16 K); the softmax scale * log2(e) and
// the K norm are applied to the fp32 scores.  fp16 K: q and K are fp16
// inputs, their products exact.  Quantized K: Rot(q) is not an fp16 value,
// so it is split into q_hi = fp16(Rot q) and q_lo = fp16(Rot q - q_hi) and S
// takes both products (16 MMAs of K = 16 per query tile instead of 8); the K
// tile holds the fp16 centroids c[idx], exact for a codebook of fp16 values
// (other codebooks are not taken by this kernel).  K and V are dequantised
// once per tile into shared memory (the 128-byte-swizzled K-major layout the
// MMA descriptors read); V transposed, [dim][token], as fp16 c[idx] * n_v (a
// tile has half as many V values as P values, so the norm goes there).
//
// CTA = 256 threads on one (batch, kv head, pair of 128-row query tiles):
// thread = one query row (tensor-memory lane) of one tile, so each K/V tile is
// dequantised once for 256 rows.  Tensor memory holds, per query tile, S (128
// columns, whose first 64 take P back as fp16 pairs for the P.V MMA) and O
// (128 columns): all 512.  The MMAs overlap the CUDA-core work and the two
// query tiles take turns on the tensor core: S(n) runs while tile 1's warps
// dequantise V(n), S_1(n) during tile 0's softmax, P.V_0(n) during tile 1's,
// and tile 0's warps dequantise K(n + 1) during tile 1's softmax and
// P.V_1(n).  Packed records of the next tiles
// stream into two staging slots by bulk copies (fp16 K by 2-D tensor-map
// copies straight into the MMA layout); every mbarrier wait is bounded.
#include <float.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

template <int KB, int VB>
struct PreCfg {
    static constexpr int kTile = 128;                           // tokens per tile = rows per CTA
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
    static constexpr int kNvOff = kColOff + kTile * 4;          // packed: fp32 n_v [128], the largest of 32 [4]
    // mbarriers stg[2], S[2], O[2] (one per query tile), V^T stored, K stored,
    // tile 1's softmax done; TMEM slot; last tile copied; the CTA's item (packed)
    static constexpr int kBarOff = kNvOff + kTile * 4 + 16;
    static constexpr int kSmem = kBarOff + 88;
    static constexpr int kSmemAlloc = kSmem + 896;              // to a 1024-byte boundary from a 128-byte one
    static_assert(kSmemAlloc <= 232448, "227 KB per CTA");
    static constexpr uint32_t kIdesc = umma_idesc_f16_f32(128, 128);
};

// Packed sequences: which query tile pair a CTA takes.  All pairs of all
// sequences are ranked by the K/V tiles they read, most first (the grid then
// ends on the shortest ones), and rank k of every KV head goes to the CTAs
// k hkv .. k hkv + hkv - 1, so CTAs that start together read different KV
// heads of the same tokens.  A pair's tile count grows with its place in the
// sequence, so the pairs of a sequence that read more than c tiles are its last
// ones, and their number is one division; the smallest c that leaves at most k
// pairs above it is found by bisection, one warp adding the sequences up.
struct PackedSeq {
    int n, ctx, lim;   // query rows, tokens before them, tokens read at most
};

__device__ __forceinline__ PackedSeq packed_seq(const PrefillParams& p, int b) {
    PackedSeq s{0, 0, 0};
    if (b >= p.batch) return s;
    const int first = p.cu[b], next = p.cu[b + 1], L = p.lengths[b];
    if (first < 0 || next < first || next > p.total) return s;   // no rows (flagged by the first CTA)
    s.n = next - first;
    s.ctx = L - s.n;
    s.lim = min(L, p.max_len);
    return s;
}

// Pairs (of `span` positions each) of a sequence that read more than c tiles.
__device__ __forceinline__ int pairs_above(const PackedSeq& s, int c, int span) {
    const int all = (s.n + span - 1) / span;
    if (c < 0) return all;
    // pair q reads past tile c where its last row does: its last token, the
    // smaller of ctx + min(n, (q + 1) span) - 1 and lim - 1, is at 128 c or after
    const int need = 128 * c + 1 - s.ctx;   // positions up to that row
    if (128 * c >= s.lim || need > s.n) return 0;
    return all - (need <= span ? 0 : (need - 1) / span);
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// (sequence, pair) of rank k, by one warp; b = -1 past the last one.
__device__ __forceinline__ void packed_find(const PrefillParams& p, int k, int lane, int& b, int& pair) {
    const int span = 2 * p.pos_per_tile;
    const PackedSeq mine = packed_seq(p, lane);
    auto above = [&](int c) {
        int v = pairs_above(mine, c, span);
        for (int bb = 32 + lane; bb < p.batch; bb += 32) v += pairs_above(packed_seq(p, bb), c, span);
        return warp_sum(v);
    };
    b = -1;
    pair = 0;
    if (k >= above(-1)) return;
    int lo = -1, hi = (p.max_len + 127) / 128;   // above(lo) > k >= above(hi) = 0
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (above(mid) > k) lo = mid;
        else hi = mid;
    }
    // the pairs of hi tiles, sequence after sequence
    int left = k - above(hi);
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const PackedSeq s = b0 == 0 ? mine : packed_seq(p, b0 + lane);
        const int skip = pairs_above(s, hi, span), here = pairs_above(s, hi - 1, span) - skip;
        int inc = here;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, inc > left);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int all = (s.n + span - 1) / span;
            b = b0 + l;
            pair = __shfl_sync(0xffffffffu, all - skip - here + (left - (inc - here)), l);
            return;
        }
        left -= __shfl_sync(0xffffffffu, inc, 31);
    }
}

template <int KB, int VB, bool PACKED>
__global__ void __launch_bounds__(256, 1)
    tq_prefill_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap kmap) {
    using C = PreCfg<KB, VB>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    // thread = (query tile tl of the CTA's two, row r = TMEM lane): warps 0-3
    // hold the rows of the first tile, warps 4-7 those of the second
    const int tl = tid >> 7, r = tid & 127;

    // this CTA's (batch, kv head, query tile pair), the sequence's query rows
    // and query tiles and its row 0 in packed q and out
    int b, h, pair, tqn, mtiles, qrow0 = 0;
    if constexpr (PACKED) {
        griddep_wait();
        int* s_item = reinterpret_cast<int*>(smem + C::kBarOff + 80);
        if (warp == 0) {
            int fb, fp;
            packed_find(p, static_cast<int>(blockIdx.x) / p.hkv, tid, fb, fp);
            if (tid == 0) {
                s_item[0] = fb;
                s_item[1] = fp;
            }
        } else if (warp == 1 && blockIdx.x == 0) {
            bool bad = false;
            for (int bb = tid - 32; bb < p.batch; bb += 32)
                bad = bad || p.cu[bb] < 0 || p.cu[bb + 1] < p.cu[bb] || p.cu[bb + 1] > p.total;
            if (bad) atomicOr(p.status, kStatusBadIndex);
        }
        __syncthreads();
        b = s_item[0];
        pair = s_item[1];
        if (b < 0) return;   // past the last pair (uniform over the CTA)
        h = static_cast<int>(blockIdx.x) % p.hkv;
        qrow0 = p.cu[b];
        tqn = p.cu[b + 1] - qrow0;
        mtiles = (tqn + p.pos_per_tile - 1) / p.pos_per_tile;
    } else {
        // heaviest (latest) query tiles first
        mtiles = p.mtiles;
        pair = (mtiles + 1) / 2 - 1 - static_cast<int>(blockIdx.x);
        b = blockIdx.y / p.hkv;
        h = blockIdx.y - b * p.hkv;
        tqn = p.tq;
        griddep_wait();  // cache, lengths and q come from earlier work on the stream
    }
    const int mt = 2 * pair + tl;
    const int unit = b * p.hkv + h;
    const int L = p.lengths[b];
    const int t_lim = min(L, p.max_len);
    // row r of tile mt: query position j, head hl of the group
    const int jl = r / p.group, hl = r - jl * p.group;
    const int j = mt * p.pos_per_tile + jl;
    const bool row_ok = mt < mtiles && jl < p.pos_per_tile && j < tqn;
    const int lim = row_ok ? min(L - tqn + j, t_lim - 1) : -1;  // last visible token
    // this tile's rows see every token up to lim_lo; the CTA's tiles end at `last`
    const int lim_lo = mt < mtiles ? min(L - tqn + mt * p.pos_per_tile, t_lim - 1) : -1;
    const int j_hi = min(tqn - 1, (2 * pair + 2) * p.pos_per_tile - 1);
    const int last = min(L - tqn + j_hi, t_lim - 1);
    // this row of q and out
    const size_t io = (PACKED ? (static_cast<size_t>(qrow0) + j) * p.hq + h * p.group + hl
                              : (static_cast<size_t>(b) * p.hq + h * p.group + hl) * tqn + j) * kD;
    const int ntiles = last >= 0 ? last / C::kTile + 1 : 0;
    const size_t row0 = static_cast<size_t>(unit) * p.cap;

    uint8_t* sQ = smem + C::kQOff;       // [2][128 x 128] fp16
    uint8_t* sVt = smem + C::kVtOff;
    // n_k * scale * log2(e) per token (quantized K), written with K's dequant
    float* colK = reinterpret_cast<float*>(smem + C::kColOff);
    const uint32_t bar_stg = smem_u32(smem + C::kBarOff);       // 2 x 8 bytes
    const uint32_t bar_s = bar_stg + 16, bar_o = bar_stg + 32, bar_v = bar_stg + 48;
    const uint32_t bar_kr = bar_stg + 56, bar_sm1 = bar_stg + 64;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 72);
    int* last_issued = reinterpret_cast<int*>(smem + C::kBarOff + 76);  // last tile whose copy was issued

    auto issue = [&](int n) {  // one thread: tile n into staging slot n & 1
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

    if (tid == 0) {
        for (int i = 0; i < 6; ++i) mbar_init(bar_stg + 8 * i, 1);  // stg[2], S[2], O[2]
        mbar_init(bar_v, 128);  // the V dequant's threads
        mbar_init(bar_kr, 1);
        mbar_init(bar_sm1, 1);
        fence_barrier_init();
        for (int n = 0; n < 2 && n < ntiles; ++n) issue(n);
        *last_issued = min(ntiles, 2) - 1;
    }
    // tensor memory: tile t at columns 256 t: S (128, its first 64 reused for
    // P as fp16 pairs), then O (128)
    if (warp == 0) tmem_alloc(smem_u32(tslot), 512);

    // ---- Q' = Rot(q) as q_hi + q_lo (quantized K) or q (fp16 K) ----
    uint8_t* sQt = sQ + tl * 32768;
    uint8_t* sQlt = smem + C::kQloOff + tl * 32768;
    {
        float x[128];
        if (row_ok) {
            const __half* qp = p.q + io;
#pragma unroll
            for (int k = 0; k < 128; k += 8) {
                const uint4 w = *reinterpret_cast<const uint4*>(qp + k);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ww[e]));
                    x[k + 2 * e] = f.x;
                    x[k + 2 * e + 1] = f.y;
                }
            }
            if constexpr (KB != 0) {
#pragma unroll
                for (int k = 0; k < 128; ++k) x[k] = ((p.signs[k >> 5] >> (k & 31)) & 1u) ? -x[k] : x[k];
                wht128_thread(x);
#pragma unroll
                for (int k = 0; k < 128; k += 2) {  // 1/sqrt(128)
                    const float2 v = __fmul2_rn(make_float2(x[k], x[k + 1]),
                                                make_float2(0.08838834764831845f, 0.08838834764831845f));
                    x[k] = v.x;
                    x[k + 1] = v.y;
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 128; ++k) x[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 128; k += 8) {
            uint32_t hv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) hv[e] = pack_half2(x[k + 2 * e], x[k + 2 * e + 1]);
            *reinterpret_cast<uint4*>(sQt + sw128_offset(r, k)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
            if constexpr (KB != 0) {  // q_lo = Rot(q) - q_hi (exact in fp32), rounded once more
                uint32_t lv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&hv[e]));
                    lv[e] = pack_half2(x[k + 2 * e] - hf.x, x[k + 2 * e + 1] - hf.y);
                }
                *reinterpret_cast<uint4*>(sQlt + sw128_offset(r, k)) = make_uint4(lv[0], lv[1], lv[2], lv[3]);
            }
        }
    }
    fence_proxy_async();  // the MMAs read Q' through the async proxy
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + 256 * tl + lane_off;         // this row of S (and of P)
    const uint32_t t_o = tmem + 256 * tl + 128 + lane_off;   // this row of O

    float m_base = -INFINITY, l_sum = 0.f;
    bool stalled = false;  // once set, waits return at once and no MMA or copy is issued
    int issued_o = 0;      // P.V batches of this thread's query tile
    const uint32_t bar_st = bar_s + 8 * tl, bar_ot = bar_o + 8 * tl;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!stalled && !mbar_wait_bounded(bar, parity)) stalled = true;
    };

    // K(n) -> sK, one token per thread of query tile 0's warps (fp16 K: the
    // tile is read in place from the staging slot)
    auto k_dequant = [&](int n) {
        if constexpr (KB != 0) {
            // (tables from the parameters at each use: none held across the loop)
            const Tables kt{p.ktab[0], p.ktab[1], p.ktab[2], p.ktab[3]};
            const uint8_t* rec = smem + C::kStgOff + (n & 1) * C::kSlot + r * C::kRbK;
            uint8_t* sK = smem + C::kKOff;
            // (packed: the quarters in an order that differs between lanes whose
            // records start in the same banks)
            const int turn = PACKED ? (KB == 4 ? r >> 1 : r >> 3) : 0;
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
    };
    // colK of tile n (n_k * scale * log2 e per token, 0 past the end)
    // (packed: in the order of the softmax's fragments, with the V norms, 0 past
    // the end; one that overflowed counts as 65504, since 0 * inf would be NaN in the
    // rows before its token, and not for the slack)
    auto k_scales = [&](int n) {
        const uint8_t* slot = smem + C::kStgOff + (n & 1) * C::kSlot;
        const bool in = n * C::kTile + r < t_lim;
        if constexpr (KB != 0) {
            const float nk = __half2float(reinterpret_cast<const __half*>(slot + C::kSK)[r]);
            colK[PACKED ? frag_place(r) : r] = in ? nk * p.scale_log2e : 0.f;
        }
        if constexpr (PACKED) {
            const float nv = in ? __half2float(reinterpret_cast<const __half*>(slot + C::kSK + C::kSKn + C::kSV)[r]) : 0.f;
            float* nvs = reinterpret_cast<float*>(smem + C::kNvOff);
            nvs[frag_place(r)] = fminf(nv, 65504.f);
            // (non-negative floats order like their bits)
            const uint32_t top = __reduce_max_sync(0xffffffffu, nv < 65536.f ? __float_as_uint(nv) : 0u);
            if ((r & 31) == 0) reinterpret_cast<uint32_t*>(nvs + C::kTile)[r >> 5] = top;
        }
    };
    // S_t(n) = Q'_t . K(n)^T into tile t's S columns
    auto issue_s = [&](int n, int t2) {
        const uint32_t kbase = (KB == 0) ? smem_u32(smem + C::kStgOff + (n & 1) * C::kSlot) : smem_u32(smem + C::kKOff);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            const uint32_t koff = (kk >> 2) * 16384 + (kk & 3) * 32;
            umma_f16(tmem + 256 * t2, umma_desc_sw128(smem_u32(sQ) + t2 * 32768 + koff),
                     umma_desc_sw128(kbase + koff), C::kIdesc, kk > 0 ? 1u : 0u);
            if constexpr (KB != 0)  // + q_lo . K^T
                umma_f16(tmem + 256 * t2, umma_desc_sw128(smem_u32(smem + C::kQloOff) + t2 * 32768 + koff),
                         umma_desc_sw128(kbase + koff), C::kIdesc, 1u);
        }
        umma_commit(bar_s + 8 * t2);
    };
    // O_t += P_t(n) . V(n), P from tensor memory over S_t
    auto issue_pv = [&](int n, int t2) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            const uint32_t koff = (kk >> 2) * 16384 + (kk & 3) * 32;
            umma_f16_ts(tmem + 256 * t2 + 128, tmem + 256 * t2 + 8 * kk,
                        umma_desc_sw128(smem_u32(sVt) + koff), C::kIdesc, (n > 0 || kk > 0) ? 1u : 0u);
        }
        umma_commit(bar_o + 8 * t2);
    };
    // V(n)^T for the 16 tokens 16 vw .. 16 vw + 15 (query tile 1's warps take
    // vw = warp - 4 and vw = warp): thread (g, t) = lane 4g + t dequantises
    // quarter t of tokens 16vw+g and 16vw+g+8 (the MMA fragment layout, so
    // stmatrix.trans writes [dim][token] rows); V^T rows are stored in the order
    // pi(d) = d ^ 2(d >> 5), which puts the 8 rows of each stored 8x8 matrix in
    // 8 different 16-byte bank groups (the epilogue reads O's columns back
    // through the same pi)
    auto v_dequant = [&](int n, int vw) {
        const Tables vt{p.vtab[0], p.vtab[1], p.vtab[2], p.vtab[3]};
        const uint8_t* slot = smem + C::kStgOff + (n & 1) * C::kSlot;
        [[maybe_unused]] const int tok0 = n * C::kTile;
        const int lane = tid & 31, g = lane >> 2, tq4 = lane & 3;
        const int ta = 16 * vw + g, tb = ta + 8;
        const uint8_t* vrec = slot + C::kSK + C::kSKn;
        [[maybe_unused]] const __half* vnorm = reinterpret_cast<const __half*>(slot + C::kSK + C::kSKn + C::kSV);
        // tokens past the end: stale records still decode to finite
        // centroids, and their norm (and weight) is 0
        uint32_t ha[16], hb[16];
        dequant_q32<VB>(vrec + ta * C::kRbV + tq4 * (C::kRbV / 4), vt, ha);
        dequant_q32<VB>(vrec + tb * C::kRbV + tq4 * (C::kRbV / 4), vt, hb);
        // n_v scales the stored values, so P itself goes to the MMA: 128 x
        // 128 multiplies a tile instead of the 256 x 128 of scaling P.  (Packed: P
        // takes the norm and V stays the centroids, exact, so a term is rounded once.)
        if constexpr (!PACKED) {
            const __half2 na = tok0 + ta < t_lim ? __half2half2(vnorm[ta]) : __float2half2_rn(0.f);
            const __half2 nb = tok0 + tb < t_lim ? __half2half2(vnorm[tb]) : __float2half2_rn(0.f);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const __half2 a = __hmul2(*reinterpret_cast<const __half2*>(&ha[k]), na);
                const __half2 b = __hmul2(*reinterpret_cast<const __half2*>(&hb[k]), nb);
                ha[k] = *reinterpret_cast<const uint32_t*>(&a);
                hb[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        // stmatrix k2 stores dim pairs 2k2 (matrices 0, 1: tokens A, B) and
        // 2k2+1 (matrices 2, 3); lane 8j + c gives row c of matrix j: dim
        // d = 32(c>>1) + 2(2k2 + (j>>1)) + (c&1), tokens 16vw + 8(j&1) .. + 7
        const int sj = lane >> 3, sc = lane & 7;
        const int tokc = 2 * (vw & 3) + (sj & 1);  // 16-byte chunk of the tokens in their row
        uint32_t vaddr[2];
#pragma unroll
        for (int par = 0; par < 2; ++par) {
            const int row = 32 * (sc >> 1) + 2 * ((((par << 1) | (sj >> 1)) ^ (sc >> 1)) & 3) + (sc & 1);
            vaddr[par] = smem_u32(sVt) + (vw >> 2) * 16384 + row * 128 + ((tokc ^ (row & 7)) << 4);
        }
#pragma unroll
        for (int k2 = 0; k2 < 8; ++k2)
            stsm_x4_trans(vaddr[k2 & 1] + 1024 * (k2 >> 1), ha[2 * k2], hb[2 * k2], ha[2 * k2 + 1],
                          hb[2 * k2 + 1]);
    };
    // softmax_t(n) of this thread's row (log2 domain): P over S_t's first 64
    // columns as fp16 pairs; O_t rescaled in place when the row's base moves
    auto softmax = [&](int n) {
        const int tok0 = n * C::kTile;
        float x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(t_s + 32 * c, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) x[32 * c + e] = __uint_as_float(v[e]);
        }
        // t = s * n_k * scale * log2(e) - base in one FFMA per score; the base moves only when a
        // score passes it by more than 4 (so p <= 16 in fp16)
        const bool fresh = (m_base == -INFINITY);
        const float base0 = fresh ? 0.f : m_base;
        // (packed pairs: one instruction per two scores)
        const float2 nb2 = make_float2(-base0, -base0);
#pragma unroll
        for (int e = 0; e < 128; e += 4) {
            const float sl = p.scale_log2e;
            float4 nk = make_float4(sl, sl, sl, sl);
            if constexpr (KB != 0) nk = *reinterpret_cast<const float4*>(colK + e);
            const float2 a = __ffma2_rn(make_float2(x[e], x[e + 1]), make_float2(nk.x, nk.y), nb2);
            const float2 b = __ffma2_rn(make_float2(x[e + 2], x[e + 3]), make_float2(nk.z, nk.w), nb2);
            x[e] = a.x;
            x[e + 1] = a.y;
            x[e + 2] = b.x;
            x[e + 3] = b.y;
        }
        if (tok0 + C::kTile - 1 > lim_lo) {  // a tile some row of this query tile sees in part
#pragma unroll
            for (int e = 0; e < 128; ++e)
                if (tok0 + e > lim) x[e] = -INFINITY;
        }
        // row max over four independent chains (16 deep instead of 64)
        float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 128; e += 8)
#pragma unroll
            for (int j = 0; j < 4; ++j) mq[j] = fmaxf(mq[j], fmaxf(x[e + 2 * j], x[e + 2 * j + 1]));
        const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
        const bool grow = fresh ? (mx > -INFINITY) : (mx > 4.f);
        if (__any_sync(0xffffffffu, grow)) {
            // rows that grow move their base up by mx (t -= mx below); the others keep it
            const float shift = grow ? mx : 0.f;
            const float alpha = grow ? (fresh ? 0.f : fast_exp2(-mx)) : 1.f;
            l_sum *= alpha;
            if (grow) m_base = base0 + mx;  // a row that saw no token yet keeps no base
#pragma unroll
            for (int e = 0; e < 128; ++e) x[e] -= shift;
            if (issued_o > 0) {  // rescale this row of O in tensor memory (P.V(n-1) is done)
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
        // row sum as four independent packed pairs (chains 16 deep instead of 64)
        float2 s2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const int k = 64 * c + 2 * e;
                const float p0 = fast_exp2(x[k]), p1 = fast_exp2(x[k + 1]);
                s2[e & 3] = __fadd2_rn(s2[e & 3], make_float2(p0, p1));
                pk[e] = pack_half2(p0, p1);
            }
            tmem_st32(t_s + 32 * c, pk);  // P over S columns 0..63 (tokens 64c..64c+63)
        }
        const float2 sa = __fadd2_rn(s2[0], s2[1]), sb = __fadd2_rn(s2[2], s2[3]);
        const float2 st = __fadd2_rn(sa, sb);
        l_sum += st.x + st.y;
    };

    // Packed: the same as MMA fragments.  Lane 4v + c of a warp has rows v + 8q (q =
    // 0..3) of its 32 and columns 2c, 2c + 1 of every eight, so a thread reads a
    // quarter of the tile's scales and norms.  A tile that every row sees takes one
    // pass, P in registers until it is known that no score passes its row's base by
    // more than the slack (which shows in the thread's sums); then, with the mask,
    // and on a row's first tile, the rows' maxima are taken first.
    float fm[4], fl[4];   // base (log2) and this thread's part of the sum
    int flim[4];          // last visible token
    if constexpr (PACKED) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int rq = 32 * (warp & 3) + ((tid & 31) >> 2) + 8 * q, jq = rq / p.group;
            fm[q] = -INFINITY;
            fl[q] = 0.f;
            flim[q] = mt < mtiles && jq < p.pos_per_tile && mt * p.pos_per_tile + jq < tqn
                          ? min(L - tqn + mt * p.pos_per_tile + jq, t_lim - 1)
                          : -1;
        }
    }
    auto softmax_frag = [&](int n) {
        const int lane = tid & 31, tok0 = n * C::kTile;
        const float* col = colK + 4 * (lane & 3);
        const float* nvs = reinterpret_cast<const float*>(smem + C::kNvOff) + 4 * (lane & 3);
        const float4 nm = *reinterpret_cast<const float4*>(smem + C::kNvOff + C::kTile * 4);
        // p n_v stays below 2^15.99
        const float slack =
            fmaxf(0.f, fminf(10.f, 15.99f - __log2f(fmaxf(fmaxf(nm.x, nm.y), fmaxf(nm.z, nm.w)))));
        const float most = fast_exp2(slack);
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
                    alpha[q] = up ? (fresh ? 0.f : fast_exp2(-mx)) : 1.f;
                    fl[q] *= alpha[q];
                    if (up) fm[q] = (fresh ? 0.f : fm[q]) + mx;
                    grow = grow || up;
                }
                if (issued_o > 0 && __any_sync(0xffffffffu, grow)) {   // rescale O (P.V(n-1) is done)
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

    // Query tile 0's warps (0-3) dequantise K and its scales and issue S_0 and
    // P.V_0 (thread 0); query tile 1's warps (4-7) dequantise V and issue S_1,
    // P.V_1 and the copies (thread 128).  Per K/V tile n the tensor core takes
    // S_0(n), S_1(n) (named barrier 3 keeps that order), P.V_0(n), P.V_1(n):
    // tile 0's softmax runs under S_1, tile 1's under P.V_0 and the K(n+1)
    // dequant.  The two groups hand over through mbarriers: bar_kr (K(n) and
    // its scales stored), bar_v (V(n)^T stored), bar_sm1 (tile 1's softmax(n)
    // is past its reads of the scales).  No thread leaves the loop early, so
    // every named barrier is met; after a wait times out the thread's later
    // waits return at once and it issues nothing more.
    if (tl == 0 && ntiles > 0) {
        wait(bar_stg, 0);
        k_dequant(0);
        k_scales(0);
    }
    for (int n = 0; n < ntiles; ++n) {
        if (tl == 0) {
            tc_fence_before();
            named_bar_sync(1, 128);  // K(n) and its scales are stored
            tc_fence_after();
            if (r == 0) {
                mbar_arrive(bar_kr);
                if (n > 0) wait(bar_o, (n - 1) & 1);  // P.V_0(n-1) has read P_0
                tc_fence_after();
                if (!stalled) issue_s(n, 0);
            }
            __syncwarp();
            if (warp == 0) named_bar_arrive(3, 64);  // S_0(n) is queued: S_1(n) may follow
            if (n > 0) wait(bar_o, (n - 1) & 1);    // O_0 and the P_0 columns are free
        } else {
            // V(n), once its records landed and both P.V(n-1) have read V(n-1)^T
            wait(bar_stg + 8 * (n & 1), (n >> 1) & 1);
            if (n > 0) {
                wait(bar_o, (n - 1) & 1);
                wait(bar_o + 8, (n - 1) & 1);
            }
            v_dequant(n, warp - 4);
            v_dequant(n, warp);
            fence_proxy_async();
            mbar_arrive(bar_v);
            if (warp == 4) {
                named_bar_sync(3, 64);
                if (r == 0) {
                    tc_fence_after();
                    if (!stalled) issue_s(n, 1);
                }
                __syncwarp();
            }
            wait(bar_kr, n & 1);  // the scales of tile n are stored
        }
        wait(bar_st, n & 1);
        tc_fence_after();
        if constexpr (PACKED) softmax_frag(n);
        else softmax(n);
        tc_fence_before();
        if (named_bar_or(1 + tl, 128, stalled)) stalled = true;  // P_tl(n) is stored
        tc_fence_after();
        if (tl == 0) {
            if (r == 0) {
                wait(bar_v, n & 1);  // V(n)^T is stored
                tc_fence_after();
                if (!stalled) issue_pv(n, 0);
            }
            if (n + 1 < ntiles) {  // K(n+1), under tile 1's softmax(n)
                wait(bar_stg + 8 * ((n + 1) & 1), ((n + 1) >> 1) & 1);
                wait(bar_s + 8, n & 1);  // S_1(n) has read K(n)
                k_dequant(n + 1);
                wait(bar_sm1, n & 1);    // tile 1's softmax(n) is done with the scales
                k_scales(n + 1);
            }
        } else if (r == 0) {
            // P.V_1(n) first: S_0(n+1) queues behind it on the tensor core
            mbar_arrive(bar_sm1);   // tile 1's softmax(n) is past its reads of the scales
            tc_fence_after();
            if (!stalled) issue_pv(n, 1);
            wait(bar_s, n & 1);     // S_0(n) is done (fp16 K reads it from the slot)
            if (!stalled && n + 2 < ntiles) {  // tile n's staging slot is consumed
                issue(n + 2);
                *last_issued = n + 2;
            }
        }
        ++issued_o;
    }

    // ---- epilogue: O / l, v_rescale, inverse rotation, fp16 ----
    bool ok = !stalled;
    if (issued_o > 0 && !mbar_wait_bounded(bar_ot, (issued_o - 1) & 1)) ok = false;
    ok = __syncthreads_and(ok) != 0;  // one decision for the whole CTA
    tc_fence_after();
    if constexpr (PACKED) {   // the sums, a row per thread from here on
        float* rows = reinterpret_cast<float*>(smem + C::kColOff);   // (scales and norms are read; 256 floats)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float l = fl[q] + __shfl_xor_sync(0xffffffffu, fl[q], 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if ((tid & 3) == 0) rows[128 * tl + 32 * (warp & 3) + ((tid & 31) >> 2) + 8 * q] = l;
        }
        __syncwarp();
        l_sum = rows[tid];
    }
    if (!ok) {
        if (tid == 0) atomicOr(p.status, kStatusPipelineStall);
    } else {
        float o[128];
        if (issued_o > 0) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // every lane: the loads are warp-collective
                uint32_t v[32];
                tmem_ld32(t_o + 32 * c, v);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[32 * c + e] = __uint_as_float(v[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 128; ++e) o[e] = 0.f;
        }
        if (row_ok) {
            float inv = 0.f;
            if (l_sum > 0.f) inv = p.v_rescale / l_sum;
            else atomicOr(p.status, kStatusShortContext);
            // 1/l, v_rescale and the rotation's 1/sqrt(128), applied after the
            // (linear) transform in one packed multiply
            const float g = inv * 0.08838834764831845f;
            // O's column pi(d) holds dim d (V^T rows were stored in pi order)
            float od[128];
#pragma unroll
            for (int d = 0; d < 128; ++d) od[d] = o[d ^ (2 * (d >> 5))];
#pragma unroll
            for (int d = 0; d < 128; ++d) o[d] = od[d];
            wht128_thread(o);
            __half* op = p.out + io;
#pragma unroll
            for (int k = 0; k < 128; k += 8) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 v = __fmul2_rn(make_float2(o[k + e], o[k + e + 1]), make_float2(g, g));
                    y[e] = ((p.signs[(k + e) >> 5] >> ((k + e) & 31)) & 1u) ? -v.x : v.x;
                    y[e + 1] = ((p.signs[(k + e + 1) >> 5] >> ((k + e + 1) & 31)) & 1u) ? -v.y : v.y;
                }
                *reinterpret_cast<uint4*>(op + k) = make_uint4(pack_half2(y[0], y[1]), pack_half2(y[2], y[3]),
                                                               pack_half2(y[4], y[5]), pack_half2(y[6], y[7]));
            }
        }  // padding rows write nothing
    }
    if (!ok) {
        // let the copies still in flight land before the shared memory goes away
        const int li = *last_issued;
        for (int m = li > 0 ? li - 1 : 0; m <= li; ++m)
            (void)mbar_wait_bounded(bar_stg + 8 * (m & 1), (m >> 1) & 1);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int KB, int VB>
static int launch_prefill_t(const PrefillParams& p, const CUtensorMap* kmap, cudaStream_t stream) {
    using C = PreCfg<KB, VB>;
    if (p.cu != nullptr) {
        static std::atomic<uint64_t> attr_done{0};
        const cudaError_t e = set_smem_attr_once(tq_prefill_kernel<KB, VB, true>, C::kSmemAlloc, attr_done);
        if (e != cudaSuccess) return e;
        return launch_pdl(tq_prefill_kernel<KB, VB, true>, dim3(p.slots * p.hkv), dim3(256), C::kSmemAlloc, stream, p,
                          *kmap);
    }
    static std::atomic<uint64_t> attr_done{0};
    const cudaError_t e = set_smem_attr_once(tq_prefill_kernel<KB, VB, false>, C::kSmemAlloc, attr_done);
    if (e != cudaSuccess) return e;
    return launch_pdl(tq_prefill_kernel<KB, VB, false>, dim3((p.mtiles + 1) / 2, p.batch * p.hkv), dim3(256),
                      C::kSmemAlloc, stream, p, *kmap);
}

int launch_prefill(int kbits, int vbits, const PrefillParams& p, const CUtensorMap* kmap,
                   cudaStream_t stream) {
    if (kbits == 16 && vbits == 4) return launch_prefill_t<0, 4>(p, kmap, stream);
    if (kbits == 16 && vbits == 3) return launch_prefill_t<0, 3>(p, kmap, stream);
    if (kbits == 3 && vbits == 3) return launch_prefill_t<3, 3>(p, kmap, stream);
    if (kbits == 4 && vbits == 4) return launch_prefill_t<4, 4>(p, kmap, stream);
    if (kbits == 4 && vbits == 3) return launch_prefill_t<4, 3>(p, kmap, stream);
    return cudaErrorInvalidValue;
}

}  // namespace tq
