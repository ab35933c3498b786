// Eviction by weight (tq_cache_evict): a sequence of L tokens keeps n of them for
// each KV head, the first `sinks`, the last `recent` and of the others the heaviest
// (the first of equal ones), in their order; records, weights and the places they
// came from move to the front, within a cache or into another one.
//
// Two kernels.  The first takes a CTA per (sequence, KV head) and finds the weight
// that n leaves as the smallest kept by its digits, from the top (11 + 11 + 10 bits
// of the order-preserving integer): a histogram of the keys that share the digits
// found so far gives the next one.  Then every token is either above that weight,
// equal to it (kept while there is room) or below, and each warp writes the places of
// its run of tokens behind those of the warps before it.
// The second moves.  In place a record may only be overwritten once it has been read:
// places ascend, so record i comes from place >= i and what is written up to a round's
// end is never read by a later round; within a round the 8 CTAs of a cluster all load
// before any stores.
//
// 32 sequences of 4,000 to 16,384 tokens brought to 2,048, 8 KV heads, turbo4, into another cache:
// 45 us, the selection 16 (its three passes over keys in registers, two CTAs an SM) and the
// move 25 (90 MB read and 70 written, 0.94 of the copy bandwidth; with plain loads, for which
// L2 fetches 128 bytes a record, 141 MB read and 30 us, 50 in all: a CTA per unit that did
// both took 49.1 then, and was not measured with the loads of today); 16 ragged sequences with
// fp16 K, in place: 36 us, 10.5 and 21.5 (23 before a round's places came with the records
// before).  Digits of the distance from the least key, which are spread better: selection 18.8.
#include <cooperative_groups.h>

#include <algorithm>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace cg = cooperative_groups;

constexpr int kSelBins = 2048;

// Integers in the weights' order; NaN counts as -inf, -0 as 0.  They are 0x007fffff ..
// 0xff800000, so that 0 is left for tokens that do not exist and kKeyHeld for those that
// stay whatever their weight.
constexpr uint32_t kKeyHeld = 0xffffffffu;
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);   // (-0 + 0 = 0)
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// The lowest r bits that are set.
__device__ __forceinline__ uint32_t lowest_bits(uint32_t mask, int r) {
    if (r >= __popc(mask)) return mask;
    uint32_t got = 0;
    for (; r > 0; --r) {
        got |= mask & (0u - mask);
        mask &= mask - 1u;
    }
    return got;
}

// T threads; a warp has a run of 32 KPT tokens, lane l every 32nd from its l-th, the
// keys in registers.  KPT = 0: runs of any length, the weights read anew a pass.
template <int T, int KPT>
__global__ void __launch_bounds__(T, T == 512 ? 2 : 1) tq_evict_select_kernel(const __grid_constant__ EvictParams p) {
    constexpr int W = T / 32;
    static_assert(KPT <= 32, "a lane keeps a group's masks");
    __shared__ uint32_t s_hist[kSelBins];
    __shared__ uint32_t s_warp[W], s_warp2[W];
    __shared__ uint32_t s_digit, s_above;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = static_cast<int>(blockIdx.x) / p.hkv, h = static_cast<int>(blockIdx.x) - b * p.hkv;
    griddep_wait();
    griddep_launch_dependents();
    const int L = p.src_lengths[b], n = p.num_keep[b];
    const int count = min(L, n);
    // (the same for every head of the sequence)
    uint32_t flag = 0;
    if (L < 0 || n < 0 || n > p.max_keep || (L > n && n < p.sinks + p.recent)) flag = kStatusBadIndex;
    else if (L > p.max_len || count > p.dst_cap) flag = kStatusCapacity;
    if (h == 0 && tid == 0) {
        p.counts[b] = flag ? -1 : count;
        if (flag) atomicOr(p.status, flag);
    }
    if (flag || n == 0) return;
    int32_t* kept = p.kept + static_cast<size_t>(blockIdx.x) * p.max_keep;
    if (L <= n) {
        for (int i = tid; i < L; i += T) kept[i] = i;
        return;
    }
    const int lo = p.sinks, hi = L - p.recent;   // tokens [lo, hi) go by their weights
    // (plain loads: a kernel before this one may have written the weights after this one began)
    const float* w = p.weights + static_cast<size_t>(blockIdx.x) * p.src_cap;
    auto key_of = [&](int t, float v) { return t >= L ? 0u : t < lo || t >= hi ? kKeyHeld : weight_key(v); };
    const int groups = (L + 31) / 32, per = KPT > 0 ? KPT : (groups + W - 1) / W;
    const int g0 = warp * per, g1 = min(groups, g0 + per);
    uint32_t key[KPT > 0 ? KPT : 1];
    if constexpr (KPT > 0) {
        float v[KPT];
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const int t = 32 * (g0 + i) + lane;
            v[i] = t >= lo && t < hi ? w[t] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < KPT; ++i) key[i] = key_of(32 * (g0 + i) + lane, v[i]);
    }
    // KPT = 0: the run's groups in order, the next one's weights in flight
    auto each = [&](auto f) {
        auto at = [&](int g) {
            const int t = 32 * g + lane;
            return t >= lo && t < hi ? w[t] : 0.f;
        };
        float next = at(g0);
        for (int g = g0; g < g1; ++g) {
            const uint32_t k = key_of(32 * g + lane, next);
            next = at(g + 1);
            f(g, k);
        }
    };
    // digits so far; how many of the keys with them are kept
    uint32_t prefix = 0, need = static_cast<uint32_t>(n);
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const int bins = pass == 2 ? 1024 : 2048;
        for (int i = tid; i < bins; i += T) s_hist[i] = 0;
        __syncthreads();
        auto add = [&](uint32_t k) {
            if (pass == 0 || ((k ^ prefix) >> (pass == 1 ? 21 : 10)) == 0) atomicAdd(&s_hist[(k >> shift) & (bins - 1)], 1u);
        };
        if constexpr (KPT > 0) {
#pragma unroll
            for (int i = 0; i < KPT; ++i)
                if (pass > 0 || g0 + i < g1) add(key[i]);
        } else {
            each([&](int, uint32_t k) { add(k); });
        }
        __syncthreads();
        // the bin whose keys, with those of the bins above it, first make `need`:
        // thread i has bins from the top, `own` of them
        const int own = bins / T;
        uint32_t mine = 0;
#pragma unroll
        for (int e = 0; e < own; ++e) mine += s_hist[bins - 1 - (tid * own + e)];
        uint32_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        inc += __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0u);
        if (inc >= need && inc - mine < need) {   // (one thread)
            uint32_t run = inc - mine;
            int e = 0;
            for (; e < own; ++e) {
                const uint32_t c = s_hist[bins - 1 - (tid * own + e)];
                if (run + c >= need) break;
                run += c;
            }
            s_digit = static_cast<uint32_t>(bins - 1 - (tid * own + e));
            s_above = run;
        }
        __syncthreads();
        prefix |= s_digit << shift;
        need -= s_above;
    }
    // Tokens above the smallest kept weight stay, of those equal to it the first `need`:
    // counted over the warp's run, then over the warps, then written.
    uint32_t above = 0, same = 0;   // KPT > 0: masks of group `lane` of the run
    uint32_t n_above = 0, n_same = 0;
    if constexpr (KPT > 0) {
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const uint32_t x = __ballot_sync(0xffffffffu, key[i] > prefix), y = __ballot_sync(0xffffffffu, key[i] == prefix);
            if (lane == i) above = x, same = y;
        }
        n_above = __popc(above);
        n_same = __popc(same);
    } else {
        each([&](int, uint32_t k) {
            n_above += k > prefix;
            n_same += k == prefix;
        });
    }
    const uint32_t all_above = __reduce_add_sync(0xffffffffu, n_above), all_same = __reduce_add_sync(0xffffffffu, n_same);
    if (lane == 0) {
        s_warp[warp] = all_above;   // (read in the last pass before its last barrier)
        s_warp2[warp] = all_same;
    }
    __syncthreads();
    uint32_t equal = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp2[lane] : 0u);
    uint32_t at = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0u) + min(equal, need);
    const uint32_t below = (1u << lane) - 1u;
    if constexpr (KPT > 0) {
        uint32_t ia = n_above, is = n_same;   // inclusive sums over the run's groups
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, ia, o), y = __shfl_up_sync(0xffffffffu, is, o);
            if (lane >= o) ia += x, is += y;
        }
        const uint32_t e0 = equal + is - n_same;   // equal ones before this group
        const uint32_t keep = above | (e0 < need ? lowest_bits(same, static_cast<int>(need - e0)) : 0u);
        // (kept before it: those above, and of the equal ones what `need` allows)
        const uint32_t first = at + (ia - n_above) + (min(e0, need) - min(equal, need));
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const uint32_t mask = __shfl_sync(0xffffffffu, keep, i), base = __shfl_sync(0xffffffffu, first, i);
            if ((mask >> lane) & 1u) kept[base + __popc(mask & below)] = 32 * (g0 + i) + lane;
        }
    } else {
        each([&](int g, uint32_t k) {
            const uint32_t same_mask = __ballot_sync(0xffffffffu, k == prefix);
            const bool keep = k > prefix || (k == prefix && equal + __popc(same_mask & below) < need);
            const uint32_t mask = __ballot_sync(0xffffffffu, keep);
            if (keep) kept[at + __popc(mask & below)] = 32 * g + lane;
            at += __popc(mask);
            equal += __popc(same_mask);
        });
    }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveCtas = kEvictMoveCtas;

// 16 bytes of a record; L2 fetches no more than the record's own 64 bytes for it.
__device__ __forceinline__ uint4 load_piece(const uint4* at) {
    uint4 v;
    asm volatile("ld.global.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(at)
                 : "memory");
    return v;
}

// CK, CV: 16-byte pieces of a K and a V record.
template <int CK, int CV, bool INPLACE>
__device__ __forceinline__ void evict_move(const EvictParams& p, int unit, int first, int step) {
    constexpr int R = CK == 16 ? 128 : 256;   // records a round
    constexpr int NK = (R * CK + kMoveThreads - 1) / kMoveThreads, NV = (R * CV + kMoveThreads - 1) / kMoveThreads;
    __shared__ int s_from[R];
    const int tid = threadIdx.x;
    const int b = unit / p.hkv, h = unit - b * p.hkv;
    const int count = p.counts[b];
    const int32_t* kept = p.kept + static_cast<size_t>(unit) * p.max_keep;
    const size_t rs = static_cast<size_t>(unit) * p.src_cap, rd = static_cast<size_t>(unit) * p.dst_cap;
    const uint4* ks = reinterpret_cast<const uint4*>(p.k_src) + rs * CK;
    const uint4* vs = reinterpret_cast<const uint4*>(p.v_src) + rs * CV;
    uint4* kd = reinterpret_cast<uint4*>(p.k_dst) + rd * CK;
    uint4* vd = reinterpret_cast<uint4*>(p.v_dst) + rd * CV;
    // places ascend: where the last one is its own, all are, and records stay in place
    const bool moves = !INPLACE || (count > 0 && kept[count - 1] != count - 1);
    // (in place every CTA of the cluster makes the same number of rounds; the places of the
    // next one are fetched beside this one's records)
    static_assert(R <= kMoveThreads, "a place a thread");
    auto place = [&](int i) { return i < count && tid < R ? kept[i] : 0; };
    int next = place(first * R + tid);
    for (int r0 = INPLACE ? 0 : first * R; r0 < count; r0 += step * R) {
        const int i0 = INPLACE ? r0 + first * R : r0;
        const int m = min(R, count - i0);   // (may be below 1)
        __syncthreads();
        if (tid < R) s_from[tid] = next;
        __syncthreads();
        next = place(i0 + step * R + tid);
        uint4 k[NK], v[NV];
#pragma unroll
        for (int e = 0; e < NK; ++e) {
            const int x = tid + e * kMoveThreads, i = x / CK;
            if (i < m && moves) k[e] = load_piece(ks + static_cast<size_t>(s_from[i]) * CK + (x - i * CK));
        }
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            const int x = tid + e * kMoveThreads, i = x / CV;
            if (i < m && moves) v[e] = load_piece(vs + static_cast<size_t>(s_from[i]) * CV + (x - i * CV));
        }
        __half nk = __ushort_as_half(0), nv = __ushort_as_half(0);
        float w = 0.f;
        const bool live = tid < m;
        if (live) {
            const size_t from = rs + s_from[tid];
            if (p.kn_src != nullptr) nk = p.kn_src[from];
            if (p.vn_src != nullptr) nv = p.vn_src[from];
            if (p.new_weights != nullptr) w = p.weights[from];
        }
        if constexpr (INPLACE) cg::this_cluster().sync();
#pragma unroll
        for (int e = 0; e < NK; ++e) {
            const int x = tid + e * kMoveThreads, i = x / CK;
            if (i < m && moves) kd[static_cast<size_t>(i0) * CK + x] = k[e];
        }
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            const int x = tid + e * kMoveThreads, i = x / CV;
            if (i < m && moves) vd[static_cast<size_t>(i0) * CV + x] = v[e];
        }
        if (live) {
            const size_t to = rd + i0 + tid;
            if (p.kn_dst != nullptr) p.kn_dst[to] = nk;
            if (p.vn_dst != nullptr) p.vn_dst[to] = nv;
            if (p.new_weights != nullptr) p.new_weights[to] = w;
        }
    }
    if (h == 0 && first == 0 && tid == 0 && count >= 0) p.dst_lengths[b] = count;
}

template <int CK, int CV>
__global__ void __launch_bounds__(kMoveThreads) tq_evict_copy_kernel(const __grid_constant__ EvictParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int unit = static_cast<int>(blockIdx.x) % (p.batch * p.hkv);
    evict_move<CK, CV, false>(p, unit, static_cast<int>(blockIdx.x) / (p.batch * p.hkv), p.move_ctas);
}

template <int CK, int CV>
__global__ void __cluster_dims__(kMoveCtas, 1, 1) __launch_bounds__(kMoveThreads)
    tq_evict_inplace_kernel(const __grid_constant__ EvictParams p) {
    griddep_wait();
    griddep_launch_dependents();
    evict_move<CK, CV, true>(p, static_cast<int>(blockIdx.x) / kMoveCtas, static_cast<int>(blockIdx.x) % kMoveCtas,
                             kMoveCtas);
}

template <int CK, int CV>
static int launch_move(EvictParams& p, cudaStream_t stream) {
    const int units = p.batch * p.hkv;
    if (p.same)
        return launch_pdl(tq_evict_inplace_kernel<CK, CV>, dim3(units * kMoveCtas), dim3(kMoveThreads), 0, stream, p);
    constexpr int R = CK == 16 ? 128 : 256;
    const long long rounds = (std::min(p.max_keep, p.max_len) + R - 1) / R;
    p.move_ctas = int(std::min<long long>(rounds, std::max<long long>(1, 0x7fffffffll / units)));
    return launch_pdl(tq_evict_copy_kernel<CK, CV>, dim3(static_cast<unsigned>(units) * p.move_ctas),
                      dim3(kMoveThreads), 0, stream, p);
}

int launch_evict(EvictParams p, cudaStream_t stream) {
    // The smallest variant that holds the keys of the longest sequence in registers; 1024
    // threads where every unit has an SM of its own.  (The whole call in us, a quarter of the
    // tokens kept, 3 bits: 4 units of 8,000 tokens, 8 keys a thread of 1024 and 16 of 512: both
    // 15.5, read anew: 19.6; 256 units of 8,000: 44.2, 41.2, 52.4; 256 of 16,000, 16 of 1024:
    // 72.8, 32 of 512: 68.8, read anew: 87.2; 4 of 32,000, 32 of 1024: 24 to 26, read anew: 38.0.)
    const unsigned units = static_cast<unsigned>(p.batch) * p.hkv;
    const bool wide = units <= host::kSMs;
    auto select = [&](auto kernel, int threads) { return launch_pdl(kernel, dim3(units), dim3(threads), 0, stream, p); };
    cudaError_t e;
    if (p.max_len > 32768) e = select(tq_evict_select_kernel<1024, 0>, 1024);
    else if (p.max_len > 16384) e = select(tq_evict_select_kernel<1024, 32>, 1024);
    else if (p.max_len > 8192) e = wide ? select(tq_evict_select_kernel<1024, 16>, 1024) : select(tq_evict_select_kernel<512, 32>, 512);
    else if (p.max_len > 4096) e = wide ? select(tq_evict_select_kernel<1024, 8>, 1024) : select(tq_evict_select_kernel<512, 16>, 512);
    else e = select(tq_evict_select_kernel<512, 8>, 512);
    if (e != cudaSuccess) return e;
    if (p.rbk == 256 && p.rbv == 64) return launch_move<16, 4>(p, stream);
    if (p.rbk == 256 && p.rbv == 48) return launch_move<16, 3>(p, stream);
    if (p.rbk == 64 && p.rbv == 64) return launch_move<4, 4>(p, stream);
    if (p.rbk == 64 && p.rbv == 48) return launch_move<4, 3>(p, stream);
    if (p.rbk == 48 && p.rbv == 48) return launch_move<3, 3>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace tq
