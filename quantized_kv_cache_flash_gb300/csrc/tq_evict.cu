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
#include <cooperative_groups.h>

#include <algorithm>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelKeysMax = 48 * 1024;   // keys that shared memory holds (192 KB); more are read anew a pass

// Integers in the weights' order; NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);   // (-0 + 0 = 0)
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) tq_evict_select_kernel(const __grid_constant__ EvictParams p) {
    extern __shared__ uint32_t s_keys[];
    __shared__ uint32_t s_hist[kSelBins];
    __shared__ uint32_t s_warp[kSelWarps], s_warp2[kSelWarps];
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
    if (flag) return;
    int32_t* kept = p.kept + static_cast<size_t>(blockIdx.x) * p.max_keep;
    if (L <= n) {
        for (int i = tid; i < L; i += kSelThreads) kept[i] = i;
        return;
    }
    // tokens [lo, hi) are weighed, m of them kept (0 <= m < hi - lo)
    const int lo = p.sinks, hi = L - p.recent, m = n - p.sinks - p.recent;
    const float* w = p.weights + static_cast<size_t>(blockIdx.x) * p.src_cap;
    const bool held = L <= p.keys_held;
    uint32_t prefix = 0, need = static_cast<uint32_t>(m);   // digits so far; how many of the keys with them are kept
    auto key_at = [&](int t) { return held ? s_keys[t] : weight_key(__ldg(w + t)); };
    if (m > 0) {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const int bins = pass == 2 ? 1024 : 2048;
            for (int i = tid; i < bins; i += kSelThreads) s_hist[i] = 0;
            __syncthreads();
            if (pass == 0) {
                for (int t = lo + tid; t < hi; t += kSelThreads) {
                    const uint32_t key = weight_key(__ldg(w + t));
                    if (held) s_keys[t] = key;
                    atomicAdd(&s_hist[key >> 21], 1u);
                }
            } else {
                const int above = shift + (pass == 1 ? 11 : 10);
                for (int t = lo + tid; t < hi; t += kSelThreads) {
                    const uint32_t key = key_at(t);
                    if ((key >> above) == (prefix >> above)) atomicAdd(&s_hist[(key >> shift) & (bins - 1)], 1u);
                }
            }
            __syncthreads();
            // the bin whose keys, with those of the bins above it, first make `need`:
            // thread i has bins from the top, per of them
            const int per = bins / kSelThreads;
            uint32_t mine = 0;
            for (int e = 0; e < per; ++e) mine += s_hist[bins - 1 - (tid * per + e)];
            uint32_t inc = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31) s_warp[warp] = inc;
            __syncthreads();
            for (int i = 0; i < warp; ++i) inc += s_warp[i];
            if (inc >= need && inc - mine < need) {   // (one thread)
                uint32_t run = inc - mine;
                int e = 0;
                for (; e < per; ++e) {
                    const uint32_t c = s_hist[bins - 1 - (tid * per + e)];
                    if (run + c >= need) break;
                    run += c;
                }
                s_digit = static_cast<uint32_t>(bins - 1 - (tid * per + e));
                s_above = run;
            }
            __syncthreads();
            prefix |= s_digit << shift;
            need -= s_above;
        }
    }
    // a warp's run of tokens (whole groups of 32): how many it keeps for sure, and
    // how many are equal to the smallest
    const int groups = (L + 31) / 32, per = (groups + kSelWarps - 1) / kSelWarps;
    const int g0 = min(groups, warp * per), g1 = min(groups, g0 + per);
    auto look = [&](int t, bool& sure, bool& same) {
        sure = t < L && (t < lo || t >= hi);
        same = false;
        if (m > 0 && t >= lo && t < hi) {
            const uint32_t key = key_at(t);
            sure = key > prefix;
            same = key == prefix;
        }
    };
    uint32_t sures = 0, sames = 0;
    for (int g = g0; g < g1; ++g) {
        bool sure, same;
        look(32 * g + lane, sure, same);
        sures += __popc(__ballot_sync(0xffffffffu, sure));
        sames += __popc(__ballot_sync(0xffffffffu, same));
    }
    __syncthreads();   // (s_warp of the last pass is read)
    if (lane == 0) {
        s_warp[warp] = sures;
        s_warp2[warp] = sames;
    }
    __syncthreads();
    uint32_t at = 0, equal = 0;   // kept tokens and equal ones before the run
    for (int i = 0; i < warp; ++i) {
        at += s_warp[i];
        equal += s_warp2[i];
    }
    at += min(equal, need);
    const uint32_t below = (1u << lane) - 1u;
    for (int g = g0; g < g1; ++g) {
        bool sure, same;
        look(32 * g + lane, sure, same);
        const unsigned same_mask = __ballot_sync(0xffffffffu, same);
        const bool keep = sure || (same && equal + __popc(same_mask & below) < need);
        const unsigned mask = __ballot_sync(0xffffffffu, keep);
        if (keep) kept[at + __popc(mask & below)] = 32 * g + lane;
        at += __popc(mask);
        equal += __popc(same_mask);
    }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveCtas = kEvictMoveCtas;

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
    // (in place every CTA of the cluster makes the same number of rounds)
    for (int r0 = INPLACE ? 0 : first * R; r0 < count; r0 += step * R) {
        const int i0 = INPLACE ? r0 + first * R : r0;
        const int m = min(R, count - i0);   // (may be below 1)
        __syncthreads();
        for (int i = tid; i < m; i += kMoveThreads) s_from[i] = kept[i0 + i];
        __syncthreads();
        uint4 k[NK], v[NV];
#pragma unroll
        for (int e = 0; e < NK; ++e) {
            const int x = tid + e * kMoveThreads, i = x / CK;
            if (i < m && moves) k[e] = ks[static_cast<size_t>(s_from[i]) * CK + (x - i * CK)];
        }
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            const int x = tid + e * kMoveThreads, i = x / CV;
            if (i < m && moves) v[e] = vs[static_cast<size_t>(s_from[i]) * CV + (x - i * CV)];
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
    static std::atomic<uint64_t> attr_done{0};
    cudaError_t e = set_smem_attr_once(tq_evict_select_kernel, kSelKeysMax * 4, attr_done);
    if (e != cudaSuccess) return e;
    p.keys_held = p.max_len <= kSelKeysMax ? p.max_len : 0;
    e = launch_pdl(tq_evict_select_kernel, dim3(p.batch * p.hkv), dim3(kSelThreads), size_t(p.keys_held) * 4, stream, p);
    if (e != cudaSuccess) return e;
    if (p.rbk == 256 && p.rbv == 64) return launch_move<16, 4>(p, stream);
    if (p.rbk == 256 && p.rbv == 48) return launch_move<16, 3>(p, stream);
    if (p.rbk == 64 && p.rbv == 64) return launch_move<4, 4>(p, stream);
    if (p.rbk == 64 && p.rbv == 48) return launch_move<4, 3>(p, stream);
    if (p.rbk == 48 && p.rbv == 48) return launch_move<3, 3>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace tq
