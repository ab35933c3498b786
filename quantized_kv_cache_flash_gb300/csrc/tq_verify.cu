// Verification of drafted tokens (tq_verify_tree): which path of a drafted tree
// the target's probabilities accept, and the token that follows it.
//
// At the path's end v the target's row p and the draft's row q are known.  Its
// children, in order, are tried against what is left of the target's row: with
// r_0 = p and Z_0 = 1, child c of token x is accepted where u_c q(x) Z_k < r_k(x);
// a rejection leaves r_{k+1} = max(r_k - Z_k q, 0), Z_{k+1} = sum r_{k+1}.  When no
// child is left the next token is drawn from r: the first whose running sum passes
// u_0 times the whole.  (Dividing r by its sum, as the rule is usually written,
// changes neither the tests nor the draw.)  The accepted path and the token are
// then distributed as the target's own samples.  Without draft rows a child is a
// point mass at its token.
//
// Decisions at a border must not depend on the order of a sum, so every value is an
// integer: a probability is taken to 2^-56 (less than what a sum in 64-bit floating
// point loses), sums are exact and the same however the row is split.
//
// A cluster of 8 CTAs takes a sequence.  All of them walk the tree alike, on the
// first tests' numbers, which are fetched together at the start; where a sum over
// the vocabulary is needed each reads an eighth of the rows and the sums meet in
// distributed shared memory.
#include <cooperative_groups.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace cg = cooperative_groups;

constexpr int kVerCtas = 8;              // of a cluster
constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerNodes = TQ_MAX_TREE_NODES;

// What is not above 0 (a NaN) counts as 0, what is above 1 as 1.
__device__ __forceinline__ float unit(float x) { return x > 0.f ? fminf(x, 1.f) : 0.f; }
// x of [0, 1] in units of 2^-56.
__device__ __forceinline__ uint64_t to_q56(float x) { return __float2ull_rz(unit(x) * 72057594037927936.f); }
// A uniform number in units of 2^-64.
__device__ __forceinline__ uint64_t to_q64(float u) {
    u = unit(u);
    return u < 1.f ? __float2ull_rz(u * 18446744073709551616.f) : ~0ull;
}
__device__ __forceinline__ uint64_t mul_q56(uint64_t a, uint64_t b) {
    return (__umul64hi(a, b) << 8) | ((a * b) >> 56);
}
__device__ __forceinline__ uint64_t sub_to_0(uint64_t a, uint64_t b) { return a > b ? a - b : 0ull; }

struct VerifyShared {
    int parent[kVerNodes];     // -1: never tried
    int token[kVerNodes];
    float u[kVerNodes], p[kVerNodes], q[kVerNodes];   // p, q: of the node's token after its parent
    uint64_t z[kVerNodes];     // Z_k at the path's end
    int gone[kVerNodes];       // without draft rows: the tokens rejected there
    int path[kVerNodes];
    uint64_t warp_sum[kVerWarps];
    uint64_t cta_sum[2][kVerCtas];
    int cur, k, len, done;
    int tested;                // the child rejected last
};

// What is left of a token after k rejections.
template <bool DRAFT>
__device__ __forceinline__ uint64_t left_of(const VerifyShared& s, int k, float p, float q, int token) {
    uint64_t w = to_q56(p);
    if constexpr (DRAFT) {
        const uint64_t d = to_q56(q);
        for (int j = 0; j < k; ++j) w = sub_to_0(w, mul_q56(s.z[j], d));
    } else {
        for (int j = 0; j < k; ++j)
            if (s.gone[j] == token) w = 0ull;
    }
    return w;
}

// Elements 4 x .. 4 x + 3 of a row that starts `off` floats behind a 16-byte
// boundary (base: that boundary); those outside [off, end) are 0.
__device__ __forceinline__ float4 row4(const float* base, int x, int off, int end) {
    const int c = 4 * x;
    if (c >= off && c + 4 <= end) return __ldg(reinterpret_cast<const float4*>(base) + x);
    float4 v;
    v.x = c >= off && c < end ? __ldg(base + c) : 0.f;
    v.y = c + 1 >= off && c + 1 < end ? __ldg(base + c + 1) : 0.f;
    v.z = c + 2 >= off && c + 2 < end ? __ldg(base + c + 2) : 0.f;
    v.w = c + 3 >= off && c + 3 < end ? __ldg(base + c + 3) : 0.f;
    return v;
}

template <bool DRAFT>
__global__ void __cluster_dims__(kVerCtas, 1, 1) __launch_bounds__(kVerThreads)
    tq_verify_kernel(const __grid_constant__ VerifyParams p) {
    __shared__ VerifyShared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int b = static_cast<int>(blockIdx.x) / kVerCtas;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_wait();
    griddep_launch_dependents();
    const size_t row0 = static_cast<size_t>(b) * p.nodes;

    // ---- the nodes, and the numbers of each one's first test ----
    bool bad = false;
    for (int i = tid; i < p.nodes; i += kVerThreads) {
        const int up = p.parents[static_cast<size_t>(b) * p.parents_per_seq + i];
        const int x = p.tokens[row0 + i];
        s.u[i] = p.uniforms[row0 + i];
        s.token[i] = x;
        const bool tried = i > 0 && up >= 0 && up < i && x >= 0 && x < p.vocab;
        // (the first node's token and parent say nothing; -1 is a padding node)
        bad = bad || (i > 0 && up != -1 && !tried);
        s.parent[i] = tried ? up : -1;
        s.p[i] = tried ? __ldg(p.target + (row0 + up) * p.ld_target + x) : 0.f;
        s.q[i] = !tried ? 0.f : DRAFT ? __ldg(p.draft + (row0 + up) * p.ld_draft + x) : 1.f;
    }
    if (bad && rank == 0) atomicOr(p.status, kStatusBadIndex);
    if (tid == 0) {
        s.cur = 0;
        s.k = 0;
        s.len = 1;
        s.path[0] = 0;
        s.z[0] = 1ull << 56;
        // (stands where no element is found: a row without positive entries, or whose sum
        // passes 2^8; the warp that finds one writes after a cluster barrier)
        if (rank == 0) p.next[b] = 0;
    }
    __syncthreads();

    // Sum of what is left of row `cur` after k rejections, over this CTA's part
    // (a contiguous run of elements a warp); then over the cluster.
    int sweeps = 0;
    int run0 = 0, run1 = 0, off = 0;   // this warp's groups of 4 elements; the row's offset
    auto left4 = [&](const float* pr, const float* qr, int x, int k, bool aligned, uint64_t (&w)[4]) {
        const int end = off + p.vocab;
        const float4 a = row4(pr, x, off, end);
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        if constexpr (DRAFT) {
            if (k > 0) {
                if (aligned) {
                    const float4 v = row4(qr, x, off, end);
                    d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (4 * x + e >= off && 4 * x + e < end) d[e] = __ldg(qr + 4 * x + e);
                }
            }
        }
        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = left_of<DRAFT>(s, k, av[e], d[e], 4 * x + e - off);
    };
    const float *pr = nullptr, *qr = nullptr;
    bool aligned = true;
    auto rows_of = [&](int cur) {
        const float* a = p.target + (row0 + cur) * p.ld_target;
        off = static_cast<int>((reinterpret_cast<uintptr_t>(a) >> 2) & 3);
        pr = a - off;
        if constexpr (DRAFT) {   // (indexed like the target's row)
            qr = p.draft + (row0 + cur) * p.ld_draft - off;
            aligned = (reinterpret_cast<uintptr_t>(qr) & 15u) == 0;
        }
        const int groups = (off + p.vocab + 3) / 4;
        const int per = (groups + kVerCtas * kVerWarps - 1) / (kVerCtas * kVerWarps);
        run0 = min(groups, (rank * kVerWarps + warp) * per);
        run1 = min(groups, run0 + per);
    };
    auto sweep = [&](int cur, int k) {
        rows_of(cur);
        uint64_t sum = 0;
        for (int x = run0 + lane; x < run1; x += 32) {
            uint64_t w[4];
            left4(pr, qr, x, k, aligned, w);
            sum += (w[0] + w[1]) + (w[2] + w[3]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s.warp_sum[warp] = sum;
        __syncthreads();
        const int par = sweeps++ & 1;
        if (tid < kVerCtas) {
            uint64_t all = 0;
            for (int i = 0; i < kVerWarps; ++i) all += s.warp_sum[i];
            // (two slots: a CTA may be at its next sweep before another has read this one)
            *cluster.map_shared_rank(&s.cta_sum[par][rank], tid) = all;
        }
        cluster.sync();
        uint64_t all = 0;
        for (int i = 0; i < kVerCtas; ++i) all += s.cta_sum[par][i];
        return all;
    };

    // ---- the walk ----
    for (;;) {
        if (warp == 0) {
            int cur = s.cur, k = s.k, len = s.len;
            int tested = len > 1 ? s.path[len - 1] : 0;
            if (k > 0) tested = s.tested;
            int done = 0;
            for (;;) {
                int child = -1;
                for (int w = (tested + 1) & ~31; w < p.nodes && child < 0; w += 32) {
                    const int i = w + lane;
                    const unsigned hit =
                        __ballot_sync(0xffffffffu, i > tested && i < p.nodes && s.parent[i] == cur);
                    if (hit) child = w + __ffs(hit) - 1;
                }
                if (child < 0) {
                    done = 1;
                    break;
                }
                tested = child;
                bool yes;
                if (k == 0) {   // (a product of 48 bits: exact)
                    yes = double(unit(s.u[child])) * double(unit(s.q[child])) < double(unit(s.p[child]));
                } else {
                    const uint64_t w = left_of<DRAFT>(s, k, s.p[child], s.q[child], s.token[child]);
                    yes = __umul64hi(to_q64(s.u[child]), mul_q56(s.z[k], to_q56(s.q[child]))) < w;
                }
                if (!yes) break;   // (the sum of what is left comes next)
                cur = child;
                k = 0;
                if (lane == 0) s.path[len] = child;
                ++len;
            }
            __syncwarp();
            if (lane == 0) {
                s.cur = cur;
                s.len = len;
                s.done = done;
                if (!done) {
                    if constexpr (!DRAFT) s.gone[k] = s.token[tested];
                    s.tested = tested;
                    s.k = k + 1;
                } else {
                    s.k = k;
                }
            }
        }
        __syncthreads();
        if (s.done) break;
        const int k = s.k;
        const uint64_t z = sweep(s.cur, k);
        __syncthreads();
        if (tid == 0) s.z[k] = z;
        __syncthreads();
    }

    // ---- the token that follows ----
    int k = s.k;
    const int cur = s.cur;
    // (after a rejection the last sweep left its sums)
    uint64_t all = 0;
    if (k > 0) {
        for (int i = 0; i < kVerCtas; ++i) all += s.cta_sum[(sweeps - 1) & 1][i];
    }
    if (all == 0) {   // a leaf, or nothing left: the target's row itself
        k = 0;
        all = sweep(cur, 0);
        __syncthreads();
    }
    if (all == 0) {
        if (rank == 0 && tid == 0) atomicOr(p.status, kStatusBadValue);
    } else {
        uint64_t t = __umul64hi(to_q64(s.u[0]), all);
        // the CTA, the warp and the element whose running sum passes t < all
        uint64_t before = 0;
        for (int i = 0; i < rank; ++i) before += s.cta_sum[(sweeps - 1) & 1][i];
        for (int i = 0; i < warp; ++i) before += s.warp_sum[i];
        if (t >= before && t - before < s.warp_sum[warp]) {   // (one warp of the cluster)
            t -= before;
            for (int x0 = run0; x0 < run1; x0 += 32) {
                uint64_t w[4] = {0, 0, 0, 0};
                if (x0 + lane < run1) left4(pr, qr, x0 + lane, k, aligned, w);
                const uint64_t own = (w[0] + w[1]) + (w[2] + w[3]);
                uint64_t inc = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, inc > t);
                if (hit) {
                    if (lane == __ffs(hit) - 1) {
                        uint64_t run = inc - own;
                        int e = 0;
                        for (; e < 3; ++e) {
                            run += w[e];
                            if (run > t) break;
                        }
                        p.next[b] = min(4 * (x0 + lane) + e - off, p.vocab - 1);
                    }
                    break;
                }
                t -= __shfl_sync(0xffffffffu, inc, 31);
            }
        }
    }
    if (rank == 0) {
        for (int i = tid; i < p.nodes; i += kVerThreads) p.keep[row0 + i] = i < s.len ? s.path[i] : -1;
        if (tid == 0) p.num_keep[b] = s.len;
    }
    cluster.sync();   // (no CTA leaves while another may still write to its shared memory)
}

int launch_verify(const VerifyParams& p, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.batch) * kVerCtas);
    if (p.draft != nullptr) return launch_pdl(tq_verify_kernel<true>, grid, dim3(kVerThreads), 0, stream, p);
    return launch_pdl(tq_verify_kernel<false>, grid, dim3(kVerThreads), 0, stream, p);
}

}  // namespace tq
