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
// Decisions at a border need more than fp32: what is left of a token is a pair of fp32
// numbers (differences and products with their rounding errors, 2^-48 or less off), a
// thread's sum is such a pair (2^-49 off per number added), and from there on sums are
// integers in units of 2^-52, of which a thread drops less than two: 2^-37 for the 2^14
// threads of a cluster.  (Everything as 64-bit integers took 63 us for 8 trees
// of 64 nodes over 131,072 tokens; a test in 64-bit floating point alone 1 us.)
//
// A cluster of 1 to 16 CTAs takes a sequence.  All of them walk the tree alike, on the
// first tests' numbers, which are fetched together at the start; where a sum over
// the vocabulary is needed each reads its part of the rows and sends its sum to all, with
// the mbarrier that the first warp of each waits on.
//
// 8 trees of 64 nodes over 131,072 tokens: 17 to 21 us, 64 looked-up chains of 11 over 50,001: 12,
// one drafted chain of 6 over 32,000: 8.3.  What is read (8 MB, 13 MB, 0.3 MB) would take 1.2,
// 1.9 and 0.04: the time is the chain of dependent steps, some 3 us a sum over a vocabulary (the
// row from memory, 128 elements a warp in double fp32 numbers, the exchange).
#include <cooperative_groups.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace cg = cooperative_groups;

constexpr int kVerCtas = 16;             // of a cluster, at most
constexpr int kVerThreads = 1024;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerNodes = TQ_MAX_TREE_NODES;
constexpr int kVerGroups = 2;            // groups of 4 elements that a thread holds
constexpr float kUnits = 4503599627370496.f;    // 2^52
// Sums are cut so that none wraps, whatever the rows hold: those of a lane and a warp at
// 2^5, of a CTA at 2^7.
constexpr uint64_t kMostWarp = 1ull << 57, kMostCta = 1ull << 59;

// What is not above 0 (a NaN) counts as 0, what is above 1 as 1.
__device__ __forceinline__ float unit(float x) { return x > 0.f ? fminf(x, 1.f) : 0.f; }
// A uniform number in units of 2^-64.
__device__ __forceinline__ uint64_t to_q64(float u) {
    u = unit(u);
    return u < 1.f ? __float2ull_rz(u * 18446744073709551616.f) : ~0ull;
}

// A number as a sum of two fp32 ones, |l| at most half a step of h.
struct Two {
    float h, l;
};
// In units of 2^-52 (of a number that is not below 0).
__device__ __forceinline__ uint64_t to_units(Two x) {
    const long long n = __float2ll_rz(x.h * kUnits) + __float2ll_rz(x.l * kUnits);
    return n > 0 ? static_cast<uint64_t>(n) : 0ull;
}
__device__ __forceinline__ Two from_units(uint64_t n) {   // (n <= 2^63, in pieces of 27, 24 and 12 bits)
    const float a = static_cast<float>(static_cast<uint32_t>(n >> 36)) * 1.52587890625e-5f;   // 2^-16
    const float b = static_cast<float>(static_cast<uint32_t>(n >> 12) & 0xffffffu) * 9.094947017729282e-13f;   // 2^-40
    const float c = static_cast<float>(static_cast<uint32_t>(n) & 0xfffu) * 2.220446049250313e-16f;   // 2^-52
    const float h = __fadd_rn(a, b);
    return Two{h, __fadd_rn(__fsub_rn(b, __fsub_rn(h, a)), c)};
}
__device__ __forceinline__ void add_to(Two& sum, Two x) {   // Knuth's two-sum, then the low parts
    const float s = __fadd_rn(sum.h, x.h), v = __fsub_rn(s, sum.h);
    const float e = __fadd_rn(__fsub_rn(sum.h, __fsub_rn(s, v)), __fsub_rn(x.h, v));
    sum.h = s;
    sum.l = __fadd_rn(sum.l, __fadd_rn(e, x.l));
}
// max(w - z q, 0)
__device__ __forceinline__ Two less(Two w, Two z, float q) {
    const float ph = __fmul_rn(z.h, q);
    const float pl = __fmaf_rn(z.l, q, __fmaf_rn(z.h, q, -ph));   // (Dekker's product, with an fma)
    const float s = __fsub_rn(w.h, ph), v = __fsub_rn(s, w.h);
    const float e = __fsub_rn(__fsub_rn(w.h, __fsub_rn(s, v)), __fadd_rn(ph, v));
    const float t = __fadd_rn(e, __fsub_rn(w.l, pl));
    const float h = __fadd_rn(s, t);
    return h > 0.f ? Two{h, __fsub_rn(t, __fsub_rn(h, s))} : Two{0.f, 0.f};
}

// Bounded wait for a phase of a barrier that other CTAs complete.
__device__ __forceinline__ bool wait_for_sums(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 255u) == 0 && global_timer_ns() - t0 > 2000000000ull) return false;
    }
}

struct VerifyShared {
    int parent[kVerNodes];     // -1: never tried
    int token[kVerNodes];
    float u[kVerNodes], p[kVerNodes], q[kVerNodes];   // p, q: of the node's token after its parent
    Two z[kVerNodes];          // Z_k at the path's end, k > 0
    uint32_t first[kVerNodes / 32];   // bit i: accepted if it is its parent's first child to be tried
    int gone[kVerNodes];       // without draft rows: the tokens rejected there
    int path[kVerNodes];
    uint64_t warp_sum[kVerWarps];
    uint64_t cta_sum[2][kVerCtas];
    int cur, k, len, done;
    int tested;                // the child rejected last
    uint64_t bar[2];           // the sums of every second sweep are here
};

// What is left of a token after rejection j, from what was before.
template <bool DRAFT>
__device__ __forceinline__ Two reject(const VerifyShared& s, int j, Two w, float q, int token) {
    if constexpr (!DRAFT) return s.gone[j] == token ? Two{0.f, 0.f} : w;
    if (j > 0) return less(w, s.z[j], q);
    const float h = __fsub_rn(w.h, q);   // (Z_0 = 1; exact with its error where p > q)
    return h > 0.f ? Two{h, __fsub_rn(__fsub_rn(w.h, h), q)} : Two{0.f, 0.f};
}
// Whether u q z < w.
__device__ __forceinline__ bool accepts(float u, float q, Two z, Two w) {
    const float h = __fmul_rn(u, q), l = __fmaf_rn(u, q, -h);     // u q, exactly
    const float ph = __fmul_rn(z.h, h);
    const float pl = __fmaf_rn(z.h, l, __fmaf_rn(z.l, h, __fmaf_rn(z.h, h, -ph)));
    // (the difference of the high parts is exact where they are near one another)
    return __fadd_rn(__fsub_rn(ph, w.h), __fsub_rn(pl, w.l)) < 0.f;
}

// A number to the shared memory of CTA `rank` of the cluster (the place and barrier that
// this CTA has at these addresses), whose barrier counts its 8 bytes.
__device__ __forceinline__ void send_u64(uint32_t at, uint32_t bar, int rank, uint64_t x) {
    asm volatile(
        "{\n .reg .b32 a, b;\n mapa.shared::cluster.u32 a, %0, %2;\n mapa.shared::cluster.u32 b, %1, %2;\n"
        " st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [a], %3, [b];\n}\n" ::"r"(at),
        "r"(bar), "r"(rank), "l"(x)
        : "memory");
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
__global__ void __launch_bounds__(kVerThreads, 1)
    tq_verify_kernel(const __grid_constant__ VerifyParams p) {
    __shared__ VerifyShared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int ctas = static_cast<int>(cluster.num_blocks());
    const int b = static_cast<int>(blockIdx.x) / ctas;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t bar = smem_u32(s.bar);
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(bar + 8, 1);
        fence_barrier_init();
    }
    __syncwarp();
    // (met before the first sum is sent: the other CTAs run and their barriers are there)
    cluster_arrive();
    griddep_wait();
    griddep_launch_dependents();
    const size_t row0 = static_cast<size_t>(b) * p.nodes;

    // ---- the nodes, and the numbers of each one's first test ----
    bool bad = false;
    static_assert(kVerNodes <= kVerThreads && kVerWarps == 32, "a node a thread, a warp's sum a lane");
    bool first = false;
    if (tid < p.nodes) {
        const int i = tid;
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
        first = accepts(unit(s.u[i]), unit(s.q[i]), Two{1.f, 0.f}, Two{unit(s.p[i]), 0.f});
    }
    const unsigned first_mask = __ballot_sync(0xffffffffu, first);
    if (lane == 0 && warp < kVerNodes / 32) s.first[warp] = first_mask;
    if (bad && rank == 0) atomicOr(p.status, kStatusBadIndex);
    if (tid == 0) {
        s.cur = 0;
        s.k = 0;
        s.len = 1;
        s.path[0] = 0;
    }
    __syncthreads();

    // Sum of what is left of row `cur` after k rejections, over this CTA's part
    // (a contiguous run of elements a warp); then over the cluster.
    int sweeps = 0;
    bool stalled = false;   // (warp 0) a sum did not come in time
    int run0 = 0, run1 = 0, off = 0;   // this warp's groups of 4 elements; the row's offset
    const float *pr = nullptr, *qr = nullptr;
    bool aligned = true;
    // a batch of groups x0 + lane + 32 i: what is left of the target's numbers, the draft's
    Two w[kVerGroups][4];
    float q[kVerGroups][4];
    auto load = [&](int x0) {
        const int end = off + p.vocab;
        float4 a[kVerGroups], d[kVerGroups];
#pragma unroll
        for (int i = 0; i < kVerGroups; ++i) {
            const int x = x0 + lane + 32 * i;
            a[i] = d[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x < run1) {
                a[i] = row4(pr, x, off, end);
                if constexpr (DRAFT) {
                    if (aligned) {
                        d[i] = row4(qr, x, off, end);
                    } else {
                        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (4 * x + e >= off && 4 * x + e < end) v[e] = __ldg(qr + 4 * x + e);
                        d[i] = make_float4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kVerGroups; ++i) {
            const float av[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, dv[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[i][e] = Two{unit(av[e]), 0.f};
                q[i][e] = unit(dv[e]);
            }
        }
    };
    auto apply = [&](int x0, int j0, int j1) {   // rejections j0 .. j1 - 1
#pragma unroll 1
        for (int j = j0; j < j1; ++j)
#pragma unroll
            for (int i = 0; i < kVerGroups; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[i][e] = reject<DRAFT>(s, j, w[i][e], q[i][e], 4 * (x0 + lane + 32 * i) + e - off);
    };
    auto rows_of = [&](int cur) {
        const float* a = p.target + (row0 + cur) * p.ld_target;
        off = static_cast<int>((reinterpret_cast<uintptr_t>(a) >> 2) & 3);
        pr = a - off;
        if constexpr (DRAFT) {   // (indexed like the target's row)
            qr = p.draft + (row0 + cur) * p.ld_draft - off;
            aligned = (reinterpret_cast<uintptr_t>(qr) & 15u) == 0;
        }
        const int groups = (off + p.vocab + 3) / 4;
        const int log2 = 5 + (31 - __clz(ctas));   // warps of the cluster
        const int per = (groups + (1 << log2) - 1) >> log2;
        run0 = min(groups, (rank * kVerWarps + warp) * per);
        run1 = min(groups, run0 + per);
        return per <= 32 * kVerGroups;
    };
    bool held = false;            // the batch is the warp's whole run of the row,
    int held_cur = -1, held_k = 0;  // of this node after that many rejections
    auto sweep = [&](int cur, int k) {
        if (cur != held_cur) held = rows_of(cur);
        Two part{0.f, 0.f};
        for (int x0 = run0; x0 < run1; x0 += 32 * kVerGroups) {
            if (!held || held_cur != cur || held_k > k) {
                load(x0);
                held_k = 0;
            }
            apply(x0, held_k, k);
#pragma unroll
            for (int i = 0; i < kVerGroups; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) add_to(part, w[i][e]);
        }
        held_cur = cur;
        held_k = k;
        uint64_t sum = min(to_units(part), kMostWarp);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum = min(sum, kMostWarp);
        if (lane == 0) s.warp_sum[warp] = sum;
        __syncthreads();
        // (two places and barriers in turn: a CTA may send its next sum before another has
        // all of this one)
        const int par = sweeps & 1;
        if (warp == 0) {
            uint64_t all = s.warp_sum[lane];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
            if (lane == 0) mbar_arrive_expect_tx(bar + 8 * par, 8 * ctas);
            __syncwarp();
            if (lane < ctas) send_u64(smem_u32(&s.cta_sum[par][rank]), bar + 8 * par, lane, min(all, kMostCta));
            stalled = stalled || !wait_for_sums(bar + 8 * par, (sweeps >> 1) & 1);
        }
        ++sweeps;
    };
    // The whole of the last sweep, for every lane of a warp.
    auto whole = [&]() {
        uint64_t all = lane < ctas ? s.cta_sum[(sweeps - 1) & 1][lane] : 0ull;
#pragma unroll
        for (int o = kVerCtas / 2; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        return __shfl_sync(0xffffffffu, all, 0);
    };

    cluster_wait();
    // ---- the walk ----
    const int up0 = lane < p.nodes ? s.parent[lane] : -1;   // (the first 32 nodes' at hand)
    for (;;) {
        if (warp == 0) {
            int cur = s.cur, k = s.k, len = s.len;
            int tested = k > 0 ? s.tested : cur;   // (children come after their parent)
            int done = 0;
            for (;;) {
                int child = -1;
                if (tested < 31) {
                    const unsigned hit = __ballot_sync(0xffffffffu, lane > tested && up0 == cur);
                    if (hit) child = __ffs(hit) - 1;
                }
                for (int x = max(32, (tested + 1) & ~31); child < 0 && x < p.nodes; x += 32) {
                    const int i = x + lane;
                    const unsigned hit = __ballot_sync(0xffffffffu, i > tested && i < p.nodes && s.parent[i] == cur);
                    if (hit) child = x + __ffs(hit) - 1;
                }
                if (child < 0) {
                    done = 1;
                    break;
                }
                tested = child;
                bool yes;
                if (k == 0) {
                    yes = (s.first[child >> 5] >> (child & 31)) & 1u;
                } else {
                    Two left{unit(s.p[child]), 0.f};
                    const float q = unit(s.q[child]);
                    for (int j = 0; j < k; ++j) left = reject<DRAFT>(s, j, left, q, s.token[child]);
                    yes = accepts(unit(s.u[child]), q, s.z[k], left);
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
        sweep(s.cur, s.k);
        if (warp == 0) {
            const uint64_t z = whole();
            if (lane == 0) s.z[s.k] = from_units(z);
            __syncwarp();
        }
    }

    // ---- the token that follows ----
    int k = s.k;
    const int cur = s.cur;
    // (after a rejection the last sweep left its sums)
    // (the other warps see the sums that warp 0 waited for behind a barrier: that of the
    // walk, or the one here)
    uint64_t all = k > 0 ? whole() : 0ull;
    if (all == 0) {   // a leaf, or nothing left: the target's row itself
        k = 0;
        sweep(cur, 0);
        __syncthreads();
        all = whole();
    }
    if (__syncthreads_or(stalled) && tid == 0) atomicOr(p.status, kStatusPipelineStall);
    __syncwarp();   // (the barrier is met by whole warps)
    // (met at the end: no CTA leaves while another may still send to it)
    cluster_arrive();
    if (all == 0) {
        if (rank == 0 && tid == 0) {
            p.next[b] = 0;
            atomicOr(p.status, kStatusBadValue);
        }
    } else {
        uint64_t t = __umul64hi(to_q64(s.u[0]), all);
        // the CTA, the warp and the element whose running sum passes t < all
        uint64_t before = (lane < rank ? s.cta_sum[(sweeps - 1) & 1][lane] : 0ull) + (lane < warp ? s.warp_sum[lane] : 0ull);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
        if (t >= before && t - before < s.warp_sum[warp]) {   // (one warp of the cluster)
            t -= before;
            bool found = false;
            int last = -1;   // the last token with anything left, so far
            for (int x0 = run0; x0 < run1 && !found; x0 += 32 * kVerGroups) {
                if (!held) {
                    load(x0);
                    apply(x0, 0, k);
                }
#pragma unroll
                for (int i = 0; i < kVerGroups; ++i) {
                    if (found) continue;   // (uniform)
                    const int at = 4 * (x0 + lane + 32 * i) - off;   // the first of the lane's four tokens
                    uint64_t n[4], own = 0;
                    int mine = -1;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        own += n[e] = to_units(w[i][e]);
                        if (w[i][e].h > 0.f) mine = at + e;
                    }
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
                                run += n[e];
                                if (run > t) break;
                            }
                            p.next[b] = min(at + e, p.vocab - 1);
                        }
                        found = true;
                    }
                    last = max(last, __reduce_max_sync(0xffffffffu, mine));
                    t -= __shfl_sync(0xffffffffu, inc, 31);
                }
            }
            // (the threads' sums and these differ in the last places: t may lie between)
            if (!found && last >= 0 && lane == 0) p.next[b] = last;
        }
    }
    if (rank == 0) {
        for (int i = tid; i < p.nodes; i += kVerThreads) p.keep[row0 + i] = i < s.len ? s.path[i] : -1;
        if (tid == 0) p.num_keep[b] = s.len;
    }
    __syncwarp();
    cluster_wait();
}

template <bool DRAFT>
static int launch_t(const VerifyParams& p, cudaStream_t stream) {
    static std::atomic<uint64_t> attr_done{0};
    const cudaError_t e = allow_large_clusters_once(tq_verify_kernel<DRAFT>, attr_done);
    if (e != cudaSuccess) return e;
    // As many CTAs as fit at once, one per SM (a chain of 5 over 131,072 tokens: 16 CTAs 14.8
    // us, 8 16.5, 4 20.8, 2 29.8, 1 47.5; over 32,000 13.4, 13.5, 14.4, 16.7, 21.0).  Of clusters
    // of 16 seven run at once: more sequences take 8 where their registers hold the rows (8
    // chains of 5 over 50,000: 15.2 us and 20.4; 8 stars of 16 over 131,072: 23.2 and 21.6).
    int ctas = kVerCtas;
    while (ctas > 1 && 1ll * p.batch * ctas > host::kSMs) ctas /= 2;
    if (ctas == 16 && p.batch > 7 && p.vocab <= 8 * kVerThreads * 4 * kVerGroups) ctas = 8;
    return launch_pdl_cluster(tq_verify_kernel<DRAFT>, dim3(static_cast<unsigned>(p.batch) * ctas), dim3(kVerThreads),
                              ctas, 0, stream, p);
}

int launch_verify(const VerifyParams& p, cudaStream_t stream) {
    return p.draft != nullptr ? launch_t<true>(p, stream) : launch_t<false>(p, stream);
}

}  // namespace tq
