// Record moves inside and between packed caches: keeping the accepted tokens
// of a drafted block (tq_cache_compact) and copying or forking sequences
// (tq_cache_copy).  Both move records as they are -- codes, norms, fp16 K rows
// -- so nothing is decoded and every bit stays what it was.
//
// A token of one KV head is a K row, a V row (16-byte multiples) and, but for
// table records, a 2-byte K norm (quantized K) and V norm.  Both kernels load
// everything a thread moves before it stores any of it: the loads of a CTA are
// in flight together, and a compaction in place reads its sources before it
// overwrites them.
#include <algorithm>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

// ---------------------------------------------------------------------------
// Compaction: record start + keep[i] -> record start + i, i = 0 .. n - 1, for
// every KV head; lengths[b] = start + n.
//
// keep is strictly ascending, so keep[i] >= i: a source is never below its
// destination, and 32 tokens at a time can be loaded, met at a barrier and
// stored without a later group's sources being overwritten (those lie at
// keep[i] >= i, above every destination written so far).  One CTA per (KV
// head, sequence); every CTA checks its sequence's list before it writes.
// The bytes are few (some KB per sequence): the call's time is a launch and
// two dependent trips to memory (the list, then the records): 2.2 us a call in a
// graph for 5 kept tokens of one sequence (4 KV heads, turbo3), 6 us issued one
// by one, which is the host's.
// ---------------------------------------------------------------------------
constexpr int kCompactGroup = 32;    // tokens loaded before any is stored
constexpr int kCompactThreads = 128;

__global__ void __launch_bounds__(kCompactThreads) tq_compact_kernel(const __grid_constant__ CompactParams p) {
    const int tid = threadIdx.x;
    const int b = static_cast<int>(blockIdx.x) / p.hkv, h = static_cast<int>(blockIdx.x) - b * p.hkv;
    griddep_wait();
    griddep_launch_dependents();
    const int start = p.start[b], n = p.num_keep[b];
    const int32_t* keep = p.keep + static_cast<size_t>(b) * p.max_keep;
    bool bad = start < 0 || start > p.cap - p.num_drafted || n < 0 || n > p.max_keep || n > p.num_drafted;
    if (!bad)
        for (int i = tid; i < n; i += kCompactThreads) {
            const int k = keep[i];
            bad = bad || k < 0 || k >= p.num_drafted || (i > 0 && keep[i - 1] >= k);
        }
    if (__syncthreads_or(bad)) {  // the sequence is left as it was
        if (tid == 0 && h == 0) atomicOr(p.status, kStatusBadIndex);
        return;
    }
    const size_t row0 = (static_cast<size_t>(b) * p.hkv + h) * p.cap + start;
    uint8_t* const kd = p.k_data + row0 * p.rbk;
    uint8_t* const vd = p.v_data + row0 * p.rbv;
    const int ck = p.rbk >> 4, cv = p.rbv >> 4;   // 16-byte pieces of a row (K: 3, 4 or 16; V: 3 or 4)
    for (int i0 = 0; i0 < n; i0 += kCompactGroup) {
        const int m = min(kCompactGroup, n - i0);
        uint4 k[4], v;
        __half norm = __ushort_as_half(0);
        // up to 32 x 16 pieces of K (four per thread), 32 x 4 of V, 32 + 32 norms
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int x = tid + e * kCompactThreads, i = x / ck;
            if (i < m) k[e] = reinterpret_cast<const uint4*>(kd + static_cast<size_t>(keep[i0 + i]) * p.rbk)[x - i * ck];
        }
        const int vi = tid / cv;
        if (vi < m) v = reinterpret_cast<const uint4*>(vd + static_cast<size_t>(keep[i0 + vi]) * p.rbv)[tid - vi * cv];
        const int ni = tid & 31;
        __half* const nrm = tid < 32 ? p.k_norm : tid < 64 ? p.v_norm : nullptr;
        const bool has = nrm != nullptr && ni < m;
        if (has) norm = nrm[row0 + keep[i0 + ni]];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int x = tid + e * kCompactThreads, i = x / ck;
            if (i < m) reinterpret_cast<uint4*>(kd + static_cast<size_t>(i0 + i) * p.rbk)[x - i * ck] = k[e];
        }
        if (vi < m) reinterpret_cast<uint4*>(vd + static_cast<size_t>(i0 + vi) * p.rbv)[tid - vi * cv] = v;
        if (has) nrm[row0 + i0 + ni] = norm;
        // (the next group's loads may go ahead of other threads' stores: its
        // sources lie above everything stored here)
    }
    if (h == 0 && tid == 0) p.lengths[b] = start + n;
}

int launch_compact(const CompactParams& p, cudaStream_t stream) {
    return launch_pdl(tq_compact_kernel, dim3(p.batch * p.hkv), dim3(kCompactThreads), 0, stream, p);
}

// ---------------------------------------------------------------------------
// Copy: the first n tokens of sequence src[m] of one cache become sequence
// dst[m] of a cache of the same format; n = num_tokens[m], or the whole source.
//
// A CTA moves 256 tokens of one (pair, KV head): 16-byte pieces, several per
// thread in flight.  The pairs are the fastest grid dimension, so the copies of
// one source run side by side and all but the first read of it hit L2.
// A pair whose destination another pair also writes or reads is skipped and
// flagged; every CTA sees the same lists, so a pair is skipped as a whole, and
// what is left has no two pairs that touch the same destination.  Bound by memory:
// eight prompts of 4,000 to 16,384 tokens (turbo4, 8 KV heads) forked to three more
// sequences each move 381 MB, the sources read once, in 60 us, 0.95 of the copy
// bandwidth; one prompt of 8,191 (turbo3, 4 KV heads) 2.7 us in a graph.
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
static_assert(kCopyThreads == kCopyTokens, "a thread moves one norm");

// `count` 16-byte pieces, this thread's every kCopyThreads-th, four loads at a time.
__device__ __forceinline__ void copy_pieces(const uint8_t* src, uint8_t* dst, int count, int tid) {
    const uint4* s = reinterpret_cast<const uint4*>(src);
    uint4* d = reinterpret_cast<uint4*>(dst);
    for (int x0 = 0; x0 < count; x0 += 4 * kCopyThreads) {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int x = x0 + e * kCopyThreads + tid;
            if (x < count) v[e] = s[x];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int x = x0 + e * kCopyThreads + tid;
            if (x < count) d[x] = v[e];
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads) tq_copy_kernel(const __grid_constant__ CopyParams p) {
    const int tid = threadIdx.x;
    // (chunk, KV head, pair), the pairs fastest
    const int u = static_cast<int>(blockIdx.x) / p.pairs, m = static_cast<int>(blockIdx.x) - u * p.pairs;
    const int chunk = u / p.hkv, h = u - chunk * p.hkv;
    const int t0 = chunk * kCopyTokens;
    griddep_wait();
    griddep_launch_dependents();
    const int s = p.src[m], d = p.dst[m];
    const bool lead = tid == 0 && t0 == 0 && h == 0;
    bool bad = s < 0 || s >= p.src_batch || d < 0 || d >= p.dst_batch;
    for (int i = tid; i < p.pairs; i += kCopyThreads)
        bad = bad || (i != m && (p.dst[i] == d || (p.same && p.src[i] == d)));
    if (__syncthreads_or(bad)) {
        if (lead) atomicOr(p.status, kStatusBadIndex);
        return;
    }
    const int L = p.src_lengths[s];
    const int n = p.num_tokens != nullptr ? p.num_tokens[m] : L;
    if (n < 0 || n > L) {
        if (lead) atomicOr(p.status, kStatusBadIndex);
        return;
    }
    if (n > p.src_cap || n > p.dst_cap || n > p.max_len) {
        if (lead) atomicOr(p.status, kStatusCapacity);
        return;
    }
    if (!(p.same && s == d) && t0 < n) {
        const int c = min(kCopyTokens, n - t0);
        const size_t rs = (static_cast<size_t>(s) * p.hkv + h) * p.src_cap + t0;
        const size_t rd = (static_cast<size_t>(d) * p.hkv + h) * p.dst_cap + t0;
        copy_pieces(p.k_src + rs * p.rbk, p.k_dst + rd * p.rbk, c * (p.rbk >> 4), tid);
        copy_pieces(p.v_src + rs * p.rbv, p.v_dst + rd * p.rbv, c * (p.rbv >> 4), tid);
        // norms: one each per thread (kCopyTokens == kCopyThreads)
        const bool live = tid < c;
        __half nk = __ushort_as_half(0), nv = __ushort_as_half(0);
        if (live && p.kn_src != nullptr) nk = p.kn_src[rs + tid];
        if (live && p.vn_src != nullptr) nv = p.vn_src[rs + tid];
        if (live && p.kn_src != nullptr) p.kn_dst[rd + tid] = nk;
        if (live && p.vn_src != nullptr) p.vn_dst[rd + tid] = nv;
    }
    if (lead) p.dst_lengths[d] = n;
}

int launch_copy(const CopyParams& p, cudaStream_t stream) {
    const long long ctas = 1ll * p.pairs * p.hkv * ((p.max_len + kCopyTokens - 1) / kCopyTokens);
    if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;   // (the entry point refuses it first)
    return launch_pdl(tq_copy_kernel, dim3(static_cast<unsigned int>(ctas)), dim3(kCopyThreads), 0, stream, p);
}

}  // namespace tq
