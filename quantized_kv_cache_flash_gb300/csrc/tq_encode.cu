// Encode/append: fp16 K/V vectors -> (fp16 norm, packed b-bit codes) written
// at each sequence's current length, then lengths[b] += t_new.
//
// Per vector:
//   n16  = fp16 round-to-nearest-even of the exact L2 norm: fp32 sum of the
//          exact squares, certified against the rounding midpoints; if it is
//          too close to call, the sum of squares is formed exactly as a
//          128-bit integer (every fp16 value is an integer multiple of 2^-24)
//          and the candidate corrected with exact integer comparisons.
//   u    = Rot(x) / n = H (s * x) / (sqrt(128) n), in fp32.
//   code = sign-magnitude index of the nearest codebook entry to u, decided
//          with thresholds that make the fp32 comparison exact against the
//          true midpoints of neighbouring centroids (ties to the lower index).
// Large appends rotate 128 vectors at a time on the tensor cores (one thread
// per vector afterwards); small appends (a decode step's tokens) give each
// vector a warp and rotate with shuffles.
// (The encode of mlxcel pull request #369, Change: seeded sign flip, Walsh-
// Hadamard rotation, nearest codebook entry, bit packing; turboquant_plus
// smem-dequant experiment, Hypothesis 1: a 128-element rotation group with
// one norm per group.)
#include <type_traits>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

struct U128 {
    unsigned long long lo, hi;
};

__device__ __forceinline__ U128 add128(U128 a, U128 b) {
    U128 r;
    r.lo = a.lo + b.lo;
    r.hi = a.hi + b.hi + (r.lo < a.lo ? 1ull : 0ull);
    return r;
}

__device__ __forceinline__ U128 sq_u128(long long m) {
    const unsigned long long a = m < 0 ? static_cast<unsigned long long>(-m)
                                       : static_cast<unsigned long long>(m);
    U128 r;
    r.lo = a * a;
    r.hi = __umul64hi(a, a);
    return r;
}

__device__ __forceinline__ int cmp128(U128 a, U128 b) {
    if (a.hi != b.hi) return a.hi < b.hi ? -1 : 1;
    if (a.lo != b.lo) return a.lo < b.lo ? -1 : 1;
    return 0;
}

// k * k for k < 2^63.
__device__ __forceinline__ U128 square_u64(unsigned long long k) {
    U128 r;
    r.lo = k * k;
    r.hi = __umul64hi(k, k);
    return r;
}

// x (fp16, finite) -> x * 2^24 as an exact integer.
__device__ __forceinline__ long long fp16_scaled_int(float x) {
    return __float2ll_rn(x * 16777216.0f);
}

// fp16 value of a non-negative finite half, and its neighbours on the grid
// (in units of 2^-25 as exact integers).
__device__ __forceinline__ unsigned long long half_units25(unsigned short bits) {
    // value * 2^25; for the overflow neighbour of 65504 use 2^16.
    if (bits >= 0x7C00u) return 65536ull << 25;
    const float f = __half2float(__ushort_as_half(bits));
    return static_cast<unsigned long long>(f * 33554432.0f);
}

// Round sqrt(S * 2^-48) (S exact) to fp16, nearest-even.  S4 = 4*S is the
// square of the target in units of 2^-50, midpoints m (units of 2^-25) compare
// as S4 <=> m^2.
__device__ __forceinline__ unsigned short norm_to_half(U128 S) {
    if (S.hi == 0 && S.lo == 0) return 0;
    U128 S4;
    S4.lo = S.lo << 2;
    S4.hi = (S.hi << 2) | (S.lo >> 62);
    // candidate from an fp32 square root
    const float sf = static_cast<float>(S.hi) * 18446744073709551616.0f + static_cast<float>(S.lo);
    const float n = sqrtf(sf) * (1.0f / 16777216.0f);
    unsigned short hb = __half_as_ushort(__float2half_rn(n));
    if (hb > 0x7C00u) hb = 0x7C00u;
    // walk at most a few steps until the candidate is the correctly rounded value
    for (int step = 0; step < 4; ++step) {
        if (hb < 0x7C00u) {
            // midpoint with the next value up
            const unsigned long long up = (half_units25(hb) + half_units25(hb + 1)) >> 1;
            const int cu = cmp128(S4, square_u64(up));
            if (cu > 0 || (cu == 0 && (hb & 1u))) { ++hb; continue; }
        }
        if (hb > 0) {
            const unsigned short dn_bits = (hb == 0x7C00u) ? 0x7BFFu : static_cast<unsigned short>(hb - 1);
            const unsigned long long lo_mid = (half_units25(dn_bits) + half_units25(hb)) >> 1;
            const int cd = cmp128(S4, square_u64(lo_mid));
            // below the lower midpoint, or on it with the lower value even
            if (cd < 0 || (cd == 0 && !(dn_bits & 1u))) { hb = dn_bits; continue; }
        }
        break;
    }
    return hb;
}


// The same of a vector that a warp holds, lane l dims 4l .. 4l + 3 (the 128-bit
// integer sums of their exact squares are added across the warp).
__device__ __forceinline__ unsigned short norm_exact_warp(float2 f0, float2 f1) {
    U128 S = sq_u128(fp16_scaled_int(f0.x));
    S = add128(S, sq_u128(fp16_scaled_int(f0.y)));
    S = add128(S, sq_u128(fp16_scaled_int(f1.x)));
    S = add128(S, sq_u128(fp16_scaled_int(f1.y)));
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        U128 o;
        o.lo = __shfl_xor_sync(0xffffffffu, S.lo, m);
        o.hi = __shfl_xor_sync(0xffffffffu, S.hi, m);
        S = add128(S, o);
    }
    return norm_to_half(S);
}

__device__ __forceinline__ float half_bits_to_float(unsigned short b) {
    return (b >= 0x7C00u) ? 65536.f : __half2float(__ushort_as_half(b));
}

// The fp16 norm (round to nearest even of the exact sqrt(sum x^2)).  Fast
// path: a fp32 sum S32 of the (exact) squares whose every term goes through
// at most d roundings is within gamma_d = d u / (1 - d u) (u = 2^-24) of the
// exact sum S, relative; so the candidate rounding of sqrt(S32) is certain
// unless S32 lies within a margin above gamma_d of the square of a rounding
// midpoint (midpoints have 12 significant bits, so their squares are exact in
// fp32); then the exact 128-bit integer path decides.  MARGIN_LOG2: the
// margin is S32 * 2^-MARGIN_LOG2 (2^-19 covers d = 18, 2^-20 covers d = 8).
// Candidate fp16 rounding of sqrt(S32) and whether it is certain.
template <int MARGIN_LOG2>
__device__ __forceinline__ unsigned short norm_candidate(float S32, bool& certain) {
    certain = true;
    if (S32 == 0.f) return 0;
    const float n = sqrtf(S32);
    unsigned short hb = __half_as_ushort(__float2half_rn(n));
    if (hb > 0x7C00u) hb = 0x7C00u;
    const float margin = S32 * (1.0f / static_cast<float>(1u << MARGIN_LOG2));
    const float hf = half_bits_to_float(hb);
    if (hb < 0x7C00u) {
        const float up = 0.5f * (hf + half_bits_to_float(hb + 1));
        certain = certain && (S32 < up * up - margin);
    }
    if (hb > 0) {
        const unsigned short db = (hb == 0x7C00u) ? 0x7BFFu : static_cast<unsigned short>(hb - 1);
        const float dn = 0.5f * (half_bits_to_float(db) + ((hb == 0x7C00u) ? 65536.f : hf));
        certain = certain && (S32 > dn * dn + margin);
    }
    return hb;
}


// Sign-magnitude code of the centroid nearest to u: rank = #{tau_k < |u|} for
// u > 0 and #{tau_k <= |u|} for u <= 0, with gt[k] / ge[k] the smallest fp32
// values above / at-or-above the exact midpoint tau_k (ascending).  gt and ge
// differ only when tau_k is itself an fp32 value, so the search runs on gt and
// a negative u sitting exactly on such a tau_k moves one rank up.  Binary
// search: BITS-1 comparisons.
template <int BITS>
__device__ __forceinline__ uint32_t quantize_code(float u, const float* gt, const float* ge,
                                                  bool any_tie) {
    constexpr int H = 1 << (BITS - 1);
    const float a = fabsf(u);
    const bool neg = !(u > 0.f);
    uint32_t rank;
    if constexpr (BITS == 3) {
        const bool b1 = a >= gt[1];
        const bool b0 = a >= (b1 ? gt[2] : gt[0]);
        rank = (b1 ? 2u : 0u) | (b0 ? 1u : 0u);
    } else {
        const bool b2 = a >= gt[3];
        const bool b1 = a >= (b2 ? gt[5] : gt[1]);
        const float t0 = b2 ? (b1 ? gt[6] : gt[4]) : (b1 ? gt[2] : gt[0]);
        const bool b0 = a >= t0;
        rank = (b2 ? 4u : 0u) | (b1 ? 2u : 0u) | (b0 ? 1u : 0u);
    }
    if (any_tie && neg && rank < H - 1) {
        // a in [ge[rank], gt[rank]) means a == tau_rank: the tie goes down (more negative)
        if (a >= ge[rank] && a < gt[rank]) rank += 1;
    }
    return (neg ? static_cast<uint32_t>(H) : 0u) | rank;
}


// The record's norm (norm format) or, for table records (tcb != nullptr), the
// eight fp16 values c_j * n16 after the 48 code bytes: c_j (fp32) times n16
// (fp16) is exact in double, so each value is one rounding of the exact
// product.
__device__ __forceinline__ void store_norm(__half* dst_norm, uint8_t* dst, const float* tcb,
                                           unsigned short nb) {
    if (tcb == nullptr) {
        dst_norm[0] = __ushort_as_half(nb);
        return;
    }
    const double n = static_cast<double>(__half2float(__ushort_as_half(nb)));
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t a = __half_as_ushort(__double2half(static_cast<double>(tcb[2 * k]) * n));
        const uint32_t b = __half_as_ushort(__double2half(static_cast<double>(tcb[2 * k + 1]) * n));
        w[k] = a | (b << 16);
    }
    *reinterpret_cast<uint4*>(dst + 48) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Packed appends: where row `tok` of the packed [total, Hkv, 128] inputs goes.
// Sequence b owns rows cu[b] .. cu[b + 1] - 1; rows behind the last sequence,
// rows of a sequence whose bounds are out of order or past the end, and rows
// of a sequence that would pass its capacity go nowhere.
struct PackedSlot {
    int b, pos;       // sequence, token position in it
    bool live;        // the row is written
    bool first_over;  // the first row of a sequence that would pass the capacity
};

__device__ __forceinline__ bool packed_seq_ok(int first, int next, int total) {
    return first >= 0 && next >= first && next <= total;
}

__device__ __forceinline__ PackedSlot packed_slot(const EncodeParams& p, int tok) {
    // the last b with cu[b] <= tok (cu has a few KB and stays in L1)
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid] <= tok) lo = mid;
        else hi = mid;
    }
    PackedSlot s;
    s.b = lo;
    const int first = p.cu[lo], next = p.cu[lo + 1], L = p.lengths[lo];
    const bool mine = packed_seq_ok(first, next, p.total) && tok >= first && tok < next;
    const bool fits = L >= 0 && L <= p.cap - (next - first);
    s.live = mine && fits;
    s.first_over = mine && !fits && tok == first;
    s.pos = s.live ? L + (tok - first) : 0;
    return s;
}

// Tokens that a packed append adds to sequence b of length L (0 where it is
// left untouched).
__device__ __forceinline__ int packed_added(const EncodeParams& p, int b, int L) {
    const int first = p.cu[b], next = p.cu[b + 1];
    if (!packed_seq_ok(first, next, p.total)) {
        atomicOr(p.status, kStatusBadIndex);
        return 0;
    }
    return L >= 0 && L <= p.cap - (next - first) ? next - first : 0;
}

// Packed appends decide every code from exact sums.  The rotated values and the
// thresholds carry rounding errors; a vector with a value within their bound, k_near or
// v_near times its norm n, of a threshold or 0 is encoded once more from its exact
// transform: the sums of +-x are integers in units of 2^-24, below 2^47, and the midpoints
// are taken in double.  So the codes do not depend on which kernel or how many tokens took
// the vector.  build_tables derives the bounds; a vector without very small entries (four
// Gaussian ones of five) gets along with less than half of the general one, and 4 in 1000
// Gaussian vectors are encoded twice with 3 bits, 9 with 4 (29,800 tokens of 8 KV heads, 4
// bits: 87 us, 95 with the general bound for all).  The distances from every threshold
// make the rest of the cost: of 20,480 tokens of 8 KV heads 41.6 us with 3 bits and 60.0
// with 4, where tq_encode_append without them takes 30.3 and 41.6.  The kernel is then
// bound by the ALU pipe (0.69 of its cycles: minima, logic, shifts; issue 0.67).

// Advance lengths[] after the last CTA of the launch has read it: one ticket
// per CTA, taken once every thread of the CTA has read lengths[] for the last
// time (so none sees an advanced length) and, for large appends, its
// producer has stopped taking tiles; the counters are back at zero for the
// next launch.
template <bool PACKED>
__device__ __forceinline__ void finish_append(const EncodeParams& p, int lane) {
    __shared__ unsigned int s_ticket;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        s_ticket = atomicAdd(p.counter, 1u);
    }
    __syncthreads();
    if (s_ticket == gridDim.x - 1 && threadIdx.x < 32) {
        __threadfence();
        for (int bb = lane; bb < p.batch; bb += 32) {
            const int Lb = *((volatile int32_t*)p.lengths + bb);
            if constexpr (PACKED) {
                p.lengths[bb] = Lb + packed_added(p, bb, Lb);
            } else {
                if (Lb >= 0 && Lb + p.t_new <= p.cap) p.lengths[bb] = Lb + p.t_new;
            }
        }
        if (lane == 0) {
            *((volatile uint32_t*)p.counter) = 0u;
            if (p.tiles_next != nullptr) *((volatile uint32_t*)p.tiles_next) = 0u;
        }
        __threadfence();
    }
}

// finish_append for the warp-per-vector kernel: lane bb of warp 0 brings
// lengths[bb] (bb < 32) read at the kernel's start -- only this launch's last
// CTA writes lengths[], after every CTA has taken its ticket -- and the ticket
// needs no fence before it: every read of lengths[] has been consumed (the
// stores' addresses) when the CTA's threads meet at the barrier.
template <bool PACKED>
__device__ __forceinline__ void finish_append_small(const EncodeParams& p, int lane, int len_pre) {
    __shared__ unsigned int s_ticket;
    if constexpr (!PACKED) __syncthreads();   // (packed: the caller's barrier)
    if (threadIdx.x == 0) s_ticket = atomicAdd(p.counter, 1u);
    __syncthreads();
    if (s_ticket == gridDim.x - 1 && threadIdx.x < 32) {
        for (int bb = lane; bb < p.batch; bb += 32) {
            const int Lb = bb < 32 ? len_pre : *((volatile int32_t*)p.lengths + bb);
            if constexpr (PACKED) {
                p.lengths[bb] = Lb + packed_added(p, bb, Lb);
            } else {
                if (Lb >= 0 && Lb + p.t_new <= p.cap) p.lengths[bb] = Lb + p.t_new;
            }
        }
        if (lane == 0) {
            *((volatile uint32_t*)p.counter) = 0u;
            if (p.tiles_next != nullptr) *((volatile uint32_t*)p.tiles_next) = 0u;
        }
        __threadfence();
    }
}

// The record of a vector whose codes the warp holds, lane l those of dims
// 4l .. 4l + 3.
template <int BITS>
__device__ __forceinline__ void store_codes_warp(const uint32_t (&code)[4], uint8_t* dst, int lane) {
    if constexpr (BITS == 4) {
        // word k = dims 8k..8k+7 (lanes 2k, 2k+1): rank of dim 8k+j in bits
        // 4j..4j+2; sign of dim 8k+j (j < 4) in bit 8j+7, of dim 8k+4+j in bit 8j+3
        const bool upper = (lane & 1) != 0;
        uint32_t part = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            part |= (code[i] & 7u) << (4 * i + (upper ? 16 : 0));
            part |= (code[i] >> 3) << (8 * i + (upper ? 3 : 7));
        }
        const uint32_t other = __shfl_down_sync(0xffffffffu, part, 1);
        if (!upper) reinterpret_cast<uint32_t*>(dst)[lane >> 1] = part | other;
    } else {
        // quarter q = lanes 8q..8q+7; lanes 8q+2k, 8q+2k+1 carry dims 32q+8k..+7
        // (word k's nibbles); lanes 8q+6, 8q+7 carry dims 32q+24..31, whose
        // code bit k goes to bit 4j+3 of word k.
        const uint32_t nib = (code[0] & 7u) | ((code[1] & 7u) << 4) | ((code[2] & 7u) << 8) |
                             ((code[3] & 7u) << 12);
        uint32_t sp[3];
#pragma unroll
        for (int k = 0; k < 3; ++k)
            sp[k] = (((code[0] >> k) & 1u) << 3) | (((code[1] >> k) & 1u) << 7) |
                    (((code[2] >> k) & 1u) << 11) | (((code[3] >> k) & 1u) << 15);
        const int qb = lane & ~7;
        const uint32_t up = __shfl_down_sync(0xffffffffu, nib, 1);
        uint32_t spw[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const uint32_t s6 = __shfl_sync(0xffffffffu, sp[k], qb + 6);
            const uint32_t s7 = __shfl_sync(0xffffffffu, sp[k], qb + 7);
            spw[k] = s6 | (s7 << 16);
        }
        const int sub = lane & 7;
        if (sub < 6 && (sub & 1) == 0) {
            const int k = sub >> 1;
            const uint32_t word = nib | (up << 16) | (k == 0 ? spw[0] : (k == 1 ? spw[1] : spw[2]));
            reinterpret_cast<uint32_t*>(dst)[(lane >> 3) * 3 + k] = word;
        }
    }
}

// The codes of one vector from its exact transform (the warp's lane l holds
// dims 4l .. 4l + 3 of x): Y = H (s * x) in integer units of 2^-24, compared
// with the midpoints of the codebook (mag: its positive half) times sqrt(128) n.
// Those are formed in double, a midpoint per lane -- double arithmetic is slow
// here -- and compared as integers: Y > t is Y > floor(t), Y >= t is Y >= ceil(t).
// Ties go to the lower index.
template <int BITS>
__device__ __noinline__ void encode_exact_warp(const uint2 raw, uint8_t* dst, const uint32_t (&signs)[4],
                                               const float* mag, int lane) {
    constexpr int H = 1 << (BITS - 1);
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
    const float x[4] = {f0.x, f0.y, f1.x, f1.y};
    double ss = 0.0;   // (the square of an fp16 value is exact in double)
    long long y[4];
    const uint32_t sn = sign_nibble(signs, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ss += static_cast<double>(x[i]) * static_cast<double>(x[i]);
        const long long v = fp16_scaled_int(x[i]);
        y[i] = ((sn >> i) & 1u) ? -v : v;
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const long long a0 = y[0] + y[1], a1 = y[0] - y[1], a2 = y[2] + y[3], a3 = y[2] - y[3];
    y[0] = a0 + a2;
    y[2] = a0 - a2;
    y[1] = a1 + a3;
    y[3] = a1 - a3;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long o = __shfl_xor_sync(0xffffffffu, y[i], m);
            y[i] = (lane & m) ? (o - y[i]) : (y[i] + o);
        }
    }
    const int k = lane < H - 1 ? lane : 0;   // this lane's midpoint, in units of 2^-24
    const double t = 0.5 * (static_cast<double>(mag[k]) + static_cast<double>(mag[k + 1])) *
                     (sqrt(128.0 * ss) * 16777216.0);
    const long long below = __double2ll_rd(t), above = __double2ll_ru(t);
    long long a[4];
    bool neg[4];
    uint32_t rank[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        neg[i] = !(y[i] > 0);
        a[i] = neg[i] ? -y[i] : y[i];
    }
#pragma unroll
    for (int j = 0; j < H - 1; ++j) {
        const long long lo = __shfl_sync(0xffffffffu, below, j), hi = __shfl_sync(0xffffffffu, above, j);
#pragma unroll
        for (int i = 0; i < 4; ++i) rank[i] += (neg[i] ? (a[i] >= hi && a[i] > 0) : a[i] > lo) ? 1u : 0u;
    }
    uint32_t code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) code[i] = (neg[i] ? static_cast<uint32_t>(H) : 0u) | rank[i];
    store_codes_warp<BITS>(code, dst, lane);
}

// Packed appends whose bounds decrease somewhere: sequences may then share rows, and
// packed_slot names one of them a row.  The rows that belong to another sequence as well
// are encoded for it here (a warp a vector, warp w of nw), so that every sequence whose
// own bounds are in order holds all its records.
template <int KB, int VB>
__device__ __noinline__ void append_shared_rows(const EncodeParams& p, long long w, long long nw, int lane) {
    for (int b = 0; b < p.batch; ++b) {
        const int first = p.cu[b], n = p.cu[b + 1] - first, L = p.lengths[b];
        if (!packed_seq_ok(first, p.cu[b + 1], p.total) || n == 0) continue;
        if (L < 0 || L > p.cap - n) {
            if (w == 0 && lane == 0) atomicOr(p.status, kStatusCapacity);
            continue;
        }
        for (long long i = w; i < 2ll * n * p.hkv; i += nw) {
            const int j = static_cast<int>((i >> 1) / p.hkv), h = static_cast<int>((i >> 1) - 1ll * j * p.hkv);
            if (packed_slot(p, first + j).b == b) continue;   // has it
            const bool is_v = (i & 1) != 0;
            const __half* x = (is_v ? p.v_new : p.k_new) + (static_cast<size_t>(first + j) * p.hkv + h) * kD;
            const uint2 raw = reinterpret_cast<const uint2*>(x)[lane];
            const size_t pos = (static_cast<size_t>(b) * p.hkv + h) * p.cap + L + j;
            if (!is_v && KB == 0) {
                reinterpret_cast<uint2*>(p.k_codes + pos * 256)[lane] = raw;
                continue;
            }
            const int bits = is_v ? VB : KB;
            uint8_t* const dst = (is_v ? p.v_codes : p.k_codes) + pos * (p.table ? 64 : bits * 16);
            const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
            const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
            const unsigned short nb = norm_exact_warp(f0, f1);
            if (lane == 0) {
                store_norm((is_v ? p.v_norm : p.k_norm) + pos, dst, p.table ? (is_v ? p.v_cb : p.k_cb) : nullptr, nb);
                if (nb >= 0x7C00u) atomicOr(p.status, kStatusNormOverflow);
            }
            if (is_v) encode_exact_warp<VB>(raw, dst, p.signs, p.v_mag, lane);
            else encode_exact_warp<(KB == 0 ? VB : KB)>(raw, dst, p.signs, p.k_mag, lane);
        }
    }
}

// ---------------------------------------------------------------------------
// Large appends on the 5th-generation tensor cores.
//
// A tile is 128 vectors of one stream (K or V).  Its rotation is one product
// Y[128 x 128] = X[128 x 128] . B^T with B[n][k] = H[n][k] s_k: the entries
// are +-1, so every product x_k B[n][k] is exact and only the fp32 sums round
// (as in a butterfly transform, in another order).  It runs as 8 tcgen05 MMAs
// of K = 16 into tensor memory; row i of Y (tensor-memory lane i) is vector
// i's H (s * x), read back by one thread, which forms the vector's exact fp16
// norm from the tile in shared memory and encodes all 128 dims against the
// thresholds scaled by sqrt(128) n.  X tiles arrive by TMA in the MMA's
// K-major 128-byte-swizzled layout (rows past the end are zero-filled).
// Persistent CTAs, two per SM, each with B resident in shared memory and two
// groups of encode warps, each group with its own X stage and tensor-memory
// accumulator: one group's copy and MMA run while the other encodes.
// ---------------------------------------------------------------------------
constexpr int kTcVecs = 128;                      // vectors per tile = tensor-memory lanes
constexpr int kTcBOff = 0;                        // B: 128 x 128 fp16 (32 KB)
constexpr int kTcXOff = 32768;                    // X stages: 2 x 32 KB
constexpr int kTcBarOff = kTcXOff + 2 * 32768;    // full[2], done[2], xfree[2], afree[2] mbarriers, TMEM slot
constexpr int kTcSmem = kTcBarOff + 128;
constexpr int kTcSmemAlloc = kTcSmem + 1024;      // base alignment slack
constexpr int kTcCtasPerSm = 2;
constexpr uint32_t kTcIdesc = umma_idesc_f16_f32(128, 128);

__device__ __forceinline__ uint32_t fbits(float f) { return __float_as_uint(f); }

// x * x + acc for an fp16 x, one rounding (the square of an fp16 value is
// exact in fp32, so this is fmaf(x, x, acc) on the converted value).
__device__ __forceinline__ float fma_sq_f16(unsigned short x, float acc) {
    float r;
    asm("fma.rn.f32.f16 %0, %1, %1, %2;" : "=f"(r) : "h"(x), "f"(acc));
    return r;
}

// Codes of the 32 dims of quarter q of a record from their rotated values
// y = H (s * x) (unnormalised) and the thresholds T_k = gt_k sqrt(128) n, so
// that |y| > T_k <=> |u| > tau_k for u = y / (sqrt(128) n).  Every decision is
// a sign bit: c_k = sign(T_k - |y|) = [|y| > T_k] (the sign of a difference
// is exact), the rank bits are XORs of the c_k (the rank counts the
// thresholds below |y|), and p = sign(0 - y) = [y > 0] (a zero y is negative:
// its tie goes to the lower index).  The bits are shifted into the words most
// significant first (funnel shifts), the sign positions inverted at the end.
//   3-bit: code = sign << 2 | rank; word k (k < 3): bits 4j..4j+2 = code of
//          dim 8k+j, bit 4j+3 = bit k of the code of dim 24+j.
//   4-bit: word k = dims 8k..8k+7: rank of dim 8k+j in bits 4j..4j+2, the
//          sign of dim 8k+j (j < 4) in bit 8j+7, of dim 8k+4+j in bit 8j+3.
//   NEAR: the smallest of near becomes at most that of all |y|'s distances from a
//   T_k or 0.
__device__ __forceinline__ float min3(float a, float b, float c) {
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Word of 8 dims of a 4-bit record (see pack_quarter).
template <bool NEAR>
__device__ __forceinline__ uint32_t pack_word4(const uint32_t* r, const float (&T)[7], float (&near)[4]) {
    auto shin = [](uint32_t acc, uint32_t v) { return __funnelshift_l(v, acc, 1); };
    uint32_t b0[8], b1[8], b2[8], p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float y = __uint_as_float(r[j]);
        const float a = fabsf(y);
        uint32_t d[7];
#pragma unroll
        for (int t = 0; t < 7; ++t) d[t] = fbits(T[t] - a);
        if constexpr (NEAR) {
            // (four chains over the elements, 3-input minima)
            auto ab = [&](int t) { return fabsf(__uint_as_float(d[t])); };
            near[j & 3] = min3(near[j & 3], min3(a, ab(0), ab(1)),
                               min3(min3(ab(2), ab(3), ab(4)), ab(5), ab(6)));
        }
        const uint32_t x135 = d[1] ^ d[3] ^ d[5];
        b2[j] = d[3];
        b1[j] = x135;
        b0[j] = x135 ^ d[0] ^ d[2] ^ d[4] ^ d[6];
        p[j] = fbits(__fsub_rn(0.f, y));
    }
    uint32_t acc = 0;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
        const int s = (j & 1) ? (j - 1) / 2 : 4 + j / 2;   // whose sign sits in bit 4j+3
        acc = shin(shin(shin(shin(acc, p[s]), b2[j]), b1[j]), b0[j]);
    }
    return acc ^ 0x88888888u;
}

template <int BITS, bool NEAR>
__device__ __forceinline__ void pack_quarter(const uint32_t (&r)[32],
                                             const float (&T)[(1 << (BITS - 1)) - 1], uint32_t* w,
                                             float (&near)[4]) {
    auto shin = [](uint32_t acc, uint32_t v) { return __funnelshift_l(v, acc, 1); };  // acc << 1 | v >> 31
    if constexpr (BITS == 3) {
        struct Bits {
            uint32_t b0, b1, p;
        };
        auto bits_of = [&](int i) {
            const float y = __uint_as_float(r[i]);
            const float a = fabsf(y);
            const float d0 = T[0] - a, d1 = T[1] - a, d2 = T[2] - a;
            if constexpr (NEAR)
                near[i & 3] = min3(near[i & 3], a, min3(fabsf(d0), fabsf(d1), fabsf(d2)));
            Bits o;
            o.b1 = fbits(d1);
            o.b0 = fbits(d0) ^ fbits(d1) ^ fbits(d2);
            o.p = fbits(__fsub_rn(0.f, y));
            return o;
        };
        uint32_t a0 = 0, a1 = 0, a2 = 0;
#pragma unroll
        for (int j = 7; j >= 0; --j) {
            const Bits e = bits_of(24 + j);
            a0 = shin(a0, e.b0);
            a1 = shin(a1, e.b1);
            a2 = shin(a2, e.p);
            const Bits x0 = bits_of(j), x1 = bits_of(8 + j), x2 = bits_of(16 + j);
            a0 = shin(shin(shin(a0, x0.p), x0.b1), x0.b0);
            a1 = shin(shin(shin(a1, x1.p), x1.b1), x1.b0);
            a2 = shin(shin(shin(a2, x2.p), x2.b1), x2.b0);
        }
        w[0] = a0 ^ 0x44444444u;
        w[1] = a1 ^ 0x44444444u;
        w[2] = a2 ^ 0xCCCCCCCCu;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = pack_word4<NEAR>(r + 8 * k, T, near);
    }
}

// Exact fp16 norm of row `row` of an X tile (the rare path of the norm): the
// warp's lane l takes dims 4l..4l+3 and the 128-bit integer sums of their
// exact squares are added across the warp.
__device__ __noinline__ unsigned short norm_exact_row(const uint8_t* xs, int row, int lane) {
    const int c = lane >> 1;  // 16-byte chunk of dims 8c..8c+7
    const uint8_t* src = xs + (c >> 3) * 16384 + row * 128 + ((((c & 7) ^ (row & 7))) << 4) + (lane & 1) * 8;
    const uint2 raw = *reinterpret_cast<const uint2*>(src);
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
    return norm_exact_warp(f0, f1);
}

// B[n][k] = H[n][k] s_k as fp16 +-1 in the K-major swizzled layout; thread
// i (< 256) writes half h = i >> 7 (dims 64h .. 64h+63) of row n = i & 127.
__device__ __forceinline__ void build_rotation_b(uint8_t* sB, const uint32_t (&signs)[4], int i) {
    const int n = i & 127, h0 = 8 * (i >> 7);
#pragma unroll 4
    for (int c = h0; c < h0 + 8; ++c) {
        uint32_t hw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t v = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = 8 * c + 2 * e + h;
                const uint32_t neg = (__popc(n & k) ^ (signs[k >> 5] >> (k & 31))) & 1u;
                v |= (0x3C00u | (neg << 15)) << (16 * h);
            }
            hw[e] = v;
        }
        *reinterpret_cast<uint4*>(sB + sw128_offset(n, 8 * c)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    }
}

// Warp roles: warps 0-7 encode in two groups of four (group g works through
// X stage g and accumulator g; warp w reads tensor-memory lanes 32 (w & 3) ..
// +31, one vector per thread), warp 8 hands out the tiles and issues the
// copies and MMAs.  Tiles ([K tiles (quantized K only) | V tiles], 128
// vectors each) are taken from one counter for the whole grid, a group's next
// tile when it has released its stage, so groups on less loaded SMs take
// more.  Hand-offs by mbarrier, per stage s: full[s] (copy landed, or the
// end: tile id -1), done[s] (MMA committed), xfree[s] (the group has read X
// stage s and seen its MMA complete), afree[s] (the group has read
// accumulator s).  KB = 0 copies the fp16 K rows instead (plain coalesced
// copies spread over the grid).
constexpr int kTcEncWarps = 8;
constexpr int kTcThreads = 32 * (kTcEncWarps + 1);

template <int KB, int VB, bool PACKED>
__global__ void __launch_bounds__(kTcThreads, kTcCtasPerSm)
    tq_encode_tc_kernel(const __grid_constant__ EncodeParams p, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) uint8_t esm_raw[];
    uint8_t* smem = esm_raw + ((1024u - (smem_u32(esm_raw) & 1023u)) & 1023u);
    __shared__ int s_tile[2];   // tile in stage s (-1: no more)
    const int tid = threadIdx.x;
    const int lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int nvec = PACKED ? p.total * p.hkv : p.batch * p.hkv * p.t_new;   // below 2^31 (the host checks)
    // a packed append's tile is 128 tokens of one KV head (rows then write
    // neighbouring records; with the vectors taken in the order of the input, a
    // token's heads next to each other, the scattered stores took twice as long),
    // the heads of a token block one after the other
    const int tiles_s = PACKED ? (p.total + kTcVecs - 1) / kTcVecs * p.hkv : (nvec + kTcVecs - 1) / kTcVecs;
    const int tiles_k = (KB == 0) ? 0 : tiles_s;
    const int tiles = tiles_k + tiles_s;
    const uint32_t bar_full = smem_u32(smem + kTcBarOff);   // + 8 s
    const uint32_t bar_done = bar_full + 16;                 // + 8 s
    const uint32_t bar_xfree = bar_full + 32;                // + 8 s
    const uint32_t bar_afree = bar_full + 48;                // + 8 s
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + kTcBarOff + 64);
    uint8_t* sB = smem + kTcBOff;

    // the producer lane: stage s takes tile t (first tiles: blockIdx.x and
    // blockIdx.x + gridDim.x; then from the counter, which counts from
    // 2 gridDim.x) or, past the last tile, the end marker; false at the end
    auto take_tile = [&](int s, bool first) -> bool {
        const int t = first ? static_cast<int>(blockIdx.x) + s * static_cast<int>(gridDim.x)
                            : static_cast<int>(atomicAdd(p.tiles_next, 1u)) + 2 * static_cast<int>(gridDim.x);
        const uint32_t bar = bar_full + 8 * s;
        if (t >= tiles) {
            s_tile[s] = -1;
            mbar_arrive(bar);
            return false;
        }
        s_tile[s] = t;
        const bool is_v = t >= tiles_k;
        const int ts = is_v ? t - tiles_k : t;
        const uint32_t dst = smem_u32(smem + kTcXOff + s * 32768);
        mbar_arrive_expect_tx(bar, 32768);
        if constexpr (PACKED) {
            const int blk = static_cast<int>((static_cast<uint64_t>(ts) * p.div_h_m) >> p.div_h_s);
            tma_g2s_3d(dst, is_v ? &vmap : &kmap, 0, ts - blk * p.hkv, blk * kTcVecs, bar);
            tma_g2s_3d(dst + 16384, is_v ? &vmap : &kmap, 64, ts - blk * p.hkv, blk * kTcVecs, bar);
        } else {
            tma_g2s_2d(dst, is_v ? &vmap : &kmap, 0, ts * kTcVecs, bar);
            tma_g2s_2d(dst + 16384, is_v ? &vmap : &kmap, 64, ts * kTcVecs, bar);
        }
        return true;
    };
    const bool producer = tid == 32 * kTcEncWarps;
    int k_tma[2] = {0, 0};     // tiles (and end markers) put into each stage (the producer lane)
    bool live[2] = {false, false};

    // prologue (nothing here reads what earlier work on the stream writes):
    // it may overlap the tail of the previous kernel
    griddep_launch_dependents();
    if (producer) {
        for (int i = 0; i < 4; ++i) mbar_init(bar_full + 8 * i, 1);
        for (int i = 0; i < 4; ++i) mbar_init(bar_xfree + 8 * i, kTcEncWarps / 2);
        fence_barrier_init();
        griddep_wait();   // inputs, lengths and the tile counter come from earlier work on the stream
        for (int s = 0; s < 2; ++s) {   // the first copies fly while B is built
            live[s] = take_tile(s, true);
            k_tma[s] = 1;
        }
    }
    if (warp == kTcEncWarps) tmem_alloc(smem_u32(tslot), 256);
    if (tid < 256) build_rotation_b(sB, p.signs, tid);
    fence_proxy_async();   // B's generic stores, seen by the tensor core
    griddep_wait();
    [[maybe_unused]] bool down = false;   // packed: whether the bounds decrease somewhere
    if constexpr (PACKED)
        for (int bb = tid; bb < p.batch; bb += kTcThreads) down = down || p.cu[bb] > p.cu[bb + 1];
    tc_fence_before();
    if constexpr (PACKED) down = __syncthreads_or(down) != 0;
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    if (warp == kTcEncWarps) {
        // ---- producer: for each stage, the MMA of its tile once the copy has
        // landed and the group has read the accumulator, then the stage's next
        // tile once the group has released the stage ----
        if (producer) {
            bool stalled = false;
            int k_mma[2] = {0, 0};
            uint64_t t_last = global_timer_ns();
            for (uint32_t spin = 0; live[0] || live[1]; ++spin) {
                bool progress = false;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (!live[s]) continue;
                    const int k = k_mma[s];
                    if (k < k_tma[s] && mbar_test_wait(bar_full + 8 * s, k & 1) &&
                        (k == 0 || mbar_test_wait(bar_afree + 8 * s, (k - 1) & 1))) {
                        tc_fence_after();
                        const uint32_t xa = smem_u32(smem + kTcXOff + s * 32768);
                        const uint32_t ba = smem_u32(sB);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint32_t koff = (kk >> 2) * 16384 + (kk & 3) * 32;
                            umma_f16(tmem + 128 * s, umma_desc_sw128(xa + koff), umma_desc_sw128(ba + koff),
                                     kTcIdesc, kk > 0 ? 1u : 0u);
                        }
                        umma_commit(bar_done + 8 * s);
                        k_mma[s] = k + 1;
                        progress = true;
                    }
                    if (k_mma[s] == k_tma[s] && mbar_test_wait(bar_xfree + 8 * s, (k_tma[s] - 1) & 1)) {
                        live[s] = take_tile(s, false);
                        ++k_tma[s];
                        progress = true;
                    }
                }
                if (progress) {
                    t_last = global_timer_ns();
                } else {
                    __nanosleep(32);
                    if ((spin & 63u) == 0 && global_timer_ns() - t_last > 2000000000ull) {
                        stalled = true;
                        break;
                    }
                }
            }
            if (stalled) {
                atomicOr(p.status, kStatusPipelineStall);
                // let the copies and MMAs still in flight land before the shared
                // memory and tensor memory go away
                for (int s = 0; s < 2; ++s) {
                    if (live[s] && k_mma[s] < k_tma[s])
                        (void)mbar_wait_bounded(bar_full + 8 * s, (k_tma[s] - 1) & 1);
                    if (k_mma[s] > 0) (void)mbar_wait_bounded(bar_done + 8 * s, (k_mma[s] - 1) & 1);
                }
            }
        }
    } else {
        // ---- encode warps ----
        const int g = warp >> 2, lq = warp & 3;
        const int r = 32 * lq + lane;   // the vector (row) of each tile
        if constexpr (KB == 0) {   // fp16 K rows: copied, 16 bytes per thread
            const long long n16 = static_cast<long long>(nvec) * 16;
            for (long long i = static_cast<long long>(blockIdx.x) * (32 * kTcEncWarps) + tid; i < n16;
                 i += static_cast<long long>(gridDim.x) * (32 * kTcEncWarps)) {
                const int v = static_cast<int>(i >> 4);
                if constexpr (PACKED) {
                    const int tok = static_cast<int>((static_cast<uint64_t>(v) * p.div_h_m) >> p.div_h_s);
                    const PackedSlot ps = packed_slot(p, tok);
                    if (!ps.live) continue;   // (the V rows raise the status)
                    const size_t pos = (static_cast<size_t>(ps.b) * p.hkv + (v - tok * p.hkv)) * p.cap + ps.pos;
                    reinterpret_cast<uint4*>(p.k_codes + pos * 256)[i & 15] = reinterpret_cast<const uint4*>(p.k_new)[i];
                    continue;
                }
                const int bh = static_cast<int>((static_cast<uint64_t>(v) * p.div_t_m) >> p.div_t_s);
                const int t = v - bh * p.t_new;
                const int b = static_cast<int>((static_cast<uint64_t>(bh) * p.div_h_m) >> p.div_h_s);
                const int L = p.lengths[b];
                if (L < 0 || L + p.t_new > p.cap) {
                    if ((i & 15) == 0 && t == 0 && bh == b * p.hkv) atomicOr(p.status, kStatusCapacity);
                    continue;
                }
                const size_t pos = static_cast<size_t>(bh) * p.cap + L + t;
                reinterpret_cast<uint4*>(p.k_codes + pos * 256)[i & 15] = reinterpret_cast<const uint4*>(p.k_new)[i];
            }
        }
        const uint8_t* xs = smem + kTcXOff + g * 32768;
        const uint32_t tacc = tmem + 128 * g + (static_cast<uint32_t>(lq * 32) << 16);
        bool stalled = false;
        for (int k = 0;; ++k) {
            const uint32_t ph = k & 1;
            if (!mbar_wait_bounded(bar_full + 8 * g, ph)) stalled = true;
            if (__any_sync(0xffffffffu, stalled)) break;
            const int t = s_tile[g];
            if (t < 0) break;
            const bool is_v = t >= tiles_k;
            int v = (is_v ? t - tiles_k : t) * kTcVecs + r;
            // where this thread's vector goes: lengths[] is read now and
            // looked at only after the norm
            bool in_range = v < nvec;
            int bh = 0, tt = 0, b = 0, L = 0;
            PackedSlot ps{};
            if constexpr (PACKED) {
                const int ts = is_v ? t - tiles_k : t;
                const int blk = static_cast<int>((static_cast<uint64_t>(ts) * p.div_h_m) >> p.div_h_s);
                const int tok = blk * kTcVecs + r;
                tt = ts - blk * p.hkv;   // the KV head
                in_range = tok < p.total;
                ps = packed_slot(p, in_range ? tok : 0);
                v = tok * p.hkv + tt;
            } else {
                bh = static_cast<int>((static_cast<uint64_t>(in_range ? v : 0) * p.div_t_m) >> p.div_t_s);
                tt = (in_range ? v : 0) - bh * p.t_new;
                b = static_cast<int>((static_cast<uint64_t>(bh) * p.div_h_m) >> p.div_h_s);
                L = p.lengths[b];
            }
            // norm: the exact squares of the fp16 inputs summed in fp32 by 8
            // accumulators of 16 terms each, then pairwise: each square goes
            // through at most 15 + 3 = 18 roundings; certified or redone exactly
            float S32;
            [[maybe_unused]] float least = 0.f;   // (packed) the smallest |x|
            {
                float acc[8];
                [[maybe_unused]] __half2 lo2[2] = {__float2half2_rn(65504.f), __float2half2_rn(65504.f)};
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const uint4 w = *reinterpret_cast<const uint4*>(xs + (c >> 3) * 16384 + r * 128 +
                                                                    ((((c & 7) ^ (r & 7))) << 4));
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float& a = acc[4 * (c & 1) + e];
                        a = fma_sq_f16(static_cast<unsigned short>(ww[e]), a);
                        a = fma_sq_f16(static_cast<unsigned short>(ww[e] >> 16), a);
                        if constexpr (PACKED)
                            lo2[e & 1] = __hmin2(lo2[e & 1], __habs2(*reinterpret_cast<const __half2*>(&ww[e])));
                    }
                }
                if constexpr (PACKED) {
                    lo2[0] = __hmin2(lo2[0], lo2[1]);
                    least = fminf(__low2float(lo2[0]), __high2float(lo2[0]));
                }
                S32 = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
            }
            bool ok;
            unsigned short nb = norm_candidate<19>(S32, ok);
            // (rows without a vector are zero and always certain)
            unsigned need = __ballot_sync(0xffffffffu, !ok);
            while (need) {
                const int src = __ffs(need) - 1;
                need &= need - 1;
                const unsigned short e = norm_exact_row(xs, 32 * lq + src, lane);
                if (lane == src) nb = e;
            }

            bool valid = in_range;
            size_t pos = 0;
            if constexpr (PACKED) {
                if (in_range && is_v && tt == 0 && ps.first_over) atomicOr(p.status, kStatusCapacity);
                valid = in_range && ps.live;
                pos = (static_cast<size_t>(ps.b) * p.hkv + tt) * p.cap + ps.pos;
            } else if (valid) {
                if (L < 0 || L + p.t_new > p.cap) {
                    if (!is_v && tt == 0 && bh == b * p.hkv) atomicOr(p.status, kStatusCapacity);
                    valid = false;
                } else {
                    pos = static_cast<size_t>(bh) * p.cap + L + tt;
                }
            }
            uint8_t* const codes = is_v ? p.v_codes : p.k_codes;
            __half* const norms = is_v ? p.v_norm : p.k_norm;
            const float* const tcb = p.table ? (is_v ? p.v_cb : p.k_cb) : nullptr;
            const int bits = is_v ? VB : KB;
            uint8_t* const dst = codes + pos * (p.table ? 64 : bits * 16);
            if (valid) {
                store_norm(norms + pos, dst, tcb, nb);
                if (nb >= 0x7C00u) atomicOr(p.status, kStatusNormOverflow);
            }

            if (!mbar_wait_bounded(bar_done + 8 * g, ph)) stalled = true;
            if (__any_sync(0xffffffffu, stalled)) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_xfree + 8 * g);   // X read here and by the MMA
            tc_fence_after();
            const float scale = sqrtf(S32) * 11.313708498984761f;   // sqrt(128) n
            float near4[4] = {INFINITY, INFINITY, INFINITY, INFINITY};
            auto encode_vec = [&](auto bits_tag) {
                constexpr int BITS = decltype(bits_tag)::value;
                constexpr int NT = (1 << (BITS - 1)) - 1;
                float T[NT];   // (constant indices: read from the constant bank)
                if (is_v) {
#pragma unroll
                    for (int i = 0; i < NT; ++i) T[i] = p.v_gt[i] * scale;
                } else {
#pragma unroll
                    for (int i = 0; i < NT; ++i) T[i] = p.k_gt[i] * scale;
                }
                if constexpr (PACKED) {
                    // few dims a turn: with the distances kept, two quarters unrolled
                    // outgrow the instruction cache
#pragma unroll 1
                    for (int q = 0; q < (BITS == 4 ? 8 : 4); ++q) {
                        if constexpr (BITS == 4) {   // 16 dims: two words
                            uint32_t ra[16];
                            tmem_ld16(tacc + 16 * q, ra);
                            const uint32_t w0 = pack_word4<true>(ra, T, near4), w1 = pack_word4<true>(ra + 8, T, near4);
                            if (valid) *reinterpret_cast<uint2*>(dst + 8 * q) = make_uint2(w0, w1);
                        } else {
                            uint32_t w[BITS], ra[32];
                            tmem_ld32(tacc + 32 * q, ra);
                            pack_quarter<BITS, true>(ra, T, w, near4);
                            if (valid) {
#pragma unroll
                                for (int i = 0; i < 3; ++i) reinterpret_cast<uint32_t*>(dst + 12 * q)[i] = w[i];
                            }
                        }
                    }
                    return;
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {   // quarters 2h, 2h+1 (bytes 8 h BITS ..)
                    uint32_t w[2 * BITS];
                    uint32_t ra[32], rb[32];
                    tmem_ld32_issue(tacc + 64 * h, ra);
                    tmem_ld32_issue(tacc + 64 * h + 32, rb);
                    tmem_ld_wait(ra, rb);
                    pack_quarter<BITS, false>(ra, T, w, near4);
                    pack_quarter<BITS, false>(rb, T, w + BITS, near4);
                    if (valid) {
                        uint8_t* d = dst + h * 8 * BITS;
                        if constexpr (BITS == 4) {
                            reinterpret_cast<uint4*>(d)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint4*>(d)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        } else if (h == 0) {   // bytes 0..23: 16 + 8
                            reinterpret_cast<uint4*>(d)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint2*>(d)[2] = make_uint2(w[4], w[5]);
                        } else {               // bytes 24..47: 8 + 16
                            reinterpret_cast<uint2*>(d)[0] = make_uint2(w[0], w[1]);
                            reinterpret_cast<uint4*>(d + 8)[0] = make_uint4(w[2], w[3], w[4], w[5]);
                        }
                    }
                }
            };
            if constexpr (KB == VB || KB == 0) {
                encode_vec(std::integral_constant<int, VB>{});
            } else {
                if (is_v) encode_vec(std::integral_constant<int, VB>{});
                else encode_vec(std::integral_constant<int, KB>{});
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_afree + 8 * g);
            if constexpr (PACKED) {
                // vectors too near a threshold, one at a time by the whole warp
                // (a zero vector's codes are right: every y and T is 0)
                const float near = fminf(fminf(near4[0], near4[1]), fminf(near4[2], near4[3]));
                const float nrm = sqrtf(S32);
                const bool fine = least >= (is_v ? p.v_fine_min : p.k_fine_min) * nrm;
                const float band = is_v ? (fine ? p.v_near_fine : p.v_near) : (fine ? p.k_near_fine : p.k_near);
                unsigned redo = __ballot_sync(0xffffffffu, valid && S32 > 0.f && near <= band * nrm);
                while (redo) {
                    const int src = __ffs(redo) - 1;
                    redo &= redo - 1;
                    const unsigned long long at =
                        __shfl_sync(0xffffffffu, static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(dst)), src);
                    const int vs = __shfl_sync(0xffffffffu, v, src);
                    const __half* x = (is_v ? p.v_new : p.k_new) + static_cast<size_t>(vs) * kD;
                    const uint2 raw = reinterpret_cast<const uint2*>(x)[lane];
                    uint8_t* const out = reinterpret_cast<uint8_t*>(static_cast<uintptr_t>(at));
                    __syncwarp();   // after that lane's own stores of the record
                    if (is_v) encode_exact_warp<VB>(raw, out, p.signs, p.v_mag, lane);
                    else encode_exact_warp<(KB == 0 ? VB : KB)>(raw, out, p.signs, p.k_mag, lane);
                }
            }
        }
        if (stalled && lane == 0) atomicOr(p.status, kStatusPipelineStall);
    }
    if constexpr (PACKED)
        if (down)
            append_shared_rows<KB, VB>(p, static_cast<long long>(blockIdx.x) * (kTcEncWarps + 1) + warp,
                                       static_cast<long long>(gridDim.x) * (kTcEncWarps + 1), lane);
    finish_append<PACKED>(p, lane);   // every thread has read lengths[] for the last time, no more tiles taken
    tc_fence_before();
    __syncthreads();
    if (warp == kTcEncWarps) tmem_dealloc(tmem, 256);
}

// Small appends (a few tokens per sequence): one warp per vector, lane l holds
// dims 4l .. 4l+3, so every vector gets its own warp and the dependent chain
// per lane is short.  Here u itself is formed and compared exactly against the
// fp32 midpoints (the large-append kernel compares the unnormalised value with
// scaled thresholds: elements within ~1e-6 of a midpoint may round the other
// way there).
template <int BITS, bool PACKED>
__device__ __forceinline__ void encode_vector_warp(const uint2 raw, uint8_t* dst,
                                                   __half* dst_norm, const float* tcb,
                                                   const uint32_t (&signs)[4], const float* gt,
                                                   const float* ge, const float* mag, float near_band,
                                                   uint32_t* status, int lane) {
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
    float x[4] = {f0.x, f0.y, f1.x, f1.y};

    float ss = fmaf(x[0], x[0], x[1] * x[1]) + fmaf(x[2], x[2], x[3] * x[3]);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const float S32 = __shfl_sync(0xffffffffu, ss, 0);
    bool ok;
    unsigned short nb = norm_candidate<20>(S32, ok);   // at most 2 + 5 roundings per square
    if (!__all_sync(0xffffffffu, ok)) {
        // exact sum of squares (units of 2^-48) as a 128-bit integer
        U128 S = sq_u128(fp16_scaled_int(x[0]));
#pragma unroll
        for (int i = 1; i < 4; ++i) S = add128(S, sq_u128(fp16_scaled_int(x[i])));
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) {
            U128 o;
            o.lo = __shfl_xor_sync(0xffffffffu, S.lo, m);
            o.hi = __shfl_xor_sync(0xffffffffu, S.hi, m);
            S = add128(S, o);
        }
        nb = norm_to_half(S);
    }
    if (lane == 0) {
        store_norm(dst_norm, dst, tcb, nb);
        if (nb >= 0x7C00u) atomicOr(status, kStatusNormOverflow);
    }

    // rotate: u = H (s * x) / (sqrt(128) n)
    const uint32_t sn = sign_nibble(signs, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = ((sn >> i) & 1u) ? -x[i] : x[i];
    wht128_lane4(x, lane);
    const float n = sqrtf(S32);
    const float inv = (n > 0.f) ? 1.0f / (n * 11.313708498984761f) : 0.f;
    constexpr int H = 1 << (BITS - 1);
    bool any_tie = false;
#pragma unroll
    for (int k = 0; k < H - 1; ++k) any_tie |= ge[k] != gt[k];
    uint32_t code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) code[i] = quantize_code<BITS>(x[i] * inv, gt, ge, any_tie);
    if constexpr (PACKED) {
        // (the values here are y / (sqrt(128) n))
        float near = INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = fabsf(x[i] * inv);
            near = fminf(near, a);
#pragma unroll
            for (int k = 0; k < H - 1; ++k) near = fminf(near, fabsf(gt[k] - a));
        }
        if (n > 0.f && __any_sync(0xffffffffu, near <= near_band * 0.08838834764831845f)) {
            encode_exact_warp<BITS>(raw, dst, signs, mag, lane);
            return;
        }
    }

    store_codes_warp<BITS>(code, dst, lane);
}

// grid: 4 warps per CTA, warp = (K-or-V, vector).  KB = 0 copies fp16 K rows.
template <int KB, int VB, bool PACKED>
__global__ void __launch_bounds__(128) tq_encode_small_kernel(const __grid_constant__ EncodeParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long gw = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const long long nvec = PACKED ? static_cast<long long>(p.total) * p.hkv
                                  : static_cast<long long>(p.batch) * p.hkv * p.t_new;
    // lengths[lane] for the last CTA's update (warp 0), read now with the rest
    const int len_pre = (threadIdx.x < 32 && lane < p.batch) ? p.lengths[lane] : 0;
    // and the bounds that this thread checks at the end
    int cu0 = 0, cu1 = 0;
    if (PACKED && threadIdx.x < static_cast<unsigned int>(p.batch)) {
        cu0 = p.cu[threadIdx.x];
        cu1 = p.cu[threadIdx.x + 1];
    }
    if (gw < 2 * nvec) {
        const int which = static_cast<int>(gw & 1);  // 0 = K, 1 = V
        const long long v = gw >> 1;
        // the vector does not depend on the length: both loads go out together
        const __half* src = (which ? p.v_new : p.k_new) + v * kD;
        const uint2 raw = reinterpret_cast<const uint2*>(src)[lane];
        bool live, first_over;   // first_over: one thread's per sequence that would pass the capacity
        size_t pos;
        if constexpr (PACKED) {
            const int tok = static_cast<int>(v / p.hkv), h = static_cast<int>(v) - tok * p.hkv;
            const PackedSlot ps = packed_slot(p, tok);
            live = ps.live;
            first_over = ps.first_over && h == 0;
            pos = (static_cast<size_t>(ps.b) * p.hkv + h) * p.cap + ps.pos;
        } else {
            const int t = static_cast<int>(v % p.t_new);
            const long long bh = v / p.t_new;
            const int b = static_cast<int>(bh / p.hkv);
            const int L = p.lengths[b];
            live = !(L < 0 || L + p.t_new > p.cap);
            first_over = !live && t == 0 && (bh % p.hkv) == 0;
            pos = static_cast<size_t>(bh) * p.cap + L + t;
        }
        if (!live) {
            if (lane == 0 && which == 0 && first_over) atomicOr(p.status, kStatusCapacity);
        } else {
            if (which == 0) {
                if constexpr (KB == 0) {
                    reinterpret_cast<uint2*>(p.k_codes + pos * 256)[lane] = raw;
                } else {
                    encode_vector_warp<KB, PACKED>(raw, p.k_codes + pos * (p.table ? 64 : KB * 16),
                                                   p.k_norm + pos, p.table ? p.k_cb : nullptr, p.signs,
                                                   p.k_gt, p.k_ge, p.k_mag, p.k_near, p.status, lane);
                }
            } else {
                encode_vector_warp<VB, PACKED>(raw, p.v_codes + pos * (p.table ? 64 : VB * 16),
                                               p.v_norm + pos, p.table ? p.v_cb : nullptr, p.signs,
                                               p.v_gt, p.v_ge, p.v_mag, p.v_near, p.status, lane);
            }
        }
    }
    if constexpr (PACKED) {
        bool down = threadIdx.x < static_cast<unsigned int>(p.batch) && cu0 > cu1;
        for (int bb = threadIdx.x + 128; bb < p.batch; bb += 128) down = down || p.cu[bb] > p.cu[bb + 1];
        if (__syncthreads_or(down)) {
            append_shared_rows<KB, VB>(p, gw, 4ll * gridDim.x, lane);
            __syncthreads();
        }
    }
    finish_append_small<PACKED>(p, lane, len_pre);
}


template <int KB, int VB, bool PACKED>
static int launch_encode_t(const EncodeParams& p, long long nvec, const CUtensorMap* kmap, const CUtensorMap* vmap,
                           cudaStream_t stream) {
    if (nvec <= kEncodeSmallMax) {   // a warp per vector: short chains for small appends
        const dim3 grid(static_cast<unsigned int>((2 * nvec + 3) / 4));
        return launch_pdl(tq_encode_small_kernel<KB, VB, PACKED>, grid, dim3(128), 0, stream, p);
    }
    if (kmap == nullptr || vmap == nullptr) return cudaErrorInvalidValue;
    const long long tiles = (KB == 0 ? 1 : 2) * (PACKED ? (p.total + kTcVecs - 1) / kTcVecs * 1ll * p.hkv
                                                        : (nvec + kTcVecs - 1) / kTcVecs);
    const dim3 grid(static_cast<unsigned int>(std::min<long long>(tiles, 152ll * kTcCtasPerSm)));
    static std::atomic<uint64_t> attr_done{0};   // two CTAs' shared memory: the largest carveout
    const cudaError_t e = set_smem_attr_once(tq_encode_tc_kernel<KB, VB, PACKED>, kTcSmemAlloc, attr_done, 100);
    if (e != cudaSuccess) return e;
    return launch_pdl(tq_encode_tc_kernel<KB, VB, PACKED>, grid, dim3(kTcThreads), kTcSmemAlloc, stream, p, *kmap,
                      *vmap);
}

template <bool PACKED>
static int launch_encode_bits(int kbits, int vbits, const EncodeParams& p, long long nvec, const CUtensorMap* kmap,
                              const CUtensorMap* vmap, cudaStream_t stream) {
    if (kbits == 16 && vbits == 4) return launch_encode_t<0, 4, PACKED>(p, nvec, kmap, vmap, stream);
    if (kbits == 3 && vbits == 3) return launch_encode_t<3, 3, PACKED>(p, nvec, kmap, vmap, stream);
    if (kbits == 4 && vbits == 4) return launch_encode_t<4, 4, PACKED>(p, nvec, kmap, vmap, stream);
    if (kbits == 16 && vbits == 3) return launch_encode_t<0, 3, PACKED>(p, nvec, kmap, vmap, stream);
    if (kbits == 4 && vbits == 3) return launch_encode_t<4, 3, PACKED>(p, nvec, kmap, vmap, stream);
    return cudaErrorInvalidValue;
}

int launch_encode(int kbits, int vbits, const EncodeParams& p, const CUtensorMap* kmap,
                  const CUtensorMap* vmap, cudaStream_t stream) {
    return launch_encode_bits<false>(kbits, vbits, p, 1ll * p.batch * p.hkv * p.t_new, kmap, vmap, stream);
}

int launch_encode_packed(int kbits, int vbits, const EncodeParams& p, const CUtensorMap* kmap,
                         const CUtensorMap* vmap, cudaStream_t stream) {
    return launch_encode_bits<true>(kbits, vbits, p, 1ll * p.total * p.hkv, kmap, vmap, stream);
}

}  // namespace tq
