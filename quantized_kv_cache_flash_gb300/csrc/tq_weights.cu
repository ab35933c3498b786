// The softmax weights that cached tokens get from a block of queries
// (tq_attention_weights), the plain way: K tiles dequantised to fp32 in shared
// memory, scores as fp32 sums, two passes over them (the rows' log-sum-exp, then the
// tokens' sums).
#include <algorithm>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

constexpr int kWtTok = 64, kWtRows = 16, kWtThreads = 128, kWtStride = kD + 1;

// Rot(q) (quantized K) or q as fp32 rows of the workspace; a warp a row.
__global__ void __launch_bounds__(128) tq_weights_rows_kernel(const __grid_constant__ WeightsParams p, int quantized) {
    const int lane = threadIdx.x & 31;
    const size_t row = static_cast<size_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    griddep_wait();
    if (row >= static_cast<size_t>(p.batch) * p.hkv * p.rows) return;
    const int unit = static_cast<int>(row / p.rows), r = static_cast<int>(row % p.rows);
    const int b = unit / p.hkv, h = unit % p.hkv, j = r / p.group, g = r % p.group;
    const __half* q = p.q + ((static_cast<size_t>(b) * p.hq + h * p.group + g) * p.tq + j) * kD + 4 * lane;
    float v[4];
    for (int i = 0; i < 4; ++i) v[i] = __half2float(q[i]);
    if (quantized) {
        const uint32_t sn = sign_nibble(p.signs, lane);
        for (int i = 0; i < 4; ++i) v[i] = ((sn >> i) & 1u) ? -v[i] : v[i];
        wht128_lane4(v, lane);
        for (int i = 0; i < 4; ++i) v[i] *= 0.08838834764831845f;
    }
    *reinterpret_cast<float4*>(p.q_rot + row * kD + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
    if (lane == 0 && min(p.lengths[b], p.max_len) - 1 < 0) atomicOr(p.status, kStatusShortContext);
    else if (lane == 0 && p.lengths[b] - p.tq + j < 0) atomicOr(p.status, kStatusShortContext);
}

// A tile of 64 tokens from tok0 as fp32 levels (times the norm, and the softmax scale).
template <int KB>
__device__ void load_k(const WeightsParams& p, size_t row0, int tok0, int lim, float* sK) {
    const Tables kt{p.ktab[0], p.ktab[1], p.ktab[2], p.ktab[3]};
    for (int x = threadIdx.x; x < kWtTok * 4; x += kWtThreads) {
        const int t = x >> 2, q = x & 3;
        uint32_t hh[16];
        float s = p.scale_log2e;
        const bool in = tok0 + t < lim;
        const size_t at = row0 + (in ? tok0 + t : 0);
        if constexpr (KB == 0) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(p.k_codes + at * 256) + 16 * q;
            for (int i = 0; i < 16; ++i) hh[i] = src[i];
        } else {
            dequant_q32<KB>(p.k_codes + at * (16 * KB) + q * 4 * KB, kt, hh);
            s *= __half2float(p.k_norm[at]);
        }
        for (int i = 0; i < 16; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hh[i]));
            sK[t * kWtStride + 32 * q + 2 * i] = in ? f.x * s : 0.f;
            sK[t * kWtStride + 32 * q + 2 * i + 1] = in ? f.y * s : 0.f;
        }
    }
}

template <int KB>
__global__ void __launch_bounds__(kWtThreads) tq_weights_lse_kernel(const __grid_constant__ WeightsParams p) {
    __shared__ float sK[kWtTok * kWtStride];
    __shared__ float sQ[kWtRows * kD];
    __shared__ float sM[kWtThreads], sL[kWtThreads];
    griddep_wait();
    const int groups = (p.rows + kWtRows - 1) / kWtRows;
    const int unit = static_cast<int>(blockIdx.x) / groups, r0 = (static_cast<int>(blockIdx.x) % groups) * kWtRows;
    const int b = unit / p.hkv, tid = threadIdx.x;
    const int L = p.lengths[b], lim = min(L, p.max_len);
    const size_t qrow = static_cast<size_t>(unit) * p.rows;
    for (int x = tid; x < kWtRows * kD; x += kWtThreads)
        sQ[x] = r0 + x / kD < p.rows ? p.q_rot[(qrow + r0) * kD + x] : 0.f;
    float m[8], l[8];
    for (int i = 0; i < 8; ++i) m[i] = -INFINITY, l[i] = 0.f;
    const int t = tid & 63, half = tid >> 6;
    const int r_last = min(p.rows - 1, r0 + kWtRows - 1);
    const int last = min(lim - 1, L - p.tq + r_last / p.group);
    for (int tok0 = 0; tok0 <= last; tok0 += kWtTok) {
        __syncthreads();
        load_k<KB>(p, static_cast<size_t>(unit) * p.cap, tok0, lim, sK);
        __syncthreads();
        float s[8] = {};
        for (int d = 0; d < kD; ++d)
            for (int i = 0; i < 8; ++i) s[i] = fmaf(sK[t * kWtStride + d], sQ[(8 * half + i) * kD + d], s[i]);
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + 8 * half + i;
            if (tok0 + t < lim && tok0 + t <= L - p.tq + r / p.group) {
                const float mn = s[i] > m[i] || s[i] != s[i] ? s[i] : m[i];
                l[i] = (m[i] == -INFINITY ? 0.f : l[i] * fast_exp2(m[i] - mn)) + fast_exp2(s[i] - mn);
                m[i] = mn;
            }
        }
    }
    for (int i = 0; i < 8; ++i) {
        __syncthreads();
        sM[tid] = m[i];
        sL[tid] = l[i];
        __syncthreads();
        if (t == 0 && r0 + 8 * half + i < p.rows) {
            float M = -INFINITY, S = 0.f;
            for (int k = 0; k < 64; ++k) M = fmaxf(M, sM[tid + k]);
            for (int k = 0; k < 64; ++k)
                if (sM[tid + k] != -INFINITY) S += sL[tid + k] * fast_exp2(sM[tid + k] - M);
            p.lse[qrow + r0 + 8 * half + i] = M == -INFINITY && S == 0.f ? INFINITY : M + log2f(S);
        }
    }
}

template <int KB>
__global__ void __launch_bounds__(kWtThreads) tq_weights_sum_kernel(const __grid_constant__ WeightsParams p) {
    __shared__ float sK[kWtTok * kWtStride];
    __shared__ float sQ[kWtRows * kD];
    __shared__ float sW[kWtThreads], sLse[kWtRows];
    griddep_wait();
    const int tiles = (p.max_len + kWtTok - 1) / kWtTok;
    const int unit = static_cast<int>(blockIdx.x) / tiles, tok0 = (static_cast<int>(blockIdx.x) % tiles) * kWtTok;
    const int b = unit / p.hkv, tid = threadIdx.x;
    const int L = p.lengths[b], lim = min(L, p.max_len);
    if (tok0 >= lim) return;
    const size_t qrow = static_cast<size_t>(unit) * p.rows;
    load_k<KB>(p, static_cast<size_t>(unit) * p.cap, tok0, lim, sK);
    const int t = tid & 63, half = tid >> 6;
    float a = 0.f;
    for (int r0 = 0; r0 < p.rows; r0 += kWtRows) {
        __syncthreads();
        for (int x = tid; x < kWtRows * kD; x += kWtThreads)
            sQ[x] = r0 + x / kD < p.rows ? p.q_rot[(qrow + r0) * kD + x] : 0.f;
        if (tid < kWtRows) sLse[tid] = r0 + tid < p.rows ? p.lse[qrow + r0 + tid] : INFINITY;
        __syncthreads();
        float s[8] = {};
        for (int d = 0; d < kD; ++d)
            for (int i = 0; i < 8; ++i) s[i] = fmaf(sK[t * kWtStride + d], sQ[(8 * half + i) * kD + d], s[i]);
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + 8 * half + i;
            if (r < p.rows && tok0 + t <= L - p.tq + r / p.group) a += fast_exp2(s[i] - sLse[8 * half + i]);
        }
    }
    sW[tid] = a;
    __syncthreads();
    if (tid < kWtTok && tok0 + tid < lim) {
        const int seen = p.seen != nullptr ? p.seen[b] : L - p.tq;
        float* w = p.weights + static_cast<size_t>(unit) * p.cap + tok0 + tid;
        const float old = tok0 + tid < seen && p.decay != 0.f ? p.decay * *w : 0.f;
        *w = old + (sW[tid] + sW[tid + 64]);
    }
}

template <int KB>
static int launch_t(const WeightsParams& p, cudaStream_t stream) {
    const long long units = 1ll * p.batch * p.hkv;
    const long long g0 = (units * p.rows + 3) / 4, g1 = units * ((p.rows + kWtRows - 1) / kWtRows),
                    g2 = units * ((p.max_len + kWtTok - 1) / kWtTok);
    if (g1 > 0x7fffffffll || g2 > 0x7fffffffll) return cudaErrorInvalidValue;
    cudaError_t e = launch_pdl(tq_weights_rows_kernel, dim3(static_cast<unsigned>(g0)), dim3(128), 0, stream, p, KB);
    if (e == cudaSuccess)
        e = launch_pdl(tq_weights_lse_kernel<KB>, dim3(static_cast<unsigned>(g1)), dim3(kWtThreads), 0, stream, p);
    if (e == cudaSuccess)
        e = launch_pdl(tq_weights_sum_kernel<KB>, dim3(static_cast<unsigned>(g2)), dim3(kWtThreads), 0, stream, p);
    return e;
}

int launch_weights(int kbits, const WeightsParams& p, cudaStream_t stream) {
    if (kbits == 16) return launch_t<0>(p, stream);
    if (kbits == 3) return launch_t<3>(p, stream);
    if (kbits == 4) return launch_t<4>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace tq
