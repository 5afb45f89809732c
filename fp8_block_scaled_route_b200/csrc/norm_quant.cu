// RMS norm with the residual's addition and 8-bit rows, and the per-row int8
// quantiser: the steps that hand bf16 rows to the expert GEMMs.
//
//   h = bf16(x + residual);  r = fp32(1 / sqrt(mean(h^2) + eps));
//   y = (h * r) * w  (fp32, two roundings);  out: bf16(y) and / or 8-bit rows of y.
//
// The mean square is summed in 64 bits.  Every other step is one elementwise
// fp32 rounding, so with a correctly rounded r the 8-bit codes do not depend
// on how a row is split over threads: a sum in 32 bits would move r by an ulp
// and flip the codes that lie next to a rounding border.  The 64-bit sum costs
// a conversion and a fused multiply-add per element, which the loads hide.
//
// 8-bit formats of a row (amax over the row's group of columns):
//   FP8    scale amax / 448 per 128 columns, codes RNE_sat(y * (448 / amax))
//   MXFP8  E8M0 scale per 32 columns as swiglu_mxfp8_quant; codes exact scaling
//   INT8   scale amax / 127 per row, codes RNE(y * (127 / amax))
// Multiplying by the once-divided reciprocal replaces a division per element;
// the product differs from the quotient in the last bit only.  Groups with
// amax < 2^-100 (448 / amax would overflow near 2^-119) get scale 1 and codes
// 0.  A NaN reaches the group's scale (max with NaN).
//
// Bound: HBM.  A row is held in registers between its two passes (statistic,
// output), so every byte is moved once.
#include <cuda_bf16.h>

#include <cstring>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr float kTinyGroup = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ void unpack8(const uint4& r, float (&f)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        memcpy(&w[i], &b, 4);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float amax8(const float (&f)[8]) {
    float m = fabsf(f[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmax_nan(m, fabsf(f[i]));
    return m;
}

// Largest value over the row's TPR threads, the same in every thread.
// red: [warps of the CTA] floats.
template <int TPR>
__device__ __forceinline__ float row_max(float m, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) red[threadIdx.y * W + warp] = m;
        __syncthreads();
        m = red[threadIdx.y * W];
        for (int i = 1; i < W; ++i) m = fmax_nan(m, red[threadIdx.y * W + i]);
    }
    return m;
}

struct GroupScale {
    float scale, inv;
};
__device__ __forceinline__ GroupScale group_scale(float amax, float top) {
    GroupScale g;
    const bool zero = amax < kTinyGroup;
    g.scale = zero ? 1.0f : __fdiv_rn(amax, top);
    g.inv = zero ? 0.0f : __fdiv_rn(top, amax);
    return g;
}

// Codes of an int8 row: a zero group's codes are 0 whatever the values.
__device__ __forceinline__ uint2 int8_codes(const float (&f)[8], float inv) {
    return make_uint2(cvt_s8x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                      cvt_s8x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

// Rows per CTA: at least 256 threads.
template <int TPR>
constexpr int kRowsPerCta = TPR >= 256 ? 1 : 256 / TPR;

// blockDim (TPR, rows per CTA): TPR threads share a row, each with V groups of
// 8 consecutive columns, TPR groups apart (coalesced 16-byte accesses).
template <int TPR, int V, int FMT>
__global__ void __launch_bounds__(TPR* kRowsPerCta<TPR>)
    rmsnorm_kernel(const RmsNormArgs p) {
    constexpr int RPC = kRowsPerCta<TPR>;
    constexpr int W = TPR / 32;
    __shared__ double sums[RPC * W];
    __shared__ float red[RPC * W];
    __shared__ float rstd[RPC];
    const int t = blockIdx.x * RPC + threadIdx.y;
    const bool row_ok = t < p.T;
    const int nvec = p.H >> 3;
    const long long base = static_cast<long long>(t) * nvec;
    const uint4* x = static_cast<const uint4*>(p.x) + base;
    const uint4* res = static_cast<const uint4*>(p.residual) + base;
    uint4 xr[V], rr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * TPR;
        const bool live = row_ok && c < nvec;
        xr[i] = live ? x[c] : make_uint4(0, 0, 0, 0);
        rr[i] = live && p.residual ? res[c] : make_uint4(0, 0, 0, 0);
    }
    float h[V][8];
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * TPR;
        unpack8(xr[i], h[i]);
        if (p.residual) {
            float a[8];
            unpack8(rr[i], a);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] += h[i][j];
            const uint4 hb = pack8(a);
            unpack8(hb, h[i]);
            if (row_ok && c < nvec && p.residual_out)
                (static_cast<uint4*>(p.residual_out) + base)[c] = hb;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const double d = static_cast<double>(h[i][j]);
            ss = fma(d, d, ss);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    float r;
    if constexpr (TPR == 32) {
        r = static_cast<float>(rsqrt(ss / p.H + p.eps));
    } else {
        if ((threadIdx.x & 31) == 0) sums[threadIdx.y * W + (threadIdx.x >> 5)] = ss;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < W; ++i) ss += sums[threadIdx.y * W + i];
            rstd[threadIdx.y] = static_cast<float>(rsqrt(ss / p.H + p.eps));
        }
        __syncthreads();
        r = rstd[threadIdx.y];
    }
    float row_amax = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * TPR;
        const bool live = c < nvec;
        float w[8] = {};
        if (live) {
            if (p.weight_bf16) {
                unpack8(__ldg(static_cast<const uint4*>(p.weight) + c), w);
            } else {
                const float4 a = __ldg(static_cast<const float4*>(p.weight) + 2 * c);
                const float4 b = __ldg(static_cast<const float4*>(p.weight) + 2 * c + 1);
                w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
                w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = live ? h[i][j] * r * w[j] : 0.0f;
        if (p.y && row_ok && live) (static_cast<uint4*>(p.y) + base)[c] = pack8(h[i]);
        if constexpr (FMT == NQ_FP8) {
            float m = amax8(h[i]);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            const GroupScale g = group_scale(m, 448.0f);
            if (row_ok && live) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = h[i][j] * g.inv;
                reinterpret_cast<uint2*>(p.q)[base + c] =
                    make_uint2(cvt_e4m3x4(f[0], f[1], f[2], f[3]), cvt_e4m3x4(f[4], f[5], f[6], f[7]));
                if ((c & 15) == 0) {
                    const int kb = c >> 4;
                    float* s = static_cast<float*>(p.q_scale);
                    if (p.scale_mn) s[static_cast<long long>(kb) * p.T + t] = g.scale;
                    else s[static_cast<long long>(t) * (p.H >> 7) + kb] = g.scale;
                }
            }
        }
        if constexpr (FMT == NQ_MXFP8) {
            float m = amax8(h[i]);
#pragma unroll
            for (int o = 2; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            // NaN and infinity: the E8M0 NaN code
            const uint32_t code = m <= 3.402823466e38f ? e8m0_code(m) : 255u;
            const float inv = e8m0_reciprocal(min(code, 254u));
            if (row_ok && live) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = h[i][j] * inv;
                reinterpret_cast<uint2*>(p.q)[base + c] =
                    make_uint2(cvt_e4m3x4(f[0], f[1], f[2], f[3]), cvt_e4m3x4(f[4], f[5], f[6], f[7]));
                if ((c & 3) == 0) {
                    const int b = c >> 2;  // 32-column block
                    uint8_t* s = static_cast<uint8_t*>(p.q_scale);
                    if (p.scale_mn) s[(static_cast<long long>(b >> 2) * p.T + t) * 4 + (b & 3)] = code;
                    else s[static_cast<long long>(t) * (p.H >> 5) + b] = code;
                }
            }
        }
        if constexpr (FMT == NQ_INT8) row_amax = fmax_nan(row_amax, amax8(h[i]));
    }
    if constexpr (FMT == NQ_INT8) {
        const GroupScale g = group_scale(row_max<TPR>(row_amax, red), 127.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * TPR;
            if (row_ok && c < nvec) reinterpret_cast<uint2*>(p.q)[base + c] = int8_codes(h[i], g.inv);
        }
        if (row_ok && threadIdx.x == 0) static_cast<float*>(p.q_scale)[t] = g.scale;
    }
}

// Row t of x [T, K] -> int8 codes and scale at rows inv_perm[t*k + j] (row t
// when inv_perm is null); entries outside [0, R) are skipped.
template <int TPR, int V>
__global__ void __launch_bounds__(TPR* kRowsPerCta<TPR>)
    int8_quant_kernel(const __nv_bfloat16* __restrict__ xin, int T, int K, int k, int R,
                      const int32_t* __restrict__ inv_perm, int8_t* __restrict__ q,
                      float* __restrict__ q_scale) {
    constexpr int RPC = kRowsPerCta<TPR>;
    __shared__ float red[RPC * (TPR / 32)];
    const int t = blockIdx.x * RPC + threadIdx.y;
    const bool row_ok = t < T;
    const int nvec = K >> 3;
    const uint4* x = reinterpret_cast<const uint4*>(xin) + static_cast<long long>(t) * nvec;
    uint4 xr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * TPR;
        xr[i] = row_ok && c < nvec ? x[c] : make_uint4(0, 0, 0, 0);
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float f[8];
        unpack8(xr[i], f);
        m = fmax_nan(m, amax8(f));
    }
    const GroupScale g = group_scale(row_max<TPR>(m, red), 127.0f);
    if (!row_ok) return;
    uint2 codes[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float f[8];
        unpack8(xr[i], f);
        codes[i] = int8_codes(f, g.inv);
    }
    for (int j = 0; j < k; ++j) {
        const int row = inv_perm ? inv_perm[static_cast<long long>(t) * k + j] : t;
        if (row < 0 || row >= R) continue;
        uint2* dst = reinterpret_cast<uint2*>(q) + static_cast<long long>(row) * nvec;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * TPR;
            if (c < nvec) dst[c] = codes[i];
        }
        if (threadIdx.x == 0) q_scale[row] = g.scale;
    }
}

template <int TPR, int V>
int launch_norm(const RmsNormArgs& p, cudaStream_t s) {
    constexpr int RPC = kRowsPerCta<TPR>;
    const dim3 block(TPR, RPC);
    const unsigned grid = static_cast<unsigned>((p.T + RPC - 1) / RPC);
    switch (p.fmt) {
        case NQ_NONE: rmsnorm_kernel<TPR, V, NQ_NONE><<<grid, block, 0, s>>>(p); break;
        case NQ_FP8: rmsnorm_kernel<TPR, V, NQ_FP8><<<grid, block, 0, s>>>(p); break;
        case NQ_MXFP8: rmsnorm_kernel<TPR, V, NQ_MXFP8><<<grid, block, 0, s>>>(p); break;
        default: rmsnorm_kernel<TPR, V, NQ_INT8><<<grid, block, 0, s>>>(p); break;
    }
    return cudaGetLastError() == cudaSuccess ? ST_OK : ST_CUDA;
}

template <int TPR, int V>
int launch_q8(const void* x, int T, int K, int k, int R, const int32_t* inv_perm, int8_t* q,
              float* q_scale, cudaStream_t s) {
    constexpr int RPC = kRowsPerCta<TPR>;
    int8_quant_kernel<TPR, V><<<static_cast<unsigned>((T + RPC - 1) / RPC), dim3(TPR, RPC), 0, s>>>(
        static_cast<const __nv_bfloat16*>(x), T, K, k, R, inv_perm, q, q_scale);
    return cudaGetLastError() == cudaSuccess ? ST_OK : ST_CUDA;
}

}  // namespace

int launch_rmsnorm(const RmsNormArgs& p, int num_sms, cudaStream_t s) {
    if (p.T == 0) return ST_OK;
    const int nvec = p.H >> 3;
    if (nvec <= 32) return launch_norm<32, 1>(p, s);
    if (nvec <= 64) return launch_norm<64, 1>(p, s);
    if (nvec <= 128) return launch_norm<128, 1>(p, s);
    if (nvec <= 256) return launch_norm<256, 1>(p, s);
    if (nvec <= 512) return launch_norm<256, 2>(p, s);
    if (nvec <= 1024) return launch_norm<256, 4>(p, s);
    if (nvec <= 2048) return launch_norm<512, 4>(p, s);
    return launch_norm<1024, 4>(p, s);
}

int launch_int8_quant(const void* x, int T, int K, int k, int R, const int32_t* inv_perm,
                      int8_t* q, float* q_scale, int num_sms, cudaStream_t s) {
    if (T == 0) return ST_OK;
    const int nvec = K >> 3;
    if (nvec <= 32) return launch_q8<32, 1>(x, T, K, k, R, inv_perm, q, q_scale, s);
    if (nvec <= 64) return launch_q8<64, 1>(x, T, K, k, R, inv_perm, q, q_scale, s);
    if (nvec <= 128) return launch_q8<128, 1>(x, T, K, k, R, inv_perm, q, q_scale, s);
    if (nvec <= 256) return launch_q8<256, 1>(x, T, K, k, R, inv_perm, q, q_scale, s);
    if (nvec <= 512) return launch_q8<256, 2>(x, T, K, k, R, inv_perm, q, q_scale, s);
    if (nvec <= 1024) return launch_q8<256, 4>(x, T, K, k, R, inv_perm, q, q_scale, s);
    if (nvec <= 2048) return launch_q8<512, 4>(x, T, K, k, R, inv_perm, q, q_scale, s);
    return launch_q8<1024, 4>(x, T, K, k, R, inv_perm, q, q_scale, s);
}

}  // namespace moe
