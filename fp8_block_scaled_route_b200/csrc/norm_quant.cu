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
#include "ptx_cluster.cuh"

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

// Largest value over the threads of a row (one warp, or blockDim.x of them),
// the same in every thread.  red: a float per warp of the CTA.
template <bool WARP>
__device__ __forceinline__ float row_max(float m, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if constexpr (!WARP) {
        const int W = blockDim.x >> 5;
        red += threadIdx.y * W;
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();
        m = red[0];
        for (int i = 1; i < W; ++i) m = fmax_nan(m, red[i]);
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

// blockDim (threads of a row, rows): a thread has V groups of 8 consecutive
// columns, blockDim.x groups apart (coalesced 16-byte accesses).  Measured at
// 8192 x 7168 with residual, bf16 and FP8 rows (530 MB, 81 us at the copy rate):
// V = 1 154 us, 2 83, 4 90, 8 159; one CTA walking over rows with the next
// row's loads in flight needs twice the registers and took 116.
template <bool WARP, int V, int FMT>
__global__ void __launch_bounds__(WARP ? 256 : V == 2 ? 512 : 1024, V == 2 && !WARP ? 3 : 1)
    rmsnorm_kernel(const RmsNormArgs p) {
    __shared__ double sums[32];
    __shared__ float red[32];
    __shared__ float rstd[8];
    pdl_launch();
    pdl_wait();
    const int TPR = blockDim.x;
    const int t = blockIdx.x * blockDim.y + threadIdx.y;
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
    if constexpr (WARP) {
        r = static_cast<float>(rsqrt(ss / p.H + p.eps));
    } else {
        const int W = TPR >> 5;
        double* row = sums + threadIdx.y * W;
        if ((threadIdx.x & 31) == 0) row[threadIdx.x >> 5] = ss;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < W; ++i) ss += row[i];
            rstd[threadIdx.y] = static_cast<float>(rsqrt(ss / p.H + p.eps));
        }
        __syncthreads();
        r = rstd[threadIdx.y];
    }
    float row_amax = 0.0f, gmax[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * TPR;
        const bool live = c < nvec;
        float w[8] = {};
        if (live) {
            if (p.weight_bf16) {
                unpack8(static_cast<const uint4*>(p.weight)[c], w);
            } else {
                const float4 a = static_cast<const float4*>(p.weight)[2 * c];
                const float4 b = static_cast<const float4*>(p.weight)[2 * c + 1];
                w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
                w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = live ? h[i][j] * r * w[j] : 0.0f;
        if (p.y && row_ok && live) (static_cast<uint4*>(p.y) + base)[c] = pack8(h[i]);
        if constexpr (FMT == NQ_FP8) {
            // 16 lanes hold a 128-column block
            gmax[i] = amax8(h[i]);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                gmax[i] = fmax_nan(gmax[i], __shfl_xor_sync(0xffffffffu, gmax[i], o));
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
    if constexpr (FMT == NQ_FP8) {
        // lane j of 16 divides for the half-warp's block j (j < V): two divisions
        // a thread instead of two a block and thread
        const int j = threadIdx.x & 15;
        float m = gmax[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = (j & (V - 1)) == i ? gmax[i] : m;
        const GroupScale g = group_scale(m, 448.0f);
        const int kb = ((threadIdx.x & ~15) + (j & (V - 1)) * TPR) >> 4;
        if (row_ok && j < V && kb < p.H >> 7) {
            float* s = static_cast<float*>(p.q_scale);
            if (p.scale_mn) s[static_cast<long long>(kb) * p.T + t] = g.scale;
            else s[static_cast<long long>(t) * (p.H >> 7) + kb] = g.scale;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * TPR;
            const float inv = __shfl_sync(0xffffffffu, g.inv, (threadIdx.x & 16) + i);
            float f[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) f[u] = h[i][u] * inv;
            if (row_ok && c < nvec)
                reinterpret_cast<uint2*>(p.q)[base + c] =
                    make_uint2(cvt_e4m3x4(f[0], f[1], f[2], f[3]), cvt_e4m3x4(f[4], f[5], f[6], f[7]));
        }
    }
    if constexpr (FMT == NQ_INT8) {
        const GroupScale g = group_scale(row_max<WARP>(row_amax, red), 127.0f);
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
// WIDE: CTAs of more than 256 threads, or several copies of a row that a CTA
// shares (without it such a row has one).
template <bool WARP, int V, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 1024 : 256, WIDE ? 1 : 6)
    int8_quant_kernel(const __nv_bfloat16* xin, int T, int K, int k, int R, const int32_t* inv_perm, int8_t* q,
                      float* q_scale) {
    // 65536 x 2048: one group a thread 92 us, four 68, and 59.0 (1.04 of the copy
    // rate) with six CTAs of 256 threads an SM (40 registers); with eight copies a
    // row the stores bound it, and fewer CTAs keep their runs longer: 8192 x 7168
    // 95 us against 101
    __shared__ float red[32];
    pdl_launch();
    pdl_wait();
    const int TPR = blockDim.x;
    const int t = blockIdx.x * blockDim.y + threadIdx.y;
    const bool row_ok = t < T;
    const int nvec = K >> 3;
    const uint4* x = reinterpret_cast<const uint4*>(xin) + static_cast<long long>(t) * nvec;
    uint4 xr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * TPR;
        xr[i] = row_ok && c < nvec ? x[c] : make_uint4(0, 0, 0, 0);
    }
    int row = t;
    if (inv_perm && row_ok) row = inv_perm[static_cast<long long>(t) * k];   // under the row's own loads
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float f[8];
        unpack8(xr[i], f);
        m = fmax_nan(m, amax8(f));
    }
    const GroupScale g = group_scale(row_max<WARP>(m, red), 127.0f);
    if (!row_ok) return;
    uint2 codes[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float f[8];
        unpack8(xr[i], f);
        codes[i] = int8_codes(f, g.inv);
    }
    const int copies = WARP || WIDE ? k : 1;
    for (int j = 0; j < copies; ++j) {
        // read ahead of the stores: for all the compiler knows they could change it
        const int next = j + 1 < copies ? inv_perm[static_cast<long long>(t) * k + j + 1] : -1;
        if (row >= 0 && row < R) {
            uint2* dst = reinterpret_cast<uint2*>(q) + static_cast<long long>(row) * nvec;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = threadIdx.x + i * TPR;
                if (c < nvec) dst[c] = codes[i];
            }
            if (threadIdx.x == 0) q_scale[row] = g.scale;
        }
        row = next;
    }
}

// Threads of a row and rows of a CTA for V groups of 8 columns a thread: at
// least 256 threads a CTA while a row takes at most 128 (the row's sums and the
// CTA's named results are sized for 32 warps and 8 rows).
dim3 row_block(int nvec, int V) {
    const int tpr = ((nvec + V - 1) / V + 31) / 32 * 32;
    return dim3(tpr, tpr <= 128 ? 256 / tpr : 1);
}

// Groups a thread.  Few rows: one, a row spread over as many warps as it can,
// while all of them are resident at about half the SMs' threads (64 x 7168 norm
// 3.5 us against 4.4 with four; 600 x 2048 4.1 against 4.6 with two).  Then two,
// and for the quantiser, which keeps less of a row, four above twice as much work
// (2400 x 4096 8.5 us with two, 7.0 with four).
int groups_a_thread(int T, int nvec, int num_sms, int most) {
    const long long work = static_cast<long long>(T) * nvec, half = 1100ll * num_sms;
    if (nvec <= 32 || (nvec <= 1024 && work <= half)) return 1;
    if (nvec <= 1024 && (most == 2 || work <= 2 * half)) return 2;
    return 4;
}

template <bool WARP, int V>
int launch_norm(const RmsNormArgs& p, dim3 block, cudaStream_t s) {
    const unsigned grid = (static_cast<unsigned>(p.T) + block.y - 1) / block.y;
    auto kern = p.fmt == NQ_NONE    ? rmsnorm_kernel<WARP, V, NQ_NONE>
                : p.fmt == NQ_FP8   ? rmsnorm_kernel<WARP, V, NQ_FP8>
                : p.fmt == NQ_MXFP8 ? rmsnorm_kernel<WARP, V, NQ_MXFP8>
                                    : rmsnorm_kernel<WARP, V, NQ_INT8>;
    return launch_dependent(kern, dim3(grid), block, 0, 0, s, p) == cudaSuccess ? ST_OK : ST_CUDA;
}

template <bool WARP, int V>
int launch_q8(const void* x, int T, int K, int k, int R, const int32_t* inv_perm, int8_t* q,
              float* q_scale, dim3 block, cudaStream_t s) {
    const unsigned grid = (static_cast<unsigned>(T) + block.y - 1) / block.y;
    const bool wide = !WARP && (k > 1 || block.x * block.y > 256);
    auto kern = wide ? int8_quant_kernel<WARP, V, !WARP> : int8_quant_kernel<WARP, V, false>;
    return launch_dependent(kern, dim3(grid), block, 0, 0, s, static_cast<const __nv_bfloat16*>(x), T, K, k,
                            R, inv_perm, q, q_scale) == cudaSuccess ? ST_OK : ST_CUDA;
}

}  // namespace

int launch_rmsnorm(const RmsNormArgs& p, int num_sms, cudaStream_t s) {
    if (p.T == 0) return ST_OK;
    const int nvec = p.H >> 3;
    const int per_thread = groups_a_thread(p.T, nvec, num_sms, 2);
    const dim3 block = row_block(nvec, per_thread);
    if (per_thread == 1)
        return block.x == 32 ? launch_norm<true, 1>(p, block, s) : launch_norm<false, 1>(p, block, s);
    if (per_thread == 2)
        return block.x == 32 ? launch_norm<true, 2>(p, block, s) : launch_norm<false, 2>(p, block, s);
    return launch_norm<false, 4>(p, block, s);
}

int launch_int8_quant(const void* x, int T, int K, int k, int R, const int32_t* inv_perm,
                      int8_t* q, float* q_scale, int num_sms, cudaStream_t s) {
    if (T == 0) return ST_OK;
    const int nvec = K >> 3;
    const int per_thread = groups_a_thread(T, nvec, num_sms, 4);
    const dim3 block = row_block(nvec, per_thread);
    const bool warp = block.x == 32;
    if (per_thread == 1)
        return warp ? launch_q8<true, 1>(x, T, K, k, R, inv_perm, q, q_scale, block, s)
                    : launch_q8<false, 1>(x, T, K, k, R, inv_perm, q, q_scale, block, s);
    if (per_thread == 2)
        return warp ? launch_q8<true, 2>(x, T, K, k, R, inv_perm, q, q_scale, block, s)
                    : launch_q8<false, 2>(x, T, K, k, R, inv_perm, q, q_scale, block, s);
    return warp ? launch_q8<true, 4>(x, T, K, k, R, inv_perm, q, q_scale, block, s)
                : launch_q8<false, 4>(x, T, K, k, R, inv_perm, q, q_scale, block, s);
}

}  // namespace moe
