// Routing and permutation: groups the T*k (token, slot) pairs by expert.
//
// The grouped layout is the m_indptr prefix array of the grouped GEMM
// interface on the page "FlashInfer SM120 MoE GEMM 최적화: 웨이브+잔여물 비용
// 모델 도입" (flashinfer PR #4318, "코드 분석 1."): rows of A grouped by
// expert, m_indptr[e] the first row of expert e.  Grouping is a stable
// counting sort on the pair id p = t*k + j, so the result is unique and
// bit-reproducible.
//
// Three launches (one for inputs of at most 8 chunks), no atomics on the
// output order:
//  1. route_hist:    one 1024-pair chunk per CTA -> per-chunk expert histogram
//  2. route_scan:    one CTA: per-expert exclusive scan over chunks, then the
//                    exclusive scan over experts -> m_indptr and the first
//                    output row of every (chunk, expert)
//  3. route_scatter: one warp per chunk walks its pairs in order, 32 at a
//                    time; lanes with the same expert are ranked with
//                    one warp ballot per expert-id bit, so each pair lands at
//                    chunk_base[e] + (earlier pairs of e in the chunk).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace moe {

// Lanes of the warp whose value equals this lane's, among the lanes with
// ok set, for values in [0, 2^nbits): one ballot per value bit (nbits
// uniform across the warp).  Used in place of the match instruction, whose
// cost grows with the number of distinct values in the warp.
__device__ __forceinline__ unsigned same_value_lanes(int v, bool ok, int nbits) {
    unsigned m = __ballot_sync(0xffffffffu, ok);
    for (int b = 0; b < nbits; ++b) {
        const bool bit = (v >> b) & 1;
        const unsigned bb = __ballot_sync(0xffffffffu, bit);
        m &= bit ? bb : ~bb;
    }
    return m;
}

__host__ __device__ inline int value_bits(int E) {
    int n = 0;
    while ((1 << n) < E) ++n;
    return n;
}

__global__ void __launch_bounds__(256) route_hist(const int32_t* __restrict__ ids, int R, int E,
                                                  int32_t* __restrict__ chunk_hist, int* status) {
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int base = blockIdx.x * kRouteChunk;
    const int end = min(R, base + kRouteChunk);
    int bad = 0;
    for (int p = base + threadIdx.x; p < end; p += blockDim.x) {
        const int e = ids[p];
        if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
        else ++bad;
    }
    if (bad) {
        atomicAdd(&status[2], bad);
        report_error(status, ST_BAD_EXPERT_ID, 0);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        chunk_hist[static_cast<long long>(blockIdx.x) * E + e] = hist[e];
}

// blockDim.x = 1024 >= E.  Each thread owns one expert; the per-chunk counts
// are read in batches of independent loads so the loop is not one memory
// latency per chunk.
__global__ void __launch_bounds__(1024) route_scan(int nchunks, int E, int32_t* __restrict__ chunk_hist,
                                                   int32_t* __restrict__ m_indptr) {
    __shared__ int warp_tot[32];
    constexpr int kBatch = 16;
    const int e = threadIdx.x;
    int count = 0;
    if (e < E) {
        for (int c0 = 0; c0 < nchunks; c0 += kBatch) {
            int h[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                h[i] = (c0 + i < nchunks) ? chunk_hist[static_cast<long long>(c0 + i) * E + e] : 0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (c0 + i < nchunks) chunk_hist[static_cast<long long>(c0 + i) * E + e] = count;  // rows of e in earlier chunks
                count += h[i];
            }
        }
    }
    // exclusive scan of count over experts
    const int lane = e & 31, w = e >> 5;
    int incl = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_tot[w] = incl;
    __syncthreads();
    if (w == 0) {
        int t = warp_tot[lane];
        int ti = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, ti, o);
            if (lane >= o) ti += v;
        }
        warp_tot[lane] = ti - t;  // exclusive prefix of warp totals
    }
    __syncthreads();
    const int excl = warp_tot[w] + incl - count;
    if (e < E) {
        m_indptr[e] = excl;
        for (int c = 0; c < nchunks; ++c) chunk_hist[static_cast<long long>(c) * E + e] += excl;
    }
    if (e == E - 1) m_indptr[E] = excl + count;
}

// blockDim.x = 32: one warp per chunk.  The chunk's expert ids are read up
// front (one batch of independent loads), then ranked 32 at a time.
__global__ void __launch_bounds__(32) route_scatter(const int32_t* __restrict__ ids, int R, int E,
                                                    const int32_t* __restrict__ chunk_base,
                                                    int32_t* __restrict__ perm,
                                                    int32_t* __restrict__ inv_perm) {
    extern __shared__ int cursor[];
    constexpr int kSteps = kRouteChunk / 32;
    const int lane = threadIdx.x;
    const int base = blockIdx.x * kRouteChunk;
    const int end = min(R, base + kRouteChunk);
    int my_ids[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int p = base + i * 32 + lane;
        my_ids[i] = p < end ? ids[p] : -1;
    }
    for (int e = lane; e < E; e += 32)
        cursor[e] = chunk_base[static_cast<long long>(blockIdx.x) * E + e];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int p = base + i * 32 + lane;
        if (base + i * 32 >= end) break;
        const bool live = p < end;
        const int e = my_ids[i];
        const bool ok = live && e >= 0 && e < E;
        const unsigned peers = same_value_lanes(e, ok, value_bits(E));
        const int rank = __popc(peers & ((1u << lane) - 1u));
        const int first = cursor[ok ? e : 0];
        __syncwarp();
        if (ok) {
            const int row = first + rank;
            perm[row] = p;
            if (inv_perm) inv_perm[p] = row;
            if (rank == 0) cursor[e] = first + __popc(peers);
        } else if (live && inv_perm) {
            inv_perm[p] = -1;
        }
        __syncwarp();
    }
}

// Small inputs (at most kSmallChunks chunks of 1024 pairs): the same three
// phases in one CTA of 1024 threads, so routing costs one launch.  The pairs
// are cut into up to 32 consecutive blocks, one per warp (as many as keep the
// per-block histograms within the default shared-memory limit), so the
// serial ranking steps of phase 3 are spread over the warps.  Phase 2 scans
// each expert's column of block counts with one warp (lane = block; rows of
// the table padded to E + 1 ints so a column read is conflict-free), then
// the experts' totals with one thread per expert.
constexpr int kSmallChunks = 8;
// 43 KB of table; with the static per-expert totals (4 KB) within 48 KB
constexpr int kSmallTabInts = 11008;

__host__ __device__ constexpr int small_route_warps(int E) {
    return (E + 1) * 32 <= kSmallTabInts ? 32 : kSmallTabInts / (E + 1);
}
static_assert(small_route_warps(kMaxRouteExperts) >= kSmallChunks,
              "route_small's pair blocks must stay within kRouteChunk pairs");

// Dynamic shared memory of route_small: the table, then the R entries of
// perm, which phase 3 writes in shared memory (scattered) and the CTA then
// copies out in order: scattered 4-byte global stores from one SM go out at
// about one sector per clock (4096 of them cost ~4 µs).
__host__ __device__ inline size_t small_route_smem(int R, int E) {
    return (static_cast<size_t>(small_route_warps(E)) * (E + 1) + R) * sizeof(int);
}
constexpr size_t kSmallRouteSmemMax = (kSmallTabInts + kSmallChunks * kRouteChunk) * sizeof(int);

// The three phases of route_small for a CTA of 1024 threads; tab is
// [small_route_warps(E)][E + 1] ints of shared memory followed by R ints.
__device__ __forceinline__ void route_small_body(const int32_t* __restrict__ ids, int R, int E,
                                                 int32_t* __restrict__ m_indptr,
                                                 int32_t* __restrict__ perm,
                                                 int32_t* __restrict__ inv_perm, int* status,
                                                 int* tab, bool clear_status) {
    __shared__ int warp_tot[32];
    __shared__ int cnt_s[kMaxRouteExperts];   // per-expert totals, then first rows
    __shared__ int valid_s;                   // pairs with a valid expert id
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int W = small_route_warps(E);
    const int Ep = E + 1;
    int* perm_s = tab + W * Ep;               // [R]: perm, staged
    // pairs per block: a multiple of 32, at most kRouteChunk (R <= 8 chunks, W >= 8)
    const int B = ((R + W - 1) / W + 31) & ~31;
    const int nchunks = B > 0 ? (R + B - 1) / B : 0;
    constexpr int kSteps = kRouteChunk / 32;
    // the caller's status words start clean before any error is reported
    if (clear_status && threadIdx.x < kStatusInts) status[threadIdx.x] = 0;
    for (int i = threadIdx.x; i < nchunks * Ep; i += blockDim.x) tab[i] = 0;
    __syncthreads();
    // phase 1: per-block histograms
    int my_ids[kSteps];
    const int base = warp * B;
    if (warp < nchunks) {
        const int end = min(R, base + B);
        int bad = 0;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int p = base + i * 32 + lane;
            my_ids[i] = p < end ? ids[p] : -1;
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int p = base + i * 32 + lane;
            if (p < end) {
                const int e = my_ids[i];
                if (e >= 0 && e < E) atomicAdd(&tab[warp * Ep + e], 1);
                else ++bad;
            }
        }
        if (bad) {
            atomicAdd(&status[2], bad);
            report_error(status, ST_BAD_EXPERT_ID, 0);
        }
    }
    __syncthreads();
    // phase 2a: per expert, exclusive scan over the blocks (warp per expert, lane = block)
    for (int ex = warp; ex < E; ex += 32) {
        const int h = lane < nchunks ? tab[lane * Ep + ex] : 0;
        int run = h;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += v;
        }
        if (lane < nchunks) tab[lane * Ep + ex] = run - h;
        if (lane == 31) cnt_s[ex] = run;
    }
    __syncthreads();
    // phase 2b: exclusive scan over the experts' totals (thread e)
    const int e = threadIdx.x;
    const int count = e < E ? cnt_s[e] : 0;
    int incl = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int t = warp_tot[lane];
        int ti = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, ti, o);
            if (lane >= o) ti += v;
        }
        warp_tot[lane] = ti - t;
    }
    __syncthreads();
    const int excl = warp_tot[warp] + incl - count;
    if (e < E) {
        m_indptr[e] = excl;
        cnt_s[e] = excl;   // only thread e read cnt_s[e] above
    }
    if (e == E - 1) {
        m_indptr[E] = excl + count;
        valid_s = excl + count;
    }
    __syncthreads();
    // phase 2c: first output row of every (block, expert)
    for (int ex = warp; ex < E; ex += 32)
        if (lane < nchunks) tab[lane * Ep + ex] += cnt_s[ex];
    __syncthreads();
    // phase 3: stable scatter, 32 pairs at a time per block
    const int nbits = value_bits(E);
    if (warp < nchunks) {
        const int end = min(R, base + B);
        int* cursor = tab + warp * Ep;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int p = base + i * 32 + lane;
            if (base + i * 32 >= end) break;
            const bool live = p < end;
            const int ex = my_ids[i];
            const bool ok = live && ex >= 0 && ex < E;
            const unsigned peers = same_value_lanes(ex, ok, nbits);
            const int rank = __popc(peers & ((1u << lane) - 1u));
            const int first = cursor[ok ? ex : 0];
            __syncwarp();
            if (ok) {
                const int row = first + rank;
                perm_s[row] = p;
                if (inv_perm) inv_perm[p] = row;
                if (rank == 0) cursor[ex] = first + __popc(peers);
            } else if (live && inv_perm) {
                inv_perm[p] = -1;
            }
            __syncwarp();
        }
    }
    __syncthreads();
    // perm out in order (rows of dropped pairs do not exist: only [0, valid) is written)
    const int valid = valid_s;
    for (int i = threadIdx.x; i < valid; i += blockDim.x) perm[i] = perm_s[i];
}

__global__ void __launch_bounds__(1024) route_small(const int32_t* __restrict__ ids, int R, int E,
                                                    int32_t* __restrict__ m_indptr,
                                                    int32_t* __restrict__ perm,
                                                    int32_t* __restrict__ inv_perm, int* status,
                                                    int clear_status) {
    extern __shared__ int tab[];  // [blocks][E + 1]: histograms, then first rows
    route_small_body(ids, R, E, m_indptr, perm, inv_perm, status, tab, clear_status != 0);
}

// Router (the step before the expert computation): one warp per token.
// Lane l holds logits l + 32 i; the k winners are taken one at a time by a
// warp-wide argmax (larger logit first, then the lower expert index), so the
// ids come out in descending logit order.  Lane j keeps the j-th winner's
// logit; the softmax subtracts the largest, takes expf per slot and sums the
// slots in order (every lane runs the same sequential sum), w_j = e_j / sum.
template <int PER>
__device__ __forceinline__ void router_token(const float* __restrict__ logits, int t, int E, int k,
                                             int32_t* __restrict__ ids, float* __restrict__ w) {
    const int lane = threadIdx.x & 31;
    const float* l = logits + static_cast<long long>(t) * E;
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        v[i] = e < E ? l[e] : 0.0f;
    }
    uint32_t taken = 0;
    float mine = 0.0f;  // logit of slot `lane`
    for (int j = 0; j < k; ++j) {
        float bv = 0.0f;
        int be = E;  // E = none
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            if (e < E && !((taken >> i) & 1u) && (be == E || v[i] > bv)) {
                bv = v[i];
                be = e;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oe = __shfl_xor_sync(0xffffffffu, be, o);
            if (oe != E && (be == E || ov > bv || (ov == bv && oe < be))) {
                bv = ov;
                be = oe;
            }
        }
        if (lane == (be & 31)) taken |= 1u << (be >> 5);
        if (lane == j) mine = bv;
        if (lane == 0) ids[static_cast<long long>(t) * k + j] = be;
    }
    const float m = __shfl_sync(0xffffffffu, mine, 0);
    const float ex = lane < k ? expf(mine - m) : 0.0f;
    float sum = 0.0f;
    for (int j = 0; j < k; ++j) sum += __shfl_sync(0xffffffffu, ex, j);
    if (lane < k) w[static_cast<long long>(t) * k + lane] = __fdiv_rn(ex, sum);
}

template <int PER>
__global__ void __launch_bounds__(256) router_topk_kernel(const float* __restrict__ logits, int T,
                                                          int E, int k, int32_t* __restrict__ ids,
                                                          float* __restrict__ w) {
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= T) return;
    router_token<PER>(logits, t, E, k, ids, w);
}

// Router and routing in one CTA of 1024 threads, for at most kSmallChunks
// chunks of pairs: each warp routes tokens warp, warp + 32, ..., then the
// CTA groups the pairs it just wrote (global writes made visible to the
// whole CTA by the barrier) with route_small's three phases.
template <int PER>
__global__ void __launch_bounds__(1024) router_route_small(const float* __restrict__ logits, int T,
                                                           int E, int k, int32_t* __restrict__ ids,
                                                           float* __restrict__ w,
                                                           int32_t* __restrict__ m_indptr,
                                                           int32_t* __restrict__ perm,
                                                           int32_t* __restrict__ inv_perm,
                                                           int* status) {
    extern __shared__ int tab[];
    for (int t = threadIdx.x >> 5; t < T; t += 32) router_token<PER>(logits, t, E, k, ids, w);
    __syncthreads();
    route_small_body(ids, T * k, E, m_indptr, perm, inv_perm, status, tab, false);
}

int launch_router_topk(const float* logits, int T, int E, int k, int32_t* ids, float* w,
                       cudaStream_t stream) {
    if (T == 0) return ST_OK;
    const unsigned blocks = static_cast<unsigned>((T + 7) / 8);
    if (E <= 256)
        router_topk_kernel<8><<<blocks, 256, 0, stream>>>(logits, T, E, k, ids, w);
    else
        router_topk_kernel<32><<<blocks, 256, 0, stream>>>(logits, T, E, k, ids, w);
    return cudaGetLastError() == cudaSuccess ? ST_OK : ST_CUDA;
}

// Opt-in of the single-CTA routing kernels to kSmallRouteSmemMax bytes of
// dynamic shared memory, once per device.
bool small_route_smem_ready() {
    static std::atomic<int> ready_dev{-1};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (ready_dev.load() == dev) return true;
    const int n = static_cast<int>(kSmallRouteSmemMax);
    if (cudaFuncSetAttribute(route_small, cudaFuncAttributeMaxDynamicSharedMemorySize, n) != cudaSuccess ||
        cudaFuncSetAttribute(router_route_small<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, n) !=
            cudaSuccess ||
        cudaFuncSetAttribute(router_route_small<32>, cudaFuncAttributeMaxDynamicSharedMemorySize, n) !=
            cudaSuccess)
        return false;
    ready_dev.store(dev);
    return true;
}

int launch_router_route(const float* logits, const RouteArgs& r, float* w, cudaStream_t stream) {
    const int R = r.T * r.k;
    if (R == 0) return launch_route_permute(r, stream);
    const int nchunks = (R + kRouteChunk - 1) / kRouteChunk;
    if (nchunks <= kSmallChunks) {
        int32_t* ids = const_cast<int32_t*>(r.topk_ids);
        const size_t smem = small_route_smem(R, r.E);
        if (!small_route_smem_ready()) return ST_CUDA;
        if (r.E <= 256)
            router_route_small<8><<<1, 1024, smem, stream>>>(logits, r.T, r.E, r.k, ids, w,
                                                             r.m_indptr, r.perm, r.inv_perm, r.status);
        else
            router_route_small<32><<<1, 1024, smem, stream>>>(logits, r.T, r.E, r.k, ids, w,
                                                              r.m_indptr, r.perm, r.inv_perm, r.status);
        return cudaGetLastError() == cudaSuccess ? ST_OK : ST_CUDA;
    }
    int st = launch_router_topk(logits, r.T, r.E, r.k, const_cast<int32_t*>(r.topk_ids), w, stream);
    if (st) return st;
    return launch_route_permute(r, stream);
}

bool route_single_launch(int R) { return (R + kRouteChunk - 1) / kRouteChunk <= kSmallChunks; }

int launch_route_permute(const RouteArgs& r, cudaStream_t stream) {
    const int R = r.T * r.k;
    const int nchunks = (R + kRouteChunk - 1) / kRouteChunk;
    const size_t hist_smem = static_cast<size_t>(r.E) * sizeof(int);
    if (nchunks <= kSmallChunks) {
        const size_t smem = small_route_smem(R, r.E);
        if (!small_route_smem_ready()) return ST_CUDA;
        route_small<<<1, 1024, smem, stream>>>(r.topk_ids, R, r.E, r.m_indptr, r.perm, r.inv_perm,
                                               r.status, r.clear_status);
        return cudaGetLastError() == cudaSuccess ? ST_OK : ST_CUDA;
    }
    {
        route_hist<<<nchunks, 256, hist_smem, stream>>>(r.topk_ids, R, r.E, r.chunk_hist, r.status);
        if (cudaGetLastError() != cudaSuccess) return ST_CUDA;
    }
    route_scan<<<1, 1024, 0, stream>>>(nchunks, r.E, r.chunk_hist, r.m_indptr);
    if (cudaGetLastError() != cudaSuccess) return ST_CUDA;
    if (nchunks > 0) {
        route_scatter<<<nchunks, 32, hist_smem, stream>>>(r.topk_ids, R, r.E, r.chunk_hist, r.perm,
                                                          r.inv_perm);
        if (cudaGetLastError() != cudaSuccess) return ST_CUDA;
    }
    return ST_OK;
}

// ------------------------------------------------------------ scored router
// Expert choice by scores (launch_router_score).  For token t, with x the
// logits and b the bias:
//   p_e = 1 / (1 + exp(-x_e)) or softmax(x)_e;  c_e = p_e + b_e (the order of
//   x without a bias);  group g = E / n_group consecutive experts, G_g = the
//   sum of its group_top (1 or 2) largest c;  candidates: the topk_group
//   groups with the largest G;  ids: the k largest c among them, descending,
//   ties to the lower index;  w_j = p_j (/ sum p) * scale.
// Masked experts (logit NaN or at most its type's lowest value, bias NaN or at
// most -FLT_MAX) rank after every other, by index, and get weight 0.
//
// One warp per token, lane l holding experts l + 32 i.  The choice is that of
// 64-bit values at 32-bit speed: c is computed in fp32, whose error is bounded
// (score_tol), and only a token with two neighbouring values closer than the
// bound (among its k winners, at the k / k + 1 border, or at the border
// between chosen and dropped groups) is decided again with 64-bit scores.
// Each winner costs one warp-wide integer maximum over order-preserving keys
// of the values (a reduction instruction, where a shuffle tree of (value,
// index) pairs takes ten shuffles and as many selects).

constexpr float kFltMax = 3.402823466e38f;
constexpr float kBf16Lowest = -3.38953138925153547590e38f;

__device__ __forceinline__ float ld_logit(const float* l, int e) { return l[e]; }
__device__ __forceinline__ float ld_logit(const __nv_bfloat16* l, int e) {
    return __bfloat162float(l[e]);
}
__device__ __forceinline__ bool logit_masked(const float*, float x) { return !(x > -kFltMax); }
__device__ __forceinline__ bool logit_masked(const __nv_bfloat16*, float x) {
    return !(x > kBf16Lowest);
}

// Order-preserving map of finite floats to [0x00800000, 0xff7fffff]; 1 is a
// masked expert, 0 no candidate.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);  // -0 and +0 compare equal
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// Bound on |difference of two fp32 selection values - the exact difference|.
// Scores use the hardware exponential, whose relative error is (2 + 1.17 |z|)
// ulp at argument z, and the correctly rounded reciprocal.
//  sigmoid + b: p (1 - p) (2 + 1.17 |x|) + 2 ulps <= 3 * 2^-24 per score, plus
//    one rounding of the sum; four scores in a difference of group sums: 2^-19
//    and 2^-21 of the values' size.
//  softmax + b: the 37-term sum's relative error 40 * 2^-24 times p, and sum
//    p <= 1: 2^-17, the same relative part.
//  no bias (group sums of scores alone): relative only; |z| <= 88 before the
//    exponential leaves fp32's normal range: (2 + 2.2 * 88 + 40) 2^-24 < 2^-15.
__device__ __forceinline__ float score_tol(const ScoreArgs& a, float v) {
    const float m = fabsf(v);
    if (!a.bias) return 3.0517578125e-05f * m;
    return (a.sigmoid ? 1.9073486328125e-06f : 7.62939453125e-06f) + 4.76837158203125e-07f * m;
}

// The choice with 64-bit scores; lane j < k returns the j-th expert.
template <int PER, typename LT>
__device__ __noinline__ int score_choose_f64(const ScoreArgs& a, const LT* l) {
    const int lane = threadIdx.x & 31;
    const int gs = a.E / a.n_group;
    const double none = -__longlong_as_double(0x7ff0000000000000ll);
    double mx = none, z = 0.0;
    if (!a.sigmoid) {
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            if (e >= a.E) break;
            const float x = ld_logit(l, e);
            const bool m = logit_masked(l, x) || (a.bias && !(a.bias[e] > -kFltMax));
            if (!m) mx = fmax(mx, static_cast<double>(fminf(x, kFltMax)));
        }
        for (int o = 16; o > 0; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            if (e >= a.E) break;
            const float x = ld_logit(l, e);
            const bool m = logit_masked(l, x) || (a.bias && !(a.bias[e] > -kFltMax));
            if (!m) z += exp(static_cast<double>(fminf(x, kFltMax)) - mx);
        }
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    // c: value the experts are ordered by; p: value that group sums add up
    double c[PER], p[PER];
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        c[i] = p[i] = none;
        if (e >= a.E) continue;
        float x = ld_logit(l, e);
        if (logit_masked(l, x) || (a.bias && !(a.bias[e] > -kFltMax))) continue;
        x = fminf(x, kFltMax);
        const double s = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(x)))
                                   : exp(static_cast<double>(x) - mx) / z;
        c[i] = a.bias ? s + static_cast<double>(fminf(a.bias[e], kFltMax)) : static_cast<double>(x);
        p[i] = a.bias || a.group_top == 1 ? c[i] : s;
    }
    uint32_t groups = 1u;
    if (a.n_group > 1) {
        double mine = none;  // lane g: group g's value
        for (int g = 0; g < a.n_group; ++g) {
            double t1 = none, t2 = none;
            for (int i = 0; i < PER; ++i) {
                const int e = lane + 32 * i;
                if (e < g * gs || e >= (g + 1) * gs) continue;
                t2 = fmax(t2, fmin(t1, p[i]));
                t1 = fmax(t1, p[i]);
            }
            for (int o = 16; o > 0; o >>= 1) {
                const double u1 = __shfl_xor_sync(0xffffffffu, t1, o);
                const double u2 = __shfl_xor_sync(0xffffffffu, t2, o);
                t2 = fmax(fmin(t1, u1), fmax(t2, u2));
                t1 = fmax(t1, u1);
            }
            const double v = a.group_top == 2 && t2 != none ? t1 + t2 : t1;
            if (lane == g) mine = v;
        }
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const double v = __shfl_sync(0xffffffffu, mine, g);
            rank += v > mine || (v == mine && g < lane) ? 1 : 0;
        }
        groups = __ballot_sync(0xffffffffu, lane < a.n_group && rank < a.topk_group);
    }
    uint32_t gone = 0;
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        if (e >= a.E || !((groups >> (e / gs)) & 1u)) gone |= 1u << i;
    }
    int chosen = 0;
    for (int j = 0; j < a.k; ++j) {
        double bv = none;
        int be = 0x7fffffff;  // none
        for (int i = 0; i < PER; ++i) {
            if ((gone >> i) & 1u) continue;
            if (be == 0x7fffffff || c[i] > bv) {
                bv = c[i];
                be = lane + 32 * i;
            }
        }
        for (int o = 16; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oe = __shfl_xor_sync(0xffffffffu, be, o);
            if (oe != 0x7fffffff && (be == 0x7fffffff || ov > bv || (ov == bv && oe < be))) {
                bv = ov;
                be = oe;
            }
        }
        if (lane == (be & 31)) gone |= 1u << (be >> 5);
        if (lane == j) chosen = be;
    }
    return chosen;
}

// One token.  scratch: E floats of this warp's shared memory (groups only).
template <int PER, typename LT>
__device__ __forceinline__ void router_score_token(const ScoreArgs& a, int t, float* scratch) {
    const int lane = threadIdx.x & 31;
    const LT* l = static_cast<const LT*>(a.logits) + static_cast<long long>(t) * a.E;
    const bool sums = a.n_group > 1 && a.group_top == 2;   // group values add scores up
    const bool need_score = a.bias != nullptr || sums;
    const bool need_z = !a.sigmoid && (need_score || !a.renorm);
    float v[PER];                  // logits, then the selection values
    uint32_t masked = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        v[i] = e < a.E ? ld_logit(l, e) : -kFltMax;
    }
    uint32_t mkey = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        const bool m = e >= a.E || logit_masked(l, v[i]) || (a.bias && !(a.bias[e] > -kFltMax));
        v[i] = fminf(v[i], kFltMax);
        masked |= (m ? 1u : 0u) << i;
        if (!m) mkey = max(mkey, order_key(v[i]));
    }
    float mx = 0.0f, zinv = 0.0f;
    if (need_z) {
        mkey = __reduce_max_sync(0xffffffffu, mkey);
        mx = mkey ? key_value(mkey) : 0.0f;
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (!((masked >> i) & 1u)) z += __expf(v[i] - mx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        zinv = z > 0.0f ? __frcp_rn(z) : 0.0f;
    }
    const int gs = a.E / a.n_group;
    bool ambiguous = false;
    uint32_t groups = 1u;
    if (need_score || a.n_group > 1) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E) {
                float g = v[i];
                if (need_score) {
                    const float s = a.sigmoid ? __frcp_rn(1.0f + __expf(-v[i]))
                                              : __expf(v[i] - mx) * zinv;
                    if (a.bias) v[i] = s + fminf(a.bias[e], kFltMax);
                    g = a.bias || !sums ? v[i] : s;
                }
                if (a.n_group > 1) scratch[e] = (masked >> i) & 1u ? -INFINITY : g;
            }
        }
    }
    if (a.n_group > 1) {
        // P lanes scan a group together (P * n_group <= 32), then merge
        __syncwarp();
        int lg = 0;
        while ((1 << lg) < a.n_group) ++lg;
        const int P = 32 >> lg;
        const int g = lane >> (5 - lg), sub = lane & (P - 1);
        float t1 = -INFINITY, t2 = -INFINITY;
        if (g < a.n_group)
            for (int i = sub; i < gs; i += P) {
                const float f = scratch[g * gs + i];
                t2 = fmaxf(t2, fminf(t1, f));
                t1 = fmaxf(t1, f);
            }
        for (int o = P >> 1; o > 0; o >>= 1) {
            const float u1 = __shfl_xor_sync(0xffffffffu, t1, o);
            const float u2 = __shfl_xor_sync(0xffffffffu, t2, o);
            t2 = fmaxf(fminf(t1, u1), fmaxf(t2, u2));
            t1 = fmaxf(t1, u1);
        }
        float gv = a.group_top == 2 && t2 > -INFINITY ? t1 + t2 : t1;
        gv = __shfl_sync(0xffffffffu, gv, (lane << (5 - lg)) & 31);  // lane g: group g's value
        int rank = 0;
        for (int o = 0; o < a.n_group; ++o) {
            const float ov = __shfl_sync(0xffffffffu, gv, o);
            rank += ov > gv || (ov == gv && o < lane) ? 1 : 0;
        }
        const bool in = lane < a.n_group && rank < a.topk_group;
        groups = __ballot_sync(0xffffffffu, in);
        if (need_score && a.topk_group < a.n_group) {
            const bool live = lane < a.n_group && gv > -INFINITY;
            const uint32_t lo = __reduce_min_sync(0xffffffffu, in && live ? order_key(gv) : 0xffffffffu);
            const uint32_t hi = __reduce_max_sync(0xffffffffu, !in && live ? order_key(gv) : 0u);
            if (lo != 0xffffffffu && hi != 0u) {
                const float fl = key_value(lo), fh = key_value(hi);
                ambiguous = !(fl - fh > fmaxf(score_tol(a, fl), score_tol(a, fh)));
            }
        }
        __syncwarp();
    }
    // keys of the candidates, and the lane's best
    uint32_t key[PER];
    const uint32_t inv_gs = ((1u << 20) + gs - 1) / gs;  // e / gs = e * inv_gs >> 20 for e, gs <= 1024
    uint32_t bk = 0;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        const bool cand = e < a.E && (a.n_group == 1 || ((groups >> ((e * inv_gs) >> 20)) & 1u));
        key[i] = !cand ? 0u : (masked >> i) & 1u ? 1u : order_key(v[i]);
        if (key[i] > bk) {
            bk = key[i];
            be = e;
        }
    }
    // one winner more than wanted where the k / k + 1 border has to be checked
    const int rounds = a.bias && a.k < a.topk_group * gs ? a.k + 1 : a.k;
    int mine = 0;
    uint32_t mine_key = 0, next_key = 0;  // next_key: of the winner after this lane's
    for (int j = 0; j < rounds; ++j) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
        const uint32_t who = __ballot_sync(0xffffffffu, bk == top);
        const int e = (who & (who - 1)) == 0
                          ? __shfl_sync(0xffffffffu, be, __ffs(who) - 1)
                          : static_cast<int>(__reduce_min_sync(0xffffffffu, bk == top ? be : 0x7fffffff));
        if (lane == j) {
            mine = e;
            mine_key = top;
        }
        if (lane == j - 1) next_key = top;
        if (lane == (e & 31)) {
            bk = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (lane + 32 * i == e) key[i] = 0;
                if (key[i] > bk) {
                    bk = key[i];
                    be = lane + 32 * i;
                }
            }
        }
    }
    if (a.bias && !ambiguous) {
        bool close = false;
        if (lane < rounds - 1 && next_key > 1u) {
            const float f0 = key_value(mine_key), f1 = key_value(next_key);
            close = !(f0 - f1 > fmaxf(score_tol(a, f0), score_tol(a, f1)));
        }
        if (__any_sync(0xffffffffu, close)) {
            // equal logits with equal biases tie exactly: their order is by index
            // (not at the k / k + 1 border, behind which more may be close)
            const int other = __shfl_down_sync(0xffffffffu, mine, 1);
            if (close && lane + 1 < a.k)
                close = !(ld_logit(l, mine) == ld_logit(l, other) && a.bias[mine] == a.bias[other]);
            ambiguous = __any_sync(0xffffffffu, close);
        }
    }
    if (ambiguous) mine = score_choose_f64<PER, LT>(a, l);
    // weights of the k winners, lane j = slot j
    const bool slot = lane < a.k;
    float x = -kFltMax;
    bool off = true;
    if (slot) {
        x = ld_logit(l, mine);
        off = logit_masked(l, x) || (a.bias && !(a.bias[mine] > -kFltMax));
        x = fminf(x, kFltMax);
    }
    float u = 0.0f;
    if (a.renorm) {
        // scaled by the largest so that no row of small scores underflows
        const uint32_t xk = __reduce_max_sync(0xffffffffu, off ? 0u : order_key(x));
        float m = xk ? key_value(xk) : 0.0f;
        if (a.sigmoid) m = fminf(m, 0.0f);
        if (!off)
            u = !a.sigmoid ? expf(x - m) : x > 0.0f ? 1.0f / (1.0f + expf(-x))
                                                    : expf(x - m) / (1.0f + expf(x));
        float sum = u;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        u = sum > 0.0f ? __fdiv_rn(u, sum) : 0.0f;
    } else if (!off) {
        u = !a.sigmoid ? expf(x - mx) * zinv : x > 0.0f ? 1.0f / (1.0f + expf(-x))
                                                        : expf(x) / (1.0f + expf(x));
    }
    if (slot) {
        a.ids[static_cast<long long>(t) * a.k + lane] = mine;
        a.w[static_cast<long long>(t) * a.k + lane] = u * a.scale;
    }
}

template <int PER, typename LT>
__global__ void __launch_bounds__(128) router_score_kernel(const ScoreArgs a) {
    extern __shared__ float group_scratch[];
    const int warp = threadIdx.x >> 5;
    const int t = blockIdx.x * 4 + warp;
    if (t >= a.T) return;
    router_score_token<PER, LT>(a, t, group_scratch + warp * a.E);
}

// Scored router and grouping in one CTA, for few tokens: the warps' group
// scratch and the grouping's table share the dynamic memory.
template <int PER, typename LT>
__global__ void __launch_bounds__(1024) router_score_route_small(const ScoreArgs a,
                                                                 int32_t* __restrict__ m_indptr,
                                                                 int32_t* __restrict__ perm,
                                                                 int32_t* __restrict__ inv_perm,
                                                                 int* status) {
    extern __shared__ int tab[];
    for (int t = threadIdx.x >> 5; t < a.T; t += 32)
        router_score_token<PER, LT>(a, t, reinterpret_cast<float*>(tab) + (threadIdx.x >> 5) * a.E);
    __syncthreads();
    route_small_body(a.ids, a.T * a.k, a.E, m_indptr, perm, inv_perm, status, tab, true);
}

template <typename LT>
int launch_score_t(const ScoreArgs& a, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>((a.T + 3) / 4);
    const size_t smem = a.n_group > 1 ? 4ull * a.E * sizeof(float) : 0;
    if (a.E <= 128) router_score_kernel<4, LT><<<grid, 128, smem, s>>>(a);
    else if (a.E <= 256) router_score_kernel<8, LT><<<grid, 128, smem, s>>>(a);
    else if (a.E <= 512) router_score_kernel<16, LT><<<grid, 128, smem, s>>>(a);
    else router_score_kernel<32, LT><<<grid, 128, smem, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? ST_OK : ST_CUDA;
}

int launch_router_score(const ScoreArgs& a, cudaStream_t s) {
    if (a.T == 0) return ST_OK;
    return a.bf16 ? launch_score_t<__nv_bfloat16>(a, s) : launch_score_t<float>(a, s);
}

template <int PER, typename LT>
int launch_score_route_inst(const ScoreArgs& a, const RouteArgs& r, cudaStream_t s) {
    size_t smem = small_route_smem(a.T * a.k, a.E);
    if (a.n_group > 1) smem = std::max<size_t>(smem, 32ull * a.E * sizeof(float));
    // opt-in once per device and kernel; a second device just sets it again
    static std::atomic<int> ready_dev{-1};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ST_CUDA;
    if (ready_dev.load() != dev) {
        const int most = static_cast<int>(std::max<size_t>(kSmallRouteSmemMax, 32ull * 32 * PER * sizeof(float)));
        if (cudaFuncSetAttribute(router_score_route_small<PER, LT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
            return ST_CUDA;
        ready_dev.store(dev);
    }
    router_score_route_small<PER, LT><<<1, 1024, smem, s>>>(a, r.m_indptr, r.perm, r.inv_perm, r.status);
    return cudaGetLastError() == cudaSuccess ? ST_OK : ST_CUDA;
}

template <typename LT>
int launch_score_route_t(const ScoreArgs& a, const RouteArgs& r, cudaStream_t s) {
    if (a.E <= 128) return launch_score_route_inst<4, LT>(a, r, s);
    if (a.E <= 256) return launch_score_route_inst<8, LT>(a, r, s);
    if (a.E <= 512) return launch_score_route_inst<16, LT>(a, r, s);
    return launch_score_route_inst<32, LT>(a, r, s);
}

// One launch for few tokens: a token costs its warp of the one CTA about as
// much as a sixteenth of the launch it saves.
constexpr int kScoreRouteTokens = 128;

int launch_router_score_route(const ScoreArgs& a, const RouteArgs& r, cudaStream_t s) {
    const int R = a.T * a.k;
    if (a.T > 0 && a.T <= kScoreRouteTokens && route_single_launch(R))
        return a.bf16 ? launch_score_route_t<__nv_bfloat16>(a, r, s) : launch_score_route_t<float>(a, r, s);
    RouteArgs rr = r;
    rr.clear_status = 1;
    if (!route_single_launch(R) &&
        cudaMemsetAsync(r.status, 0, sizeof(int) * kStatusInts, s) != cudaSuccess)
        return ST_CUDA;
    if (int st = launch_router_score(a, s)) return st;
    return launch_route_permute(rr, s);
}

}  // namespace moe
