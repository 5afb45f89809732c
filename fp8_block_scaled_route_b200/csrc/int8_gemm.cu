// Grouped int8 GEMM with a scale per row and per output channel.
//
//   S[r, n] = sum_k a[r, k] * b[e, n, k]          (exact, 32-bit integers)
//   G[r, n] = (float(S) * a_scale[r]) * b_scale[e, n]
//   out     = G, or gated silu(G[:, :N/2]) * G[:, N/2:], rounded once
// for rows r of expert e ([m_indptr[e], m_indptr[e+1])).  tcgen05.mma kind::i8
// sums the whole K range in tensor memory, so no scale is applied inside the
// main loop and integer partial sums of a split K range add up exactly in any
// order.
//
// Orientation: the weights are the MMA's M operand (128 tensor-memory lanes =
// 128 weight rows), the token rows its N operand, whose size is an argument
// of the instruction: an expert with 5 rows costs an N = 16 MMA and a 16-row
// load.  A warp's 32 lanes are 32 consecutive output channels of one token
// row, so plain stores are whole 32-byte sectors without a transpose.  Gated:
// the 128 lanes are granules of 16 gate rows and the 16 up rows that belong to
// them, so lanes l and l + 16 of a warp hold one output's two halves.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "gemm_common.cuh"
#include "kernels.h"
#include "ptx_cluster.cuh"

namespace moe {

namespace {

constexpr int kKB = 128;             // K bytes per stage
constexpr int kWRows = 128;          // weight rows per CTA tile
constexpr int kWBytes = kWRows * kKB;
constexpr int kGran = 16;            // gate / up rows of a granule
constexpr int kWBox = 128;           // weight rows per TMA box
constexpr int MAX_E = kMaxRouteExperts;
constexpr int kMaxSplit = 8;         // CTAs of a cluster that share a K range

struct I8Params {
    const float* a_scale;
    const float* b_scale;
    const int32_t* m_indptr;
    void* out;
    int R, N, E, nkb;
    int wtiles;   // narrow kernel: weight tiles of an expert
    int bt;       // pair kernel: token rows of a tile (64, 128 or 256)
    int nst;      // pair kernel: stages
    int w_gran;   // gated with N / 2 not a multiple of 16: weight boxes of one half granule
    int* status;
    unsigned long long timeout_ns;
};

// Rows of expert e, clamped to [0, R].
__device__ __forceinline__ void expert_rows(const I8Params& p, int e, int& lo, int& hi) {
    lo = 0;
    hi = p.R;
    if (p.m_indptr) {
        lo = min(max(p.m_indptr[e], 0), p.R);
        hi = min(max(p.m_indptr[e + 1], lo), p.R);
    }
}

template <bool BF16>
__device__ __forceinline__ void store_out(const I8Params& p, long long at, float v) {
    if constexpr (BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(v);
    else static_cast<float*>(p.out)[at] = v;
}
// Two neighbouring outputs, `at` even.
template <bool BF16>
__device__ __forceinline__ void store_out2(const I8Params& p, long long at, float a, float b) {
    if constexpr (BF16)
        reinterpret_cast<__nv_bfloat162*>(p.out)[at >> 1] = __floats2bfloat162_rn(a, b);
    else
        reinterpret_cast<float2*>(p.out)[at >> 1] = make_float2(a, b);
}

// A lane's NW output pairs of rows `rows` apart: pair i at element `at` + i *
// pitch, stored while its row i * rows is below lim.
template <bool BF16, int NW>
__device__ __forceinline__ void store_rows(const I8Params& p, const float2 (&v)[NW], long long at,
                                           long long pitch, int rows, int lim) {
    if (lim >= rows * (NW - 1) + 1) {
#pragma unroll
        for (int i = 0; i < NW; ++i) store_out2<BF16>(p, at + i * pitch, v[i].x, v[i].y);
    } else {
#pragma unroll
        for (int i = 0; i < NW; ++i)
            if (i * rows < lim) store_out2<BF16>(p, at + i * pitch, v[i].x, v[i].y);
    }
}

// What a lane of the epilogue keeps for one weight tile: its weight row's
// output column and scale.
struct LaneCol {
    int col;      // output column (gated: channel)
    float scale;  // b_scale of the lane's weight row, 0 past the end
    bool ok;
};

template <bool GATED>
__device__ __forceinline__ LaneCol lane_col(const I8Params& p, int e, int wt, int pos) {
    LaneCol c;
    const float* bs = p.b_scale + static_cast<long long>(e) * p.N;
    if constexpr (!GATED) {
        c.col = wt * kWRows + pos;
        c.ok = c.col < p.N;
        c.scale = c.ok ? bs[c.col] : 0.0f;
    } else {
        const int half = p.N >> 1;
        c.col = wt * (kWRows / 2) + (pos >> 5) * kGran + (pos & 15);
        c.ok = c.col < half;
        c.scale = c.ok ? bs[((pos & 16) ? half : 0) + c.col] : 0.0f;
    }
    return c;
}

// A warp copies the scales of n <= 128 token rows from row0 on into its own
// shared-memory buffer; rows at or past hi count as 0.
__device__ __forceinline__ void stage_row_scales(const I8Params& p, float* as, int row0, int n, int hi) {
    __syncwarp();
    for (int i = threadIdx.x & 31; i < n; i += 32) as[i] = row0 + i < hi ? p.a_scale[row0 + i] : 0.0f;
    __syncwarp();
}

// SiLU for an output that is kept in fp32: z e / (1 + e) or z / (1 + e) with
// e = exp(-|z|) = 2^h (1 + c), h = fp32(-|z| log2 e) and c = -|z| - h ln 2, what h's
// rounding left out (one fused multiply-add; the second order, below 2^-34, does
// not count).  silu_fast leaves c out and is off by 2 + 1.17 |z| ulps, which only
// a rounding to bf16 or FP8 hides.  Here, in units of 2^-24: 2^h 4, 1 + c 1, ln 2's
// own rounding 0.05 |z|, 1 + e 1, reciprocal 2, products 2.  8192 x 4096 x 2048 with
// fp32 output: 53.4 us with silu_fast, 55.4 with this, 77 with expf and a division.
__device__ __forceinline__ float silu_f32(float z) {
    const float a = fminf(fabsf(z), 110.0f);   // e is 0 from 104 on; an infinite h would make c NaN
    const float h = a * -1.442695041f;
    const float p = ex2_approx(h);
    const float e = fmaf(p, fmaf(h, -0.6931471806f, -a), p);
    return (z < 0.0f ? z * e : z) * rcp_approx(1.0f + e);
}

// Output of NC token columns: s[j] is the integer sum of token row row0 + j
// and this lane's weight row; as[j] is that token row's scale (shared memory,
// 8-byte aligned).  Rows at or past hi are not stored.  Called by whole warps.
//
// Neighbouring lanes swap half of their results so that each stores two
// neighbouring outputs of one row: half as many stores, and two columns' scale
// products go through one packed multiply.  (One store per output, with the
// row scales fetched by shuffles, took ~20 instructions an output and bounded
// tiles of K = 2048: 8192 x 7168 x 2048 ran 105-130 us against 77 us for the
// main loop alone.)
template <bool GATED, bool BF16, int NC>
__device__ __forceinline__ void emit(const I8Params& p, const int (&s)[NC], const LaneCol& lc,
                                     const float* as, int row0, int hi) {
    const int lane = threadIdx.x & 31;
    const int n_out = GATED ? p.N >> 1 : p.N;
    const float2 bs = make_float2(lc.scale, lc.scale);
    // G of token rows row0 + j and row0 + j + 1
    auto two = [&](int j) {
        const float2 f = make_float2(__int2float_rn(s[j]), __int2float_rn(s[j + 1]));
        return __fmul2_rn(__fmul2_rn(f, *reinterpret_cast<const float2*>(as + j)), bs);
    };
    const bool odd = lane & 1;
    const bool wide = (n_out & 1) == 0;
    // all results first, then the stores: their predicates would otherwise fence
    // the chains of conversions, products and shuffles off from each other
    constexpr int NW = NC / 2 / (GATED ? 2 : 1);   // pair stores of a lane
    if constexpr (!GATED) {
        if (wide) {
            // the even lane finishes rows j, the odd lane rows j + 1
            float2 v[NW];
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const float2 f = two(2 * i);
                const float got = __shfl_xor_sync(0xffffffffu, odd ? f.x : f.y, 1);
                v[i] = make_float2(odd ? got : f.x, odd ? f.y : got);
            }
            store_rows<BF16>(p, v, static_cast<long long>(row0 + (odd ? 1 : 0)) * p.N + (lc.col & ~1),
                             2ll * p.N, 2, lc.ok ? hi - row0 - (odd ? 1 : 0) : 0);
        } else {
#pragma unroll
            for (int j = 0; j < NC; j += 2) {
                const float2 f = two(j);
                const long long at = static_cast<long long>(row0 + j) * p.N + lc.col;
                if (lc.ok && row0 + j < hi) store_out<BF16>(p, at, f.x);
                if (lc.ok && row0 + j + 1 < hi) store_out<BF16>(p, at + p.N, f.y);
            }
        }
    } else {
        const bool up = lane & 16;
        // the gate lane gets the output of row j, the up lane that of row j + 1
        auto gate_up = [&](int j) {
            const float2 f = two(j);
            const float got = __shfl_xor_sync(0xffffffffu, up ? f.x : f.y, 16);
            const float z = up ? got : f.x;
            return (BF16 ? silu_fast(z) : silu_f32(z)) * (up ? f.y : got);
        };
        const int first = up ? 1 : 0;
        if (NW > 0 && wide) {
            const int mine = first + (odd ? 2 : 0);
            float2 v[NW > 0 ? NW : 1];
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const float v0 = gate_up(4 * i), v1 = gate_up(4 * i + 2);
                const float got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
                v[i] = make_float2(odd ? got : v0, odd ? v1 : got);
            }
            store_rows<BF16>(p, v, static_cast<long long>(row0 + mine) * n_out + (lc.col & ~1),
                             4ll * n_out, 4, lc.ok ? hi - row0 - mine : 0);
        } else {
#pragma unroll
            for (int j = 0; j < NC; j += 2) {
                const float v = gate_up(j);
                const int row = row0 + j + first;
                if (lc.ok && row < hi)
                    store_out<BF16>(p, static_cast<long long>(row) * n_out + lc.col, v);
            }
        }
    }
}

// First work item of every expert (start[0..E], start[E] = their number) for
// token blocks of bt rows and `wtiles` weight tiles, by one warp: a lane sums
// the items of its experts, then a scan.
__device__ __forceinline__ void item_table(const I8Params& p, int bt, int wtiles, int* start) {
    const int lane = threadIdx.x & 31;
    const int per = (p.E + 31) >> 5;
    const int e0 = min(p.E, lane * per), e1 = min(p.E, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        int lo, hi;
        expert_rows(p, e, lo, hi);
        start[e] = (hi - lo + bt - 1) / bt * wtiles;   // items, replaced below
        sum += start[e];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    int run = incl - sum;
    for (int e = e0; e < e1; ++e) {
        const int n = start[e];
        start[e] = run;
        run += n;
    }
    if (lane == 31) start[p.E] = incl;
}

// Weight tile wt and token rows [row0, row0 + rows) of expert e.
struct Item {
    int e, wt, row0, rows;
};

// Item i of the table: token blocks inner, so that items that run side by side
// share weight tiles.
__device__ __forceinline__ Item item_of(const I8Params& p, int bt, const int* start, int i) {
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid; else hi = mid;
    }
    int r0, r1;
    expert_rows(p, lo, r0, r1);
    const int local = i - start[lo];
    const int blocks = (r1 - r0 + bt - 1) / bt;
    Item x;
    x.e = lo;
    x.wt = local / blocks;
    x.row0 = r0 + (local - x.wt * blocks) * bt;
    x.rows = min(bt, r1 - x.row0);
    return x;
}

// ------------------------------------------------------------ narrow kernel
// Tiles of 128 weight rows x up to BT token rows, two CTAs an SM, each with a
// ring of NST stages (with BT = 16 the item table leaves room for both up to 895
// experts; beyond, the grid's second half runs after the first).
//  SPLIT = false: CTAs walk over the item table, the next items' loads running
//    under an item's epilogue (4096 rows of 128 experts 1536 x 2048 gated: one
//    CTA per tile 73 us, walking 70.8; and a crowded expert's token blocks are
//    items of their own, where a CTA that looped over them took up to twice as
//    long as the rest).
//  SPLIT = true: few tiles and at most BT rows in all; a cluster of S CTAs
//    shares a tile (grid S * weight tiles, experts), each with the S-th part of
//    the K range.
template <int BT>
struct Narrow {
    static constexpr int NST = BT <= 16 ? 6 : BT <= 32 ? 5 : BT <= 64 ? 4 : 3;
    static constexpr int STAGE = kWBytes + BT * kKB;
    static constexpr int XBOX = BT < 64 ? BT : 64;   // token rows per TMA box
    static constexpr int COLS = 2 * BT < 32 ? 32 : 2 * BT;   // two accumulators
    // warps: 0 TMA, 1 MMA, then 4 epilogue warps, or 8 that share the columns
    static constexpr int PARTS = BT >= 32 ? 2 : 1;
    static constexpr int EPI_WARPS = 4 * PARTS;
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
    static constexpr int PCOLS = BT / PARTS;         // columns of a warp
    static constexpr int AS = EPI_WARPS * PCOLS * 4; // row scales, PCOLS per epilogue warp
    static constexpr int SMEM = 1024 + NST * STAGE + AS + 256;   // and the item table, (E + 1) ints
};

// Weight boxes of a stage: lane i < w_boxes loads box i of the 128-row tile wt
// of expert e.  Plain: one box of 128 rows.  Gated: one box of four granules
// (the map's dimensions are K, 16 rows, gate / up, granules, experts), or, when
// granules would run over the end of a half, eight boxes of 16 rows.  Few large
// boxes: the copies' issue bounded the CTA-pair kernel with 2 KB boxes (a K
// block took ~1150 clocks against 512 of MMA; 8192^3 615 us) and still cost 8%
// with 8 KB ones (381 us against 350).
template <bool GATED>
__device__ __forceinline__ int w_boxes(const I8Params& p) {
    return GATED && p.w_gran ? kWRows / kGran : kWRows / kWBox;
}

template <bool GATED, bool PAIR>
__device__ __forceinline__ void load_weights(const I8Params& p, const CUtensorMap* map, uint8_t* stage,
                                             uint64_t* bar, int kb, int e, int wt, int i) {
    const int x = kb * kKB;
    if (!GATED || p.w_gran) {
        const int row = !GATED ? e * p.N + wt * kWRows + i * kWBox
                               : e * p.N + ((i & 1) ? (p.N >> 1) : 0) + wt * (kWRows / 2) + (i >> 1) * kGran;
        uint8_t* dst = stage + i * (GATED ? kGran : kWBox) * kKB;
        if constexpr (PAIR) tma_load_2d_pair(dst, map, bar, x, row);
        else tma_load_2d(dst, map, bar, x, row);
    } else {
        uint8_t* dst = stage + i * kWBox * kKB;
        const int gran = (wt * (kWRows / kWBox) + i) * (kWBox / (2 * kGran));
        if constexpr (PAIR) tma_load_5d_pair(dst, map, bar, x, 0, 0, gran, e);
        else tma_load_5d(dst, map, bar, x, 0, 0, gran, e);
    }
}

template <int BT, bool GATED, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(Narrow<BT>::THREADS, 2)
    int8_narrow_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                       const I8Params p, int S) {
    using C = Narrow<BT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float* as_all = reinterpret_cast<float*>(base + C::NST * C::STAGE);
    uint64_t* full = reinterpret_cast<uint64_t*>(base + C::NST * C::STAGE + C::AS);
    uint64_t* empty = full + C::NST;
    uint64_t* tfull = empty + C::NST;    // [2]
    uint64_t* tempty = tfull + 2;        // [2]
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_s + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], C::EPI_WARPS);
        }
        mbar_init(drain, 1);
        *abort_s = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    int* start = reinterpret_cast<int*>(base + C::NST * C::STAGE + C::AS + 256);
    pdl_launch();
    pdl_wait();
    // SPLIT: the CTA's only item and its part of the K range
    Item own{};
    int ks = 0;
    if constexpr (SPLIT) {
        own.wt = blockIdx.x / S;
        own.e = blockIdx.y;
        ks = blockIdx.x - own.wt * S;
        int r0, r1;
        expert_rows(p, own.e, r0, r1);
        own.row0 = r0;
        own.rows = min(BT, r1 - own.row0);
        if (own.rows <= 0) return;           // the whole cluster
    } else if (warp == 2) {
        item_table(p, BT, p.wtiles, start);
    }
    if (warp == 1) {
        tmem_alloc(tmem_s, C::COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    const WaitCtl wc{abort_s, p.status, p.timeout_ns};
    const int kb0 = SPLIT ? static_cast<int>(static_cast<long long>(p.nkb) * ks / S) : 0;
    const int kb1 = SPLIT ? static_cast<int>(static_cast<long long>(p.nkb) * (ks + 1) / S) : p.nkb;
    const int items = SPLIT ? 1 : start[p.E];
    const int first = SPLIT ? 0 : blockIdx.x, step = SPLIT ? 1 : gridDim.x;

    if (warp == 0) {
        // lanes 0..7: weight boxes, lanes 8..: token boxes
        const int wb = w_boxes<GATED>(p);
        uint32_t stage = 0, phase = 0, armed = 0, armed_par = 0;
        bool ok = true;
        for (int i = first; i < items && ok; i += step) {
            const Item x = SPLIT ? own : item_of(p, BT, start, i);
            const int boxes = (x.rows + C::XBOX - 1) / C::XBOX;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!warp_wait_spin(&empty[stage], phase ^ 1, wc, 1)) { ok = false; break; }
                uint8_t* st = base + stage * C::STAGE;
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[stage], kWBytes + boxes * C::XBOX * kKB);
                __syncwarp();
                if (lane < wb)
                    load_weights<GATED, false>(p, &tmW, st, &full[stage], kb, x.e, x.wt, lane);
                else if (lane >= 8 && lane < 8 + boxes)
                    tma_load_2d(st + kWBytes + (lane - 8) * C::XBOX * kKB, &tmX, &full[stage], kb * kKB,
                                x.row0 + (lane - 8) * C::XBOX);
                __syncwarp();
                armed |= 1u << stage;
                armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
                if (++stage == C::NST) { stage = 0; phase ^= 1; }
            }
        }
        for (int st = 0; st < C::NST; ++st)
            if ((armed >> st) & 1u) wait_bar(&full[st], (armed_par >> st) & 1u, wc, 2, /*drain=*/true);
        __syncwarp();
    } else if (warp == 1) {
        uint32_t stage = 0, phase = 0, it = 0;
        bool ok = true;
        for (int i = first; i < items && ok; i += step, ++it) {
            const Item x = SPLIT ? own : item_of(p, BT, start, i);
            const uint32_t idesc = idesc_s8_s32(kWRows, (x.rows + 15) & ~15);
            const uint32_t acc = tmem + (it & 1) * BT;
            if (!warp_wait_spin(&tempty[it & 1], ((it >> 1) & 1) ^ 1, wc, 3)) break;
            tc_fence_after();
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!warp_wait_spin(&full[stage], phase, wc, 4)) { ok = false; break; }
                tc_fence_after();
                const uint32_t sw = smem_u32(base + stage * C::STAGE);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_i8(acc, smem_desc_k_sw128(sw + kk * 32),
                                smem_desc_k_sw128(sw + kWBytes + kk * 32), idesc, kb > kb0 || kk > 0);
                    umma_commit(&empty[stage]);
                    if (kb == kb1 - 1) umma_commit(&tfull[it & 1]);
                }
                __syncwarp();
                if (++stage == C::NST) { stage = 0; phase ^= 1; }
            }
        }
        if (elect_one()) umma_commit(drain);
        __syncwarp();
        wait_bar(drain, 0, wc, 5, /*drain=*/true);
        __syncwarp();
    } else {
        const int q = warp & 3;
        const int pos = q * 32 + lane;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const int c0 = (warp - 2) / 4 * C::PCOLS;    // this warp's columns of a block
        float* as = as_all + (warp - 2) * C::PCOLS;
        uint32_t it = 0;
        for (int i = first; i < items; i += step, ++it) {
            const Item x = SPLIT ? own : item_of(p, BT, start, i);
            const LaneCol lc = lane_col<GATED>(p, x.e, x.wt, pos);
            const int row0 = x.row0 + c0, hi = x.row0 + x.rows;
            const int nt = min(C::PCOLS, hi - row0);     // may be none
            stage_row_scales(p, as, row0, C::PCOLS, hi);
            if (!warp_wait(&tfull[it & 1], (it >> 1) & 1, wc, 6)) break;
            tc_fence_after();
            const uint32_t acc = lane_addr + (it & 1) * BT + c0;
            if constexpr (!SPLIT) {
                for (int c = 0; c < nt; c += 16) {
                    uint32_t v[16];
                    tmem_ld16_async(acc + c, v);
                    tmem_wait_ld(v);
                    int s[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] = static_cast<int>(v[j]);
                    emit<GATED, BF16, 16>(p, s, lc, as + c, row0 + c, hi);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[it & 1]);
            } else {
                // one block per CTA: its partial sums go to shared memory, column by
                // column (the pipeline's stages are free: every MMA has completed)
                int* part = reinterpret_cast<int*>(base);
                for (int c = 0; c < nt; c += 16) {
                    uint32_t v[16];
                    tmem_ld16_async(acc + c, v);
                    tmem_wait_ld(v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(c0 + c + j) * kWRows + pos] = static_cast<int>(v[j]);
                }
            }
        }
    }
    if constexpr (SPLIT) {
        // every thread of the cluster: partial sums visible; then the pair
        // columns (2 i, 2 i + 1) are added up and written, i mod S by CTA, then
        // in turn by the CTA's groups of four epilogue warps
        __syncwarp();
        cluster_sync_all();
        if (warp >= 2 && !*abort_s) {
            const int pos = (warp & 3) * 32 + lane;
            const uint32_t mine = smem_u32(base) + pos * 4;
            const LaneCol lc = lane_col<GATED>(p, own.e, own.wt, pos);
            for (int c = 2 * (ks + S * ((warp - 2) / 4)); c < own.rows; c += 2 * S * C::PARTS) {
                int t[kMaxSplit][2];     // every load in flight before the sums
#pragma unroll
                for (int r = 0; r < kMaxSplit; ++r) {
                    t[r][0] = t[r][1] = 0;
                    if (r < S) {
                        const uint32_t at = mapa_shared(mine, r) + c * kWRows * 4;
                        t[r][0] = ld_shared_cluster_s32(at);
                        t[r][1] = ld_shared_cluster_s32(at + kWRows * 4);
                    }
                }
                int s[2] = {0, 0};
#pragma unroll
                for (int r = 0; r < kMaxSplit; ++r) {
                    s[0] += t[r][0];
                    s[1] += t[r][1];
                }
                // column c's scales are in the buffer of the warp of its part and lanes
                const float* as = as_all + ((c / C::PCOLS) * 4 + ((warp - 2) & 3)) * C::PCOLS + c % C::PCOLS;
                emit<GATED, BF16, 2>(p, s, lc, as, own.row0 + c, own.row0 + own.rows);
            }
        }
        __syncwarp();
        cluster_sync_all();   // peers have read this CTA's sums
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::COLS);
}

// ------------------------------------------------------------ pair kernel
// Persistent CTA pairs (cta_group::2), one per two SMs.  A tile is two
// neighbouring 128-row weight tiles (one per CTA) x up to 256 token rows of
// one expert; each CTA stages its own weight rows and half of the token rows,
// so a 128-byte K block costs an SM 32 KB of loads for 512 clocks of MMA, two
// thirds of what a single-CTA 128 x 256 tile loads.  Two 256-column
// accumulators in tensor memory let the epilogue of one tile run under the
// next tile's main loop.
// The ring holds as many stages as fit whatever the tile (6 of 32 KB to 9 of
// 20 KB): a copy takes ~1.8 us under load, so the bytes in flight set the rate.
struct Pair {
    static constexpr int BT = 256;                   // largest tile; accumulators are this far apart
    static constexpr int MAX_NST = 9;
    static constexpr int RING = 6 * (kWBytes + BT / 2 * kKB);
    static constexpr int EPI_WARPS = 8;
    static constexpr int THREADS = 64 + 32 * EPI_WARPS;
    static constexpr int AS = EPI_WARPS * 128 * 4;   // row scales, 128 per epilogue warp
    static constexpr int TABLE = ((MAX_E + 1) * 4 + 15) / 16 * 16;
    static constexpr int SMEM = 1024 + RING + AS + TABLE + 256;
    static_assert(SMEM <= 232448, "shared memory budget");
    static constexpr int stage_bytes(int bt) { return kWBytes + bt / 2 * kKB; }
    static constexpr int stages(int bt) {
        return RING / stage_bytes(bt) < MAX_NST ? RING / stage_bytes(bt) : MAX_NST;
    }
    static constexpr int xbox(int bt) { return bt / 2; }   // token rows per TMA box
};

// SPLIT: few tiles (one expert); a cluster of S pairs shares each, a pair summing
// the S-th part of the K range.  Every CTA then lays its 128 weight rows' sums out
// in shared memory and adds up, over the pairs, every S-th 16 columns of them.
// 256 rows x 4096 x 7168: 19.3 us with one pair a tile, 15.6 with two.
template <bool GATED, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(Pair::THREADS, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                     const I8Params p, int S) {
    using C = Pair;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float* as_all = reinterpret_cast<float*>(base + C::RING);
    int* tstart = reinterpret_cast<int*>(base + C::RING + C::AS);   // [E + 1] first tile
    uint64_t* full = reinterpret_cast<uint64_t*>(base + C::RING + C::AS + C::TABLE);
    uint64_t* empty = full + C::MAX_NST;
    uint64_t* tfull = empty + C::MAX_NST;    // [2]
    uint64_t* tempty = tfull + 2;        // [2], the even CTA's
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_s = reinterpret_cast<volatile int*>(tmem_s + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();
    const uint32_t rank = crank & 1;                 // place in the pair
    const int ks = SPLIT ? static_cast<int>(crank >> 1) : 0;
    const int nst = p.nst, stage_bytes = kWBytes + p.bt * (kKB / 2);
    if (threadIdx.x == 0) {
        for (int i = 0; i < nst; ++i) {
            mbar_init(&full[i], 1);      // the even CTA's producer; both CTAs' bytes
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * C::EPI_WARPS);
        }
        mbar_init(drain, 1);
        *abort_s = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_s, 512);
        tmem_relinquish_pair();
    }
    const int wtiles = GATED ? ((p.N >> 1) + 127) >> 7 : (p.N + 255) >> 8;   // of 256 weight rows
    pdl_launch();
    pdl_wait();
    if (warp == 2) item_table(p, p.bt, wtiles, tstart);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();    // the peer's barriers and tensor memory are ready
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    const WaitCtl wc{abort_s, p.status, p.timeout_ns};
    const int kb0 = SPLIT ? static_cast<int>(static_cast<long long>(p.nkb) * ks / S) : 0;
    const int kb1 = SPLIT ? static_cast<int>(static_cast<long long>(p.nkb) * (ks + 1) / S) : p.nkb;
    // SPLIT: the cluster's only tile (the grid has as many clusters as R rows make
    // tiles; m_indptr may name fewer rows)
    const int first = SPLIT ? blockIdx.x / (2 * S) : blockIdx.x >> 1;
    const int total = SPLIT ? min(first + 1, tstart[p.E]) : tstart[p.E];
    const int stride = SPLIT ? 1 : gridDim.x >> 1;

    // this CTA's half of tile t
    auto decode = [&](int t) {
        Item x = item_of(p, p.bt, tstart, t);
        x.wt = 2 * x.wt + static_cast<int>(rank);
        return x;
    };

    if (warp == 0) {
        const int wb = w_boxes<GATED>(p);
        const int xbox = p.bt >> 1;          // token rows per box
        uint32_t stage = 0, phase = 0, armed = 0, armed_par = 0;
        bool ok = true;
        for (int t = first; t < total && ok; t += stride) {
            const Item x = decode(t);
            const int half = ((x.rows + 31) & ~31) >> 1;      // token rows of this CTA
            const int boxes = (half + xbox - 1) / xbox;
            const int xrow = x.row0 + static_cast<int>(rank) * half + (lane - 8) * xbox;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!warp_wait_spin(&empty[stage], phase ^ 1, wc, 1)) { ok = false; break; }
                uint8_t* st = base + stage * stage_bytes;
                if (rank == 0 && lane == 0)
                    mbar_arrive_expect_tx(&full[stage], 2 * (kWBytes + boxes * xbox * kKB));
                __syncwarp();
                if (lane < wb)
                    load_weights<GATED, true>(p, &tmW, st, &full[stage], kb, x.e, x.wt, lane);
                else if (lane >= 8 && lane < 8 + boxes)
                    tma_load_2d_pair(st + kWBytes + (lane - 8) * xbox * kKB, &tmX, &full[stage],
                                     kb * kKB, xrow);
                __syncwarp();
                armed |= 1u << stage;
                armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
                if (++stage == nst) { stage = 0; phase ^= 1; }
            }
        }
        // No copy and no arrival may still be on its way when the CTA ends.  The
        // even CTA's barriers count both CTAs' copies; the odd CTA waits until
        // the MMAs have released its stages.  After an abort one wait runs out
        // (2 s, long after any copy has landed) and the rest are skipped.
        uint64_t* last = rank == 0 ? full : empty;
        for (int st = 0; st < nst; ++st)
            if (((armed >> st) & 1u) &&
                !wait_bar(&last[st], (armed_par >> st) & 1u, wc, 2, /*drain=*/true))
                break;
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint16_t both = static_cast<uint16_t>(3u << crank);   // this pair's CTAs
            uint32_t stage = 0, phase = 0, it = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += stride, ++it) {
                const Item x = decode(t);
                const uint32_t idesc = idesc_s8_s32(2 * kWRows, (x.rows + 31) & ~31);
                const uint32_t acc = tmem + (it & 1) * C::BT;
                if (!warp_wait_spin(&tempty[it & 1], ((it >> 1) & 1) ^ 1, wc, 3)) break;
                tc_fence_after();
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!warp_wait_spin(&full[stage], phase, wc, 4)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sw = smem_u32(base + stage * stage_bytes);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_i8_pair(acc, smem_desc_k_sw128(sw + kk * 32),
                                         smem_desc_k_sw128(sw + kWBytes + kk * 32), idesc, kb > kb0 || kk > 0);
                        umma_commit_pair(&empty[stage], both);
                        if (kb == kb1 - 1) umma_commit_pair(&tfull[it & 1], both);
                    }
                    __syncwarp();
                    if (++stage == nst) { stage = 0; phase ^= 1; }
                }
            }
            if (elect_one()) umma_commit_pair_local(drain);
            __syncwarp();
            wait_bar(drain, 0, wc, 5, /*drain=*/true);
            __syncwarp();
        }
    } else {
        const int q = warp & 3;
        const int part = (warp - 2) >> 2;    // columns [128 part, 128 part + 128)
        const int pos = q * 32 + lane;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const uint32_t tempty0 = mapa_shared(smem_u32(tempty), crank & ~1u);
        float* as = as_all + (warp - 2) * 128;
        uint32_t it = 0;
        for (int t = first; t < total; t += stride, ++it) {
            const Item x = decode(t);
            const int hi = x.row0 + x.rows;
            const int c0 = part * 128, end = min(x.rows, c0 + 128);
            const LaneCol lc = lane_col<GATED>(p, x.e, x.wt, pos);
            stage_row_scales(p, as, x.row0 + c0, 128, hi);
            if (!warp_wait(&tfull[it & 1], (it >> 1) & 1, wc, 6)) break;
            tc_fence_after();
            const uint32_t acc = lane_addr + (it & 1) * C::BT;
            for (int c = c0; c < end; c += 32) {
                uint32_t v[32];
                tmem_ld32_async(acc + c, v);
                tmem_wait_ld(v);
                if (c + 32 >= end) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(tempty0 + (it & 1) * 8);
                }
                int s[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) s[j] = static_cast<int>(v[j]);
                if constexpr (!SPLIT) {
                    emit<GATED, BF16, 32>(p, s, lc, as + (c - c0), x.row0 + c, hi);
                } else {
                    // the pipeline's stages are free: every MMA has completed
                    int* part_sums = reinterpret_cast<int*>(base);
#pragma unroll
                    for (int j = 0; j < 32; ++j) part_sums[(c + j) * kWRows + pos] = s[j];
                }
            }
            if (end <= c0 && lane == 0) mbar_arrive_cluster(tempty0 + (it & 1) * 8);
        }
    }
    if constexpr (SPLIT) {
        __syncwarp();
        cluster_sync_all();    // every pair's sums are visible
        if (warp >= 2 && first < total && !*abort_s) {
            const Item x = decode(first);
            const int pos = (warp & 3) * 32 + lane;
            const LaneCol lc = lane_col<GATED>(p, x.e, x.wt, pos);
            const uint32_t mine = smem_u32(base) + pos * 4;
            // 16 columns at a time: chunk i by pair i mod S, then in turn by the
            // CTA's two groups of four warps
            for (int c = 16 * (ks + S * ((warp - 2) >> 2)); c < x.rows; c += 32 * S) {
                int s[16] = {};
                for (int r = 0; r < S; ++r) {
                    const uint32_t at = mapa_shared(mine, 2 * r + rank) + c * kWRows * 4;
                    int v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = ld_shared_cluster_s32(at + j * kWRows * 4);
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] += v[j];
                }
                // the scales of column c are in its part's buffers
                const float* as = as_all + ((c >> 7) * 4 + ((warp - 2) & 3)) * 128 + (c & 127);
                emit<GATED, BF16, 16>(p, s, lc, as, x.row0 + c, x.row0 + x.rows);
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();    // all CTAs done with barriers, operands and tensor memory
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

bool encode(CUtensorMap* m, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    auto fn = encode_fn();
    const cuuint32_t es[5] = {1u, 1u, 1u, 1u, 1u};
    auto once = [&] {
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(ptr), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    if (!fn) return false;
    CUresult r = once();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {
        // a thread's first use of CUDA: the driver has no context for it yet, and no
        // runtime call came before this one to give it the current device's
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return false;
        r = once();
    }
    return r == CUDA_SUCCESS;
}

// Map of a row-major int8 matrix [rows, cols] with boxes of box_rows x 128
// bytes and the 128-byte swizzle; bytes past either end read 0.
bool make_map(CUtensorMap* m, const void* ptr, long long rows, int cols, int box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kKB), static_cast<cuuint32_t>(box_rows)};
    return encode(m, ptr, 2, dims, strides, box);
}

// Map of gated weights [E, 2, N/2, K] whose boxes are four granules: 16 gate
// rows, their 16 up rows, four times.
bool make_gated_map(CUtensorMap* m, const void* ptr, int E, int N, int K) {
    const cuuint64_t k = K, half = N / 2;
    const cuuint64_t dims[5] = {k, kGran, 2, half / kGran, static_cast<cuuint64_t>(E)};
    const cuuint64_t strides[4] = {k, half * k, kGran * k, 2 * half * k};
    const cuuint32_t box[5] = {kKB, kGran, 2, kWBox / (2 * kGran), 1};
    return encode(m, ptr, 5, dims, strides, box);
}

// Opt-in of a kernel to its dynamic shared memory, once per device and kernel
// (`ready_dev` is the kernel's own; alternating devices just set it again).
template <typename Kern>
bool smem_ready(Kern kern, int bytes, std::atomic<int>& ready_dev) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (ready_dev.load() == dev) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return false;
    ready_dev.store(dev);
    return true;
}

int weight_tiles(const I8GemmArgs& g) {
    return g.gated ? (g.N / 2 + 63) / 64 : (g.N + 127) / 128;
}

// Token rows of a pair tile and pairs that share one: the fewest clocks for a
// balanced routing.  A 128-byte K block costs an SM its loads, 16 KB of weights
// and 64 bytes a token row at ~58 B/clk (measured), or 2 clocks of MMA a token
// row; a tile adds ~3000 clocks of pipeline fill and epilogue, a split one ~2000
// and 16 a token row for laying out and exchanging its sums.  Only the tiles of
// one expert are split (their number has to be known here), and only where
// their clusters all run side by side (B200: 33 of 4 CTAs, 15 of 8; 16 of 8 took
// a second round, 31 us where 19 would do).
struct PairPlan {
    int bt, S;
};

// Clusters of `ctas` CTAs of the split pair kernel that the current device runs
// at once; asked once per device.
int pair_clusters(int ctas) {
    static std::atomic<int> known[2] = {{-1}, {-1}};       // device << 16 | clusters
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::atomic<int>& k = known[ctas == 4 ? 0 : 1];
    const int have = k.load();   // once: another thread may put another device's in
    if (have >= 0 && have >> 16 == dev) return have & 0xffff;
    static std::atomic<int> ready_dev{-1};
    auto kern = int8_pair_kernel<false, true, true>;
    if (!smem_ready(kern, Pair::SMEM, ready_dev)) return 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas * 64);
    cfg.blockDim = dim3(Pair::THREADS);
    cfg.dynamicSmemBytes = Pair::SMEM;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();   // not this call's error: no split then
        return 0;
    }
    k.store(dev << 16 | n);
    return n;
}

PairPlan pair_plan(const I8GemmArgs& g, int per, int tiles) {
    const long long pairs = g.num_sms / 2, nkb = (g.K + kKB - 1) / kKB;
    const long long w = static_cast<long long>(std::min(g.E, g.R)) * ((tiles + 1) / 2);
    PairPlan best{256, 1};
    long long best_cost = 0;
    for (int bt = 256; bt >= 64; bt /= 2) {
        const long long n = w * ((per + bt - 1) / bt);
        const int kblock = std::max(2 * bt, (16384 + 64 * bt) / 58);
        for (int S = 1; S <= 4; S *= 2) {
            if (S > 1 && (g.E != 1 || nkb < 4 * S || n * S > pairs || n > pair_clusters(2 * S))) break;
            const long long waves = S > 1 ? 1 : (n + pairs - 1) / pairs;
            const long long cost =
                waves * ((nkb + S - 1) / S * kblock + 3000) + (S > 1 ? 2000 + 16 * bt : 0);
            if (best_cost == 0 || cost < best_cost) {
                best = PairPlan{bt, S};
                best_cost = cost;
            }
        }
    }
    return best;
}

template <int BT, bool GATED, bool BF16>
int launch_narrow(const CUtensorMap& mw, const CUtensorMap& mx, const I8Params& p, int S,
                  int num_sms, cudaStream_t stream) {
    using C = Narrow<BT>;
    const size_t smem = C::SMEM + (S > 1 ? 0 : (p.E + 1) * sizeof(int));
    const int most = C::SMEM + (MAX_E + 1) * static_cast<int>(sizeof(int));
    if (S > 1) {
        static std::atomic<int> ready_dev{-1};
        auto kern = int8_narrow_kernel<BT, GATED, BF16, true>;
        if (!smem_ready(kern, most, ready_dev)) return ST_CUDA;
        return launch_dependent(kern, dim3(p.wtiles * S, p.E), dim3(C::THREADS), S, smem, stream, mw, mx, p,
                                S) == cudaSuccess ? ST_OK : ST_CUDA;
    }
    static std::atomic<int> ready_dev{-1};
    auto kern = int8_narrow_kernel<BT, GATED, BF16, false>;
    if (!smem_ready(kern, most, ready_dev)) return ST_CUDA;
    // at most as many items as this (one block more an expert than the rows fill)
    const long long items = static_cast<long long>(p.wtiles) * (p.R / BT + std::min(p.E, p.R));
    const unsigned grid = static_cast<unsigned>(std::min<long long>(items, 2 * num_sms));
    return launch_dependent(kern, dim3(grid), dim3(C::THREADS), 0, smem, stream, mw, mx, p, 1) == cudaSuccess
               ? ST_OK : ST_CUDA;
}

template <bool GATED, bool BF16>
int launch_pair(const CUtensorMap& mw, const CUtensorMap& mx, const I8Params& p, int S, int num_sms,
                cudaStream_t stream) {
    if (S > 1) {
        static std::atomic<int> ready_dev{-1};
        auto kern = int8_pair_kernel<GATED, BF16, true>;
        if (!smem_ready(kern, Pair::SMEM, ready_dev)) return ST_CUDA;
        const int tiles = (p.wtiles + 1) / 2 * ((p.R + p.bt - 1) / p.bt);
        return launch_dependent(kern, dim3(tiles * 2 * S), dim3(Pair::THREADS), 2 * S, Pair::SMEM, stream, mw,
                                mx, p, S) == cudaSuccess ? ST_OK : ST_CUDA;
    }
    static std::atomic<int> ready_dev{-1};
    auto kern = int8_pair_kernel<GATED, BF16, false>;
    if (!smem_ready(kern, Pair::SMEM, ready_dev)) return ST_CUDA;
    return launch_dependent(kern, dim3(num_sms & ~1), dim3(Pair::THREADS), 2, Pair::SMEM, stream, mw, mx, p,
                            1) == cudaSuccess ? ST_OK : ST_CUDA;
}

// Whether the item table's sums stay below 2^31 whatever m_indptr holds (each
// expert's rows are clamped to [0, R], but a wrong table may name rows twice).
bool items_fit(const I8GemmArgs& g, int bt, int tiles) {
    return static_cast<long long>(g.E) * ((g.R + static_cast<long long>(bt) - 1) / bt) * tiles < 0x7fffffffll;
}

template <bool GATED, bool BF16>
int launch_t(const I8GemmArgs& g, cudaStream_t stream) {
    const int nkb = (g.K + kKB - 1) / kKB;
    const int w_gran = GATED && (g.N / 2) % kGran ? 1 : 0;
    I8Params p{g.a_scale, g.b_scale, g.m_indptr, g.out, g.R, g.N, g.E, nkb, weight_tiles(g), 0, 0, w_gran,
                     g.status, g.timeout_ns};
    CUtensorMap mw, mx;
    if (GATED && !w_gran ? !make_gated_map(&mw, g.b, g.E, g.N, g.K)
                         : !make_map(&mw, g.b, static_cast<long long>(g.E) * g.N, g.K, GATED ? kGran : kWBox))
        return ST_CUDA;
    const int tiles = weight_tiles(g);
    const int per = (g.R + g.E - 1) / g.E;   // rows per expert, balanced
    if (per > 128) {
        const PairPlan plan = pair_plan(g, per, tiles);
        p.bt = plan.bt;
        if (!items_fit(g, p.bt, tiles)) return ST_UNSUPPORTED;
        p.nst = Pair::stages(p.bt);
        if (!make_map(&mx, g.a, g.R, g.K, Pair::xbox(p.bt))) return ST_CUDA;
        return launch_pair<GATED, BF16>(mw, mx, p, plan.S, g.num_sms, stream);
    }
    // rows of one expert of a balanced routing, with three standard deviations
    const int want = g.E == 1 ? g.R : std::min(g.R, per + static_cast<int>(3.0f * sqrtf(per)));
    const int bt = want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 ? 64 : 128;
    // split K where the weight tiles leave SMs idle and an expert's rows are one block
    int S = 1;
    if (g.R <= bt) {
        const long long units = static_cast<long long>(tiles) * std::min(g.E, g.R);
        while (S < kMaxSplit && units * S * 2 <= 2 * g.num_sms && nkb >= S * 2 * 4) S *= 2;
    }
    if (!items_fit(g, bt, tiles)) return ST_UNSUPPORTED;
    if (!make_map(&mx, g.a, g.R, g.K, bt < 64 ? bt : 64)) return ST_CUDA;
    switch (bt) {
        case 16: return launch_narrow<16, GATED, BF16>(mw, mx, p, S, g.num_sms, stream);
        case 32: return launch_narrow<32, GATED, BF16>(mw, mx, p, S, g.num_sms, stream);
        case 64: return launch_narrow<64, GATED, BF16>(mw, mx, p, S, g.num_sms, stream);
        default: return launch_narrow<128, GATED, BF16>(mw, mx, p, S, g.num_sms, stream);
    }
}

}  // namespace

int launch_int8_gemm(const I8GemmArgs& g, cudaStream_t stream) {
    if (g.R == 0) return ST_OK;
    if (g.gated) return g.out_bf16 ? launch_t<true, true>(g, stream) : launch_t<true, false>(g, stream);
    return g.out_bf16 ? launch_t<false, true>(g, stream) : launch_t<false, false>(g, stream);
}

}  // namespace moe
