// gemm_grouped.cu -- products of rows in expert order with their expert's
// low-bit weight on tcgen05 tensor cores.
//
// The product is turned round: the weight gives the MMA's M rows and the rows
// of one expert its N columns, N being what the expert has (rounded up to 16 or
// 32).  So a ragged group costs its rows and no more, in MMA time and in the
// bytes of X that a stage loads, and with few rows per expert (a decode step)
// the ring's bytes are nearly all weight, which has to be read once anyway.
//
// Two kernels, chosen on the host from the sizes it knows:
//   k_gemm_grouped_pair   CTA pairs (cta_group::2), 256 features x up to 128 or
//                         256 rows, persistent over (expert, features, rows)
//   k_gemm_grouped_split  where there are so few such items that SMs would
//                         idle: K split over a cluster of 2 or 4 CTAs
// Warps of both:
//   warp 0      TMA producer into a ring of K stages: 128 weight rows x 128
//               bytes, the box of 16 / 32 / 64 / 128 rows of X that fits, the
//               scale atoms of both
//   warp 1      TMEM allocation and the thread that issues the MMAs
//   warps 2-5   epilogue, one per TMEM lane quarter (pairs may have 6-9 too)
//   the rest    (block-scaled formats) a thread per scale atom of a stage, which
//               copies it to TMEM: a tcgen05.cp holds up the thread that issues
//               it, and NVFP4 has eight a stage (one token, 8 of 64 experts,
//               2048 x 4096: 15.1 us with the MMA thread issuing them, 12.7 with
//               a thread for each, 12.0 as the kernels now are)
// Every wait is bounded; one that runs out latches the error word, the CTA
// lets what is in flight land and exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstring>

#include "groups.cuh"
#include "mxq_formats.cuh"
#include "mxq_internal.h"
#include "tc_ptx.cuh"

namespace mxq {
namespace {

constexpr int GG_W = 128 * 128;   // a stage's weight: 128 rows x 128 bytes of K
constexpr unsigned int kErrGrouped = 512u;

struct GroupedParams {
    CUtensorMap w, sfw, sfx, x[4];   // x[i]: boxes of 16 << i rows
    const int32_t *offsets;
    int n_groups, rows;
    const float *x_row_scale, *w_row_scale;   // INT8
    const float *x_ts, *w_ts;                 // NVFP4, FP8: X's scalar, one per expert
    void *y;
    int n, kbytes, num_k_tiles, s4, y_bf16, y_vec;
    int n_tiles, w_tiles;   // feature tiles of an expert, and 128-row tiles of its scales
    int max_tiles;          // row blocks of all experts at most
    unsigned int *err;
    unsigned long long wait_ns;
};

// ---- pieces of both kernels; CG: cta_group, 1 or 2

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <int F>
__host__ __device__ constexpr int gg_atoms() { return F == kNVFP4 ? 4 : F == kMXFP4 ? 2 : F == kMXFP8 ? 1 : 0; }
template <int F>
__host__ __device__ constexpr int gg_threads() { return 192 + 32 * gg_atoms<F>(); }
// K-major operands; M / 16 at bit 24 and N / 8 at bit 17 are or-ed in.
template <int F>
__host__ __device__ constexpr uint32_t gg_idesc() {
    return F == kNVFP4       ? (1u << 7) | (1u << 10)                 // E2M1, UE4M3 scales
           : F == kMXFP4     ? (1u << 7) | (1u << 10) | (1u << 23)    // E2M1, UE8M0 scales
           : F == kMXFP8     ? (1u << 23)                             // E4M3, UE8M0 scales
           : F == kFP8Tensor ? (1u << 4)                              // E4M3 -> fp32
                             : (2u << 4) | (1u << 7) | (1u << 10);    // s8 -> s32
}

#define MXQ_MMA_SCALED(CG, KIND)                                                                                    \
    asm volatile(                                                                                                   \
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                                           \
        "tcgen05.mma.cta_group::" CG ".kind::" KIND " [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),              \
        "l"(a), "l"(b), "r"(id), "r"(acc), "r"(sa), "r"(sb))
#define MXQ_MMA_PLAIN(CG, KIND)                                                                                     \
    asm volatile(                                                                                                   \
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                                           \
        "tcgen05.mma.cta_group::" CG ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(d),                          \
        "l"(a), "l"(b), "r"(idesc), "r"(acc))

// One 32-byte k-step.  sf: the stage's scale columns, `pitch` per atom: W's 4,
// then X's.  An NVFP4 atom serves one k-step, an MXFP4 atom two (scale columns
// 0-1, then 2-3), an MXFP8 atom four.
template <int F, int CG>
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t sf,
                                         uint32_t pitch, int ks) {
    const int atom = F == kNVFP4 ? ks : F == kMXFP4 ? ks >> 1 : 0;
    const uint32_t col = F == kMXFP4 ? (uint32_t)(ks & 1) * 2 : F == kMXFP8 ? (uint32_t)ks : 0u;
    const uint32_t id = idesc | (col << 29) | (col << 4), sa = sf + pitch * atom, sb = sa + 4;
    if (F == kNVFP4) {
        if (CG == 1) MXQ_MMA_SCALED("1", "mxf4nvf4.block_scale.scale_vec::4X");
        else MXQ_MMA_SCALED("2", "mxf4nvf4.block_scale.scale_vec::4X");
    } else if (F == kMXFP4) {
        if (CG == 1) MXQ_MMA_SCALED("1", "mxf4nvf4.block_scale.scale_vec::2X");
        else MXQ_MMA_SCALED("2", "mxf4nvf4.block_scale.scale_vec::2X");
    } else if (F == kMXFP8) {
        if (CG == 1) MXQ_MMA_SCALED("1", "mxf8f6f4.block_scale.scale_vec::1X");
        else MXQ_MMA_SCALED("2", "mxf8f6f4.block_scale.scale_vec::1X");
    } else if (F == kFP8Tensor) {
        if (CG == 1) MXQ_MMA_PLAIN("1", "f8f6f4");
        else MXQ_MMA_PLAIN("2", "f8f6f4");
    } else {
        if (CG == 1) MXQ_MMA_PLAIN("1", "i8");
        else MXQ_MMA_PLAIN("2", "i8");
    }
}

// The box of X (its log2 over 16 rows) that holds `rows` rows.
__device__ __forceinline__ int box_of(int rows) { return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3; }

// Eight neighbouring values of a row of y from their sums: scaled as
// mxq_qlinear does it, rounded once, stored.
template <int F>
__device__ __forceinline__ void store_row8(const GroupedParams &p, float (&v)[8], int group, int row, int col, float alpha) {
    if (F == kINT8Row) {
        const float xs = __ldg(p.x_row_scale + row);
        const float *ws = p.w_row_scale + (int64_t)group * p.n + col;
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = __fmul_rn(__fmul_rn(v[i], xs), col + i < p.n ? __ldg(ws + i) : 0.0f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = __fmul_rn(v[i], alpha);
    }
    const int64_t at = (int64_t)row * p.n + col;
    const bool whole = p.y_vec && col + 8 <= p.n;
    if (p.y_bf16) {
        __nv_bfloat16 *y = reinterpret_cast<__nv_bfloat16 *>(p.y) + at;
        if (whole) {
            *reinterpret_cast<uint4 *>(y) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                       pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (col + i < p.n) y[i] = __float2bfloat16_rn(v[i]);
        }
    } else {
        float *y = reinterpret_cast<float *>(p.y) + at;
        if (whole) {
            reinterpret_cast<float4 *>(y)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4 *>(y)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (col + i < p.n) y[i] = v[i];
        }
    }
}
// A lane's feature `col` of up to 32 rows from row0 on (`left` of them exist),
// r[j] the sum of row j: scaled, rounded once and stored without a detour
// through shared memory.  A row's 32 features of a warp are 64 bytes in bf16,
// two whole sectors: neighbouring lanes exchange halves so that even lanes
// hold two features of an even row and odd lanes of the next.
template <int F>
__device__ __forceinline__ void store_chunk(const GroupedParams &p, const uint32_t (&r)[32], int row0, int left, int col,
                                            float alpha, float ws, int lane) {
    float xs = 0.0f;   // INT8: lane j has row j's scale
    if (F == kINT8Row && lane < left) xs = __ldg(p.x_row_scale + row0 + lane);
    auto value = [&](int j) {
        if (F == kINT8Row) return __fmul_rn(__fmul_rn((float)(int)r[j], __shfl_sync(0xFFFFFFFFu, xs, j)), ws);
        return __fmul_rn(__uint_as_float(r[j]), alpha);
    };
    const bool mine = col < p.n;
    if (!p.y_bf16) {
        float *y = reinterpret_cast<float *>(p.y) + (int64_t)row0 * p.n + col;
#pragma unroll
        for (int j = 0; j < 32; j++, y += p.n) {
            const float v = value(j);
            if (mine && j < left) *y = v;
        }
    } else if ((p.n & 1) == 0) {
        const int odd = lane & 1;
        const uint32_t pick = odd ? 0x3276u : 0x5410u;
        __nv_bfloat16 *y = reinterpret_cast<__nv_bfloat16 *>(p.y) + (int64_t)(row0 + odd) * p.n + (col - odd);
#pragma unroll
        for (int j = 0; j < 32; j += 2, y += 2 * (int64_t)p.n) {
            const uint32_t own = pack_bf16x2(value(j), value(j + 1));
            const uint32_t w = __byte_perm(own, __shfl_xor_sync(0xFFFFFFFFu, own, 1), pick);
            if (mine && j + odd < left) *reinterpret_cast<uint32_t *>(y) = w;
        }
    } else {   // rows that start at odd elements
        __nv_bfloat16 *y = reinterpret_cast<__nv_bfloat16 *>(p.y) + (int64_t)row0 * p.n + col;
#pragma unroll
        for (int j = 0; j < 32; j++, y += p.n) {
            const float v = value(j);
            if (mine && j < left) *y = __float2bfloat16_rn(v);
        }
    }
}
template <int F>
__device__ __forceinline__ float scale_of(const GroupedParams &p, int group) {
    return F == kNVFP4 || F == kFP8Tensor ? __fmul_rn(__ldg(p.x_ts), __ldg(p.w_ts + group)) : 1.0f;
}
template <int F>
__device__ __forceinline__ void prefetch_maps(const GroupedParams &p, int warp, int lane) {
    if (warp == 0 && lane < (gg_atoms<F>() ? 7 : 5)) {
        const CUtensorMap *m = lane < 4 ? p.x + lane : lane == 4 ? &p.w : lane == 5 ? &p.sfw : &p.sfx;
        asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
}
// Whether all epilogue threads of a pair's CTA say so: they meet at barriers,
// so they go on together or not at all.
template <int THREADS>
__device__ __forceinline__ bool all_epilogue(bool ok) {
    int all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.and.pred q, 2, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((int)ok), "n"(THREADS)
        : "memory");
    return all != 0;
}

// An item: a feature tile of an expert times a block of 128 (or, WIDE, 256) of
// its rows.  An expert's blocks of one feature tile are neighbours.
struct Item {
    int group, tile_n, row0, n_rows, sf_tile;
};
template <bool WIDE>
__device__ __forceinline__ Item item_at(const Groups &g, int n_groups, int n_tiles, int item) {
    const int *before = WIDE ? g.wide : g.tile;
    const int key = item / n_tiles;   // the item's row block, counted over all groups
    int lo = 0, hi = n_groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= key) lo = mid;
        else hi = mid;
    }
    constexpr int R = WIDE ? 256 : 128;
    const int blocks = before[lo + 1] - before[lo], within = item - before[lo] * n_tiles;
    Item it;
    it.group = lo;
    it.tile_n = within / blocks;
    const int block = within - it.tile_n * blocks;
    it.row0 = g.off[lo] + block * R;
    const int left = g.off[lo + 1] - it.row0;
    it.n_rows = left < R ? left : R;
    it.sf_tile = g.tile[lo] + block * (R / 128);
    return it;
}

// ---- pairs
//
// A pair of CTAs (cta_group::2) computes 256 features x a block of up to NB
// rows: each stages its 128 weight rows and half of the block's rows of X,
// holds the scales of its weight rows and of all rows of X, and its 128
// features x N accumulator.  N is the block's rows rounded up to 32, so a
// ragged block costs what it has.  The first CTA's MMA and scale threads serve
// both.  An expert's blocks of one feature tile are neighbours among the items,
// so the weight's second read is served by L2; two accumulator stages let an
// item's loads and MMAs run under the epilogue of the one before.
//   NB = 128: two accumulators of 128 columns leave every stage of the ring
//     its own scale columns, so the copies run as far ahead as the loads.
//   NB = 256: the accumulator stages lie at columns 0 and 160 and share columns
//     with a full block (two of 256 do not fit beside the scales): the epilogue
//     takes the shared chunks to registers first and releases them; two stages'
//     scales in TMEM at a time.
template <int F, int NB, int SP>
struct Pair {
    static constexpr int kAtoms = gg_atoms<F>();
    static constexpr int kEpi = 4 * SP;   // epilogue warps: SP per TMEM lane quarter, which take its chunks in turn
    static constexpr int kThreads = 32 * (2 + kEpi + kAtoms);
    static constexpr int kXBytes = NB / 2 * 128;
    static constexpr int kSfBytes = 2048 + NB * 16;        // W's atoms, then X's by 128 rows
    static constexpr int kStage = GG_W + kXBytes + kSfBytes;
    static constexpr int kStages = NB == 128 ? 7 : 5;
    static constexpr int kSmem = kStages * kStage + (int)sizeof(Groups) + 256 + 1024;
    static constexpr uint32_t kPitch = 4 + NB / 32;        // scale columns per atom
    static constexpr uint32_t kSfCols = 4 * kPitch;        // per stage
    static constexpr uint32_t kSfGroups = NB == 128 ? kStages : 2;   // stages whose scales TMEM holds
    static constexpr uint32_t kTmemSf = 512 - kSfGroups * kSfCols;
    static constexpr uint32_t kAcc1 = NB == 128 ? 128 : kAtoms ? 160 : 256;
    static constexpr int kShared = NB == 256 && kAtoms ? 3 : 0;      // 32-column chunks that both accumulators use
    static_assert(kStage % 1024 == 0 && kSmem <= 227 * 1024, "shared memory budget");
    static_assert(kAcc1 + NB <= (kAtoms ? kTmemSf : 512u) && kAcc1 + 32 * kShared >= (uint32_t)NB, "TMEM budget");
};

template <int F, int NB, int SP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Pair<F, NB, SP>::kThreads, 1)
    k_gemm_grouped_pair(const __grid_constant__ GroupedParams p) {
    using P = Pair<F, NB, SP>;
    constexpr int ST = P::kStages;
    constexpr bool WIDE = NB == 256;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + ST * P::kStage);   // (used in the first CTA)
    uint64_t *empty = full + ST;
    uint64_t *accf = empty + ST;      // [2] accumulator stage full
    uint64_t *acce = accf + 2;        // [2] drained (first CTA)
    uint64_t *ovlf = acce + 2;        // shared columns drained (first CTA)
    uint64_t *drain = ovlf + 1;
    uint64_t *sfready = drain + 1;    // [ST] a stage's scales in TMEM (first CTA)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sfready + ST);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    Groups &groups = *reinterpret_cast<Groups *>(smem + ST * P::kStage + 256);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int cid = (int)cluster_id(), ncl = (int)cluster_count();
    constexpr int NSF = gg_atoms<F>();

    prefetch_maps<F>(p, warp, lane);
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; s++) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
            mbar_init(sfready + s, NSF ? NSF : 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(accf + i, 1);
            mbar_init(acce + i, 2 * P::kEpi);   // the epilogue warps of both CTAs
        }
        mbar_init(ovlf, 2 * P::kEpi);
        mbar_init(drain, 1 + NSF);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();
    load_groups(groups, p.offsets, p.n_groups, p.rows, blockIdx.x == 0 ? p.err : nullptr);
    const int blocks = (WIDE ? groups.wide : groups.tile)[p.n_groups];   // above max_tiles only for offsets out of order
    const int items = (blocks < p.max_tiles ? blocks : p.max_tiles) * p.n_tiles;

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (int item = cid; item < items && !*abort_flag; item += ncl) {
                const Item w = item_at<WIDE>(groups, p.n_groups, p.n_tiles, item);
                const int half = ((w.n_rows + 31) >> 5) << 4;   // rows of X in each CTA
                const int box = box_of(half);
                const bool hi = WIDE && w.n_rows > 128;         // X's second scale tile
                const uint32_t bytes = 2u * (GG_W + (2048u << box)) + NSF * 512u * 2u * (hi ? 3u : 2u);
                const int wrow = w.group * p.n + w.tile_n * 256 + (int)rank * 128, xrow = w.row0 + (int)rank * half;
                const int wsf = w.group * p.w_tiles + w.tile_n * 2 + (int)rank;
                for (int kt = 0; kt < p.num_k_tiles; kt++, it++) {
                    const int s = it % ST;
                    if (!mbar_wait(empty + s, ((it / ST) & 1) ^ 1, p.wait_ns)) {
                        atomicOr(p.err, kErrGrouped);
                        *abort_flag = 1;
                    }
                    if (*abort_flag) break;
                    uint8_t *sw = smem + s * P::kStage, *sf = sw + GG_W + P::kXBytes;
                    const uint32_t bar = map_to_rank(full + s, 0);
                    if (rank == 0) mbar_arrive_expect_tx(full + s, bytes);
                    tma_load_pair(&p.w, sw, bar, kt * 128, wrow);
                    tma_load_pair(&p.x[box], sw + GG_W, bar, kt * 128, xrow);
                    if (NSF) {
                        tma_load_pair(&p.sfw, sf, bar, 0, wsf * p.s4 + kt * NSF);
                        tma_load_pair(&p.sfx, sf + 2048, bar, 0, w.sf_tile * p.s4 + kt * NSF);
                        if (hi) tma_load_pair(&p.sfx, sf + 4096, bar, 0, (w.sf_tile + 1) * p.s4 + kt * NSF);
                    }
                }
            }
            if (*abort_flag && rank == 0)   // wait (bounded) for the loads that may still be in flight
                for (int i = (it > ST ? it - ST : 0); i < it; i++)
                    mbar_wait(full + (i % ST), (i / ST) & 1, p.wait_ns);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int it = 0, count = 0, s = 0;
            uint32_t ph = 0;
            const uint64_t ad0 = sdesc_sw128(smem), bd0 = sdesc_sw128(smem + GG_W);
            for (int item = cid; item < items && !*abort_flag; item += ncl, count++) {
                const Item w = item_at<WIDE>(groups, p.n_groups, p.n_tiles, item);
                const uint32_t idesc = gg_idesc<F>() | (16u << 24) | ((uint32_t)((w.n_rows + 31) >> 5) << 19);
                const int st = count & 1;
                const uint32_t acc = tmem + (st ? P::kAcc1 : 0u);
                // this stage drained (item count - 2) and the shared columns (item count - 1), in both CTAs
                bool ok = mbar_wait_spin<true>(acce + st, ((count >> 1) & 1) ^ 1, p.wait_ns);
                if (P::kShared && ok && count > 0) ok = mbar_wait_spin<true>(ovlf, (count - 1) & 1, p.wait_ns);
                tc_fence_after();
                for (int kt = 0; kt < p.num_k_tiles && ok && !*abort_flag; kt++, it++) {
                    ok = mbar_wait_spin(NSF ? sfready + s : full + s, ph, p.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sft = tmem + P::kTmemSf + P::kSfCols * ((uint32_t)it % P::kSfGroups);
                    const int left = (p.kbytes - kt * 128) >> 5;
                    const uint64_t off = (uint64_t)(s * (P::kStage >> 4));
#pragma unroll
                    for (int ks = 0; ks < 4; ks++)
                        if (ks < left)
                            mma_step<F, 2>(acc, ad0 + off + 2 * ks, bd0 + off + 2 * ks, idesc, (kt | ks) != 0, sft, P::kPitch, ks);
                    tc_commit_pair(empty + s);
                    if (++s == ST) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) {
                    atomicOr(p.err, kErrGrouped);
                    *abort_flag = 1;
                }
                if (*abort_flag) break;
                tc_commit_pair(accf + st);
            }
            if (*abort_flag) {   // what is in flight lands before the TMEM is freed
                tc_commit_pair_self(drain);
                mbar_wait(drain, 0, p.wait_ns);
            }
        }
    } else if (warp >= 2 + P::kEpi) {
        const int atom = warp - 2 - P::kEpi;
        if (NSF && lane == 0 && rank == 0) {
            int it = 0;
            for (int item = cid; item < items && !*abort_flag; item += ncl) {
                const bool hi = WIDE && item_at<WIDE>(groups, p.n_groups, p.n_tiles, item).n_rows > 128;
                for (int kt = 0; kt < p.num_k_tiles; kt++, it++) {
                    const int s = it % ST;
                    bool ok = mbar_wait(full + s, (it / ST) & 1, p.wait_ns);
                    // these columns were last read by the MMAs of k-tile it - kSfGroups (a stage of its own: when it was loaded)
                    const int prev = it - (int)P::kSfGroups;
                    if ((int)P::kSfGroups < ST && ok && prev >= 0) ok = mbar_wait(empty + prev % ST, (prev / ST) & 1, p.wait_ns);
                    if (!ok) {
                        atomicOr(p.err, kErrGrouped);
                        *abort_flag = 1;
                    }
                    if (*abort_flag) break;
                    tc_fence_after();
                    if (atom * (4 / (NSF ? NSF : 1)) * 32 < p.kbytes - kt * 128) {
                        const uint8_t *sf = smem + s * P::kStage + GG_W + P::kXBytes + 512 * atom;
                        const uint32_t to = tmem + P::kTmemSf + P::kSfCols * ((uint32_t)it % P::kSfGroups) + P::kPitch * atom;
                        tc_cp_pair(to, sdesc_atom(sf));
                        tc_cp_pair(to + 4, sdesc_atom(sf + 2048));
                        if (hi) tc_cp_pair(to + 8, sdesc_atom(sf + 4096));
                    }
                    tc_commit_pair_self(sfready + s);
                }
            }
            if (*abort_flag) {
                tc_commit_pair_self(drain);
                mbar_wait(drain, 0, p.wait_ns);
            }
        }
    } else {
        const int q = warp & 3, feature = q * 32 + lane;   // TMEM lane quarter and lane
        const int part = (warp - 2) >> 2;                  // this warp's chunks: part, part + SP, ..
        const uint32_t ovl_to = map_to_rank(ovlf, 0), acce_to = map_to_rank(acce, 0);   // acce + 1: 8 bytes on
        int count = 0;
        for (int item = cid; item < items; item += ncl, count++) {
            const Item w = item_at<WIDE>(groups, p.n_groups, p.n_tiles, item);
            const int st = count & 1;
            const bool ok = !*abort_flag && mbar_wait(accf + st, (count >> 1) & 1, p.wait_ns);
            if (!all_epilogue<32 * P::kEpi>(ok)) {
                if (!ok && !*abort_flag) atomicOr(p.err, kErrGrouped);
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            const float alpha = scale_of<F>(p, w.group);
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (st ? P::kAcc1 : 0u);
            const int col = w.tile_n * 256 + (int)rank * 128 + feature, n_chunks = (w.n_rows + 31) >> 5;
            const float ws = F == kINT8Row && col < p.n ? __ldg(p.w_row_scale + (int64_t)w.group * p.n + col) : 0.0f;
            auto process = [&](int c, const uint32_t (&r)[32]) {   // 32 rows of the block
                store_chunk<F>(p, r, w.row0 + c * 32, w.n_rows - c * 32, col, alpha, ws, lane);
            };
            // chunks [first, first + shared) lie in columns that the other stage uses too
            constexpr int kShared = P::kShared;
            int first = 0, shared = 0;
            if constexpr (kShared > 0) {
                constexpr int kOwn = (kShared + SP - 1) / SP;
                first = st ? 0 : 5;
                shared = n_chunks - first < 0 ? 0 : n_chunks - first < kShared ? n_chunks - first : kShared;
                uint32_t ro[kOwn][32];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kOwn; i++)
                    if (SP * i + part < shared) tmem_ld_32x32b_x32_async(acc + 32u * (first + SP * i + part), ro[i]);
                tmem_ld_wait(ro[kOwn - 1]);
#pragma unroll
                for (int i = 0; i + 1 < kOwn; i++) tmem_reg_tie(ro[i]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_relaxed(ovl_to);
#pragma unroll
                for (int i = 0; i < kOwn; i++)
                    if (SP * i + part < shared) process(first + SP * i + part, ro[i]);
            }
            const int others = n_chunks - shared;
            if (part >= others) {   // none for this warp
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_relaxed(acce_to + 8u * st);
            }
#pragma unroll 1
            for (int i = part; i < others; i += SP) {
                const int c = st ? shared + i : i;
                uint32_t r[32];
                __syncwarp();
                tmem_ld_32x32b_x32(acc + 32u * c, r);
                if (i + SP >= others) {   // this warp's last
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote_relaxed(acce_to + 8u * st);
                }
                process(c, r);
            }
        }
    }

    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
    }
}

// ---- K split over a cluster
//
// A cluster holds one item, 128 features x up to 128 rows; CTA r of S does
// k-tiles [KT r / S, KT (r + 1) / S) with cta_group::1 MMAs, leaves its sums in
// the shared memory of the ring, which is done with, and adds its share of the
// rows from all CTAs over distributed shared memory in rank order: no atomics,
// no workspace, the same bits from run to run.  INT8 sums are added as
// integers.

constexpr int GS_STAGES = 5;
constexpr int GS_X = 128 * 128;
constexpr int GS_SF = 2048;   // up to 4 atoms, for W and for X
constexpr int GS_STAGE = GG_W + GS_X + 2 * GS_SF;
constexpr int GS_SMEM = GS_STAGES * GS_STAGE + (int)sizeof(Groups) + 256 + 1024;
static_assert(128 * 128 * 4 <= GS_STAGES * GS_STAGE, "the sums of a block in the ring");
constexpr uint32_t GS_TMEM_SF = 128;   // the accumulator's 128 columns, then 32 of scales per stage
static_assert(GS_TMEM_SF + 32 * GS_STAGES <= 512, "TMEM budget");
static_assert(GS_SMEM <= 227 * 1024, "shared memory budget");

template <int F>
__global__ void __launch_bounds__(gg_threads<F>(), 1) k_gemm_grouped_split(const __grid_constant__ GroupedParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint32_t *sums = reinterpret_cast<uint32_t *>(smem);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + GS_STAGES * GS_STAGE);
    uint64_t *empty = full + GS_STAGES;
    uint64_t *sfready = empty + GS_STAGES;   // [GS_STAGES] a stage's scales in TMEM
    uint64_t *accf = sfready + GS_STAGES;    // the sums are in TMEM
    uint64_t *ready = accf + 1;              // every CTA's sums are in its shared memory
    uint64_t *drain = ready + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    Groups &groups = *reinterpret_cast<Groups *>(smem + GS_STAGES * GS_STAGE + 256);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t split;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    const uint32_t rank = cluster_rank();
    const int item = (int)cluster_id();
    constexpr int NSF = gg_atoms<F>();

    prefetch_maps<F>(p, warp, lane);
    if (threadIdx.x == 0) {
        for (int s = 0; s < GS_STAGES; s++) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
            mbar_init(sfready + s, NSF ? NSF : 1);
        }
        mbar_init(accf, 1);
        mbar_init(ready, 4 * split);
        mbar_init(drain, 1 + NSF);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();
    load_groups(groups, p.offsets, p.n_groups, p.rows, blockIdx.x == 0 ? p.err : nullptr);
    const int blocks = groups.tile[p.n_groups];   // above max_tiles only for offsets out of order
    const bool work = item < (blocks < p.max_tiles ? blocks : p.max_tiles) * p.n_tiles;   // (the grid has the most items there can be)

    if (work) {
        const Item w = item_at<false>(groups, p.n_groups, p.n_tiles, item);
        const int kt0 = (int)((int64_t)p.num_k_tiles * rank / split), n_kt = (int)((int64_t)p.num_k_tiles * (rank + 1) / split) - kt0;
        if (warp == 0) {
            if (lane == 0) {
                const int box = box_of(w.n_rows);
                const uint32_t bytes = GG_W + (2048u << box) + NSF * 1024u;
                int it = 0;
                for (; it < n_kt; it++) {
                    const int s = it % GS_STAGES, kt = kt0 + it;
                    if (!mbar_wait(empty + s, ((it / GS_STAGES) & 1) ^ 1, p.wait_ns)) {
                        atomicOr(p.err, kErrGrouped);
                        *abort_flag = 1;
                    }
                    if (*abort_flag) break;
                    uint8_t *sw = smem + s * GS_STAGE, *sf = sw + GG_W + GS_X;
                    mbar_arrive_expect_tx(full + s, bytes);
                    tma_load_2d(&p.w, sw, full + s, kt * 128, w.group * p.n + w.tile_n * 128);
                    tma_load_2d(&p.x[box], sw + GG_W, full + s, kt * 128, w.row0);
                    if (NSF) {
                        tma_load_2d(&p.sfw, sf, full + s, 0, (w.group * p.w_tiles + w.tile_n) * p.s4 + kt * NSF);
                        tma_load_2d(&p.sfx, sf + GS_SF, full + s, 0, w.sf_tile * p.s4 + kt * NSF);
                    }
                }
                if (*abort_flag)   // wait (bounded) for the loads that may still be in flight
                    for (int i = (it > GS_STAGES ? it - GS_STAGES : 0); i < it; i++)
                        mbar_wait(full + (i % GS_STAGES), (i / GS_STAGES) & 1, p.wait_ns);
            }
        } else if (warp == 1) {
            if (lane == 0) {
                const uint64_t ad0 = sdesc_sw128(smem), bd0 = sdesc_sw128(smem + GG_W);
                const uint32_t idesc = gg_idesc<F>() | (8u << 24) | ((uint32_t)((w.n_rows + 15) >> 4) << 18);
                for (int it = 0; it < n_kt; it++) {
                    const int s = it % GS_STAGES;
                    if (!mbar_wait_spin(NSF ? sfready + s : full + s, (it / GS_STAGES) & 1, p.wait_ns)) {
                        atomicOr(p.err, kErrGrouped);
                        *abort_flag = 1;
                    }
                    if (*abort_flag) break;
                    tc_fence_after();
                    const int left = (p.kbytes - (kt0 + it) * 128) >> 5;
                    const uint64_t off = (uint64_t)(s * (GS_STAGE >> 4));
#pragma unroll
                    for (int ks = 0; ks < 4; ks++)
                        if (ks < left)
                            mma_step<F, 1>(tmem, ad0 + off + 2 * ks, bd0 + off + 2 * ks, idesc, (it | ks) != 0,
                                           tmem + GS_TMEM_SF + 32u * s, 8, ks);
                    tc_commit(empty + s);
                }
                if (!*abort_flag) {
                    tc_commit(accf);
                } else {   // what is in flight lands before the TMEM is freed
                    tc_commit(drain);
                    mbar_wait(drain, 0, p.wait_ns);
                }
            }
        } else if (warp >= 6) {
            const int atom = warp - 6;
            if (lane == 0) {
                for (int it = 0; it < n_kt; it++) {
                    const int s = it % GS_STAGES;
                    if (!mbar_wait(full + s, (it / GS_STAGES) & 1, p.wait_ns)) {
                        atomicOr(p.err, kErrGrouped);
                        *abort_flag = 1;
                    }
                    if (*abort_flag) break;
                    tc_fence_after();
                    if (atom * (4 / (NSF ? NSF : 1)) * 32 < p.kbytes - (kt0 + it) * 128) {
                        const uint8_t *sf = smem + s * GS_STAGE + GG_W + GS_X + 512 * atom;
                        const uint32_t to = tmem + GS_TMEM_SF + 32u * s + 8u * atom;
                        tc_cp(to, sdesc_atom(sf));
                        tc_cp(to + 4, sdesc_atom(sf + GS_SF));
                    }
                    tc_commit(sfready + s);
                }
                if (*abort_flag) {
                    tc_commit(drain);
                    mbar_wait(drain, 0, p.wait_ns);
                }
            }
        } else {
            const int q = warp & 3, feature = q * 32 + lane;   // TMEM lane quarter and lane
            const int et = threadIdx.x - 64, v8 = et & 15;     // 0 .. 127 among the epilogue threads; 8 features to store
            const float alpha = scale_of<F>(p, w.group);
            bool ok = mbar_wait(accf, 0, p.wait_ns) && !*abort_flag;
            tc_fence_after();
            for (int c = 0; c < (w.n_rows + 31) >> 5; c++) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld_32x32b_x32(tmem + ((uint32_t)(q * 32) << 16) + 32u * c, r);
#pragma unroll
                for (int j = 0; j < 32; j++) sums[(c * 32 + j) * 128 + feature] = r[j];
            }
            __syncwarp();
            if (lane < (int)split) mbar_arrive_remote(map_to_rank(ready, lane));
            if (ok) ok = mbar_wait<true>(ready, 0, p.wait_ns);
            // every split-th eight rows, 8 features per thread
            for (int j = (int)rank * 8 + (et >> 4); j < w.n_rows && ok; j += 8 * (int)split) {
                float v[8] = {};
                int vi[8] = {};
                for (uint32_t s = 0; s < split; s++) {
                    const uint32_t at = map_to_rank(sums + j * 128 + v8 * 8, s);
                    const float4 a = ld_cluster_f4(at), b = ld_cluster_f4(at + 16);
                    const float u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        if (F == kINT8Row) vi[i] += __float_as_int(u[i]);
                        else v[i] = __fadd_rn(v[i], u[i]);
                    }
                }
                if (F == kINT8Row) {
#pragma unroll
                    for (int i = 0; i < 8; i++) v[i] = (float)vi[i];
                }
                store_row8<F>(p, v, w.group, w.row0 + j, w.tile_n * 128 + v8 * 8, alpha);
            }
            if (!ok) {
                if (!*abort_flag) atomicOr(p.err, kErrGrouped);
                *abort_flag = 1;
            }
        }
    }

    tc_fence_before();
    cluster_sync();   // no CTA leaves while another may read its sums
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
    }
}

// ------------------------------------------------------------------ host

template <int F>
cudaError_t launch_split(const GroupedParams &p, int clusters, int split, cudaStream_t s) {
    static PerDeviceOnce smem_opt_in;
    cudaError_t e = smem_opt_in.run([] {
        return cudaFuncSetAttribute(k_gemm_grouped_split<F>, cudaFuncAttributeMaxDynamicSharedMemorySize, GS_SMEM);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * split), 1, 1);
    cfg.blockDim = dim3(gg_threads<F>(), 1, 1);
    cfg.dynamicSmemBytes = GS_SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2] = {pdl_attribute()};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_gemm_grouped_split<F>, p);
}

template <int F, int NB, int SP>
cudaError_t launch_pair(const GroupedParams &p, int clusters, cudaStream_t s) {
    constexpr int smem = Pair<F, NB, SP>::kSmem;
    static PerDeviceOnce smem_opt_in;
    cudaError_t e = smem_opt_in.run([] {
        return cudaFuncSetAttribute(k_gemm_grouped_pair<F, NB, SP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * clusters), 1, 1);
    cfg.blockDim = dim3(Pair<F, NB, SP>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_gemm_grouped_pair<F, NB, SP>, p);
}

// The host knows the rows of all experts together, not of each, and those by
// capacity: dropped choices and, in a call on a part of the experts, the rows of
// the others count as rows.  Blocks: what they can need at most.  (kernel_of in tests/test_gpu_experts.py restates the
// rule, so that a case there names the kernel it is for.)
//   K is split S ways while the items leave SMs idle (items S 2 <= SMs) and
//   every CTA keeps two k-tiles, up to 4 (one token, 2 of 8 experts, MXFP8: 2048
//   x 4096 8.4 against 15.4 us by pairs; 1024 x 2048 11.2 us with clusters of 8,
//   9.6 by pairs).
//   Else pairs; blocks of 128 rows up to a mean of 80 rows per expert, of 256
//   above (8 experts of 4096 x 4096, MXFP8: mean 64 30.8 against 33.9 us, mean
//   128 42.6 against 36.0).
//   Blocks of 256 rows get two epilogue warps per TMEM lane quarter where the
//   epilogue shows, in two rounds of items at most or with fewer than eight k-tiles (8
//   experts of 1160 x 4608, 2000 rows: NVFP4 17.3 us with one, 16.5 with two; 32
//   of 4096 x 512, 32,768 rows 132 and 109), and always in INT8 and FP8 (the
//   2000 rows in INT8 23.4 and 21.2).  Else one: with block scales two more
//   cost (32 of 4096 x 4096, 32,768 rows, NVFP4 323 us with one, 335 with two).
constexpr int kMaxSplit = 4;
template <int F>
cudaError_t launch_fmt(GroupedParams &p, const GroupedOperands &op, cudaStream_t s) {
    const int sms = sm_count();
    const int64_t ragged = op.rows < op.n_groups ? op.rows : op.n_groups;   // blocks that may be partly filled
    p.n_tiles = p.w_tiles;
    p.max_tiles = (int)(op.rows / 128 + ragged);
    int64_t items = (int64_t)p.max_tiles * p.n_tiles;
    int split = 1;
    while (split < kMaxSplit && items * split * 2 <= sms && p.num_k_tiles >= split * 4) split *= 2;
    if (split > 1) return launch_split<F>(p, (int)items, split, s);
    const bool wide = op.rows > 80 * (int64_t)op.n_groups;
    p.n_tiles = (int)((op.n + 255) / 256);
    if (wide) p.max_tiles = (int)(op.rows / 256 + ragged);
    items = (int64_t)p.max_tiles * p.n_tiles;
    const int clusters = (int)(items < sms / 2 ? items : sms / 2);
    if (!wide) return launch_pair<F, 128, 1>(p, clusters, s);
    if (gg_atoms<F>() == 0 || items <= 2 * clusters || p.num_k_tiles < 8) return launch_pair<F, 256, 2>(p, clusters, s);
    return launch_pair<F, 256, gg_atoms<F>() ? 1 : 2>(p, clusters, s);
}

}  // namespace

cudaError_t launch_qlinear_grouped(const GroupedOperands &op, cudaStream_t s) {
    GroupedParams p;
    memset(&p, 0, sizeof(p));
    const int64_t kbytes = fmt_is4(op.fmt) ? op.k / 2 : op.k;
    const auto SW128 = CU_TENSOR_MAP_SWIZZLE_128B, NOSW = CU_TENSOR_MAP_SWIZZLE_NONE;
    const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, U64 = CU_TENSOR_MAP_DATA_TYPE_UINT64;
    if (!encode_2d(&p.w, U8, op.w_codes, kbytes, op.n * op.n_groups, kbytes, 128, 128, SW128)) return cudaErrorInvalidValue;
    for (int i = 0; i < 4; i++)
        if (!encode_2d(&p.x[i], U8, op.x_codes, kbytes, op.rows, kbytes, 128, 16u << i, SW128)) return cudaErrorInvalidValue;
    p.w_tiles = (int)((op.n + 127) / 128);
    if (fmt_byte_scales(op.fmt)) {
        // scale atoms as rows of 64 x 8 bytes
        const int64_t s_pad = (op.k / fmt_block(op.fmt) + 15) / 16 * 16;
        p.s4 = (int)(s_pad / 4);
        const uint32_t atoms = op.fmt == kNVFP4 ? 4 : op.fmt == kMXFP4 ? 2 : 1;
        const uint64_t w_atoms = (uint64_t)op.n_groups * p.w_tiles * p.s4;
        const uint64_t x_atoms = (uint64_t)grouped_scale_tiles(op.rows, op.n_groups) * p.s4;
        if (!encode_2d(&p.sfw, U64, op.w_scales, 64, w_atoms, 512, 64, atoms, NOSW) ||
            !encode_2d(&p.sfx, U64, op.x_scales, 64, x_atoms, 512, 64, atoms, NOSW))
            return cudaErrorInvalidValue;
    }
    p.offsets = op.offsets;
    p.n_groups = op.n_groups;
    p.rows = (int)op.rows;
    p.x_row_scale = (const float *)op.x_scales;
    p.w_row_scale = (const float *)op.w_scales;
    p.x_ts = op.x_tensor_scale;
    p.w_ts = op.w_tensor_scales;
    p.y = op.y;
    p.n = (int)op.n;
    p.kbytes = (int)kbytes;
    p.num_k_tiles = (int)((kbytes + 127) / 128);
    p.y_bf16 = op.y_bf16;
    p.y_vec = op.n % 8 == 0;   // (y itself is 16-byte aligned)
    p.wait_ns = 2000000000ull;   // 2 s
    const cudaError_t e = error_word_address(&p.err);
    if (e != cudaSuccess) return e;
    switch (op.fmt) {
    case kNVFP4: return launch_fmt<kNVFP4>(p, op, s);
    case kMXFP4: return launch_fmt<kMXFP4>(p, op, s);
    case kMXFP8: return launch_fmt<kMXFP8>(p, op, s);
    case kFP8Tensor: return launch_fmt<kFP8Tensor>(p, op, s);
    case kINT8Row: return launch_fmt<kINT8Row>(p, op, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace mxq
