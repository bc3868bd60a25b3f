// gemm_grouped.cu -- products of rows in expert order with their expert's
// low-bit weight, for few rows per expert (a decode step, a small batch): the
// memory-bound end, where every busy expert's weight has to be read once and
// the tensor cores have time to spare.  gemm.cu's grouped kernel takes over
// where experts have many rows.
//
// The product is turned round: the weight is the 128-row operand of a
// cta_group::1 MMA and the rows of one expert are its N = 16 .. 128 columns,
// N being the expert's rows rounded up to 16 (up to 128 at a time).  So a
// tile reads no more of X than there is, and the ring's bytes are nearly all
// weight.  Per CTA:
//   warp 0      TMA producer into a 5-stage ring: 128 weight rows x 128 bytes,
//               16 / 32 / 64 / 128 rows of X by the box that fits, scale atoms
//   warp 1      TMEM allocation and the thread that issues the MMAs
//   warps 2-5   epilogue: TMEM -> shared staging [32 rows][128 features] ->
//               scaled rows of y
//   warps 6-    a thread per scale atom of a stage that copies it (X's and
//               W's) to TMEM, each stage having its own columns: a tcgen05.cp
//               holds up the thread that issues it, and NVFP4 has eight a
//               stage (one token, 8 of 64 experts, 2048 x 4096: 15.1 us with
//               the MMA thread issuing them)
// The kernel is persistent over items (expert, 128 features, 128 rows); an
// expert's row blocks of one weight tile are neighbours, so the weight's
// second read is served by L2.  Two accumulator stages let an item's loads and
// MMAs run under the epilogue of the one before.
//
// With fewer items than SMs, K is split over a cluster of 2, 4 or 8 CTAs.
// Each leaves its partial sums in its staging buffer and adds a share of the
// rows from all of them over distributed shared memory, in rank order: no
// atomics, no workspace, the same bits from run to run.  INT8 partials are
// added as integers.
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

constexpr int GN_STAGES = 5;
constexpr int GN_W = 128 * 128;        // 128 weight rows x 128 bytes of K
constexpr int GN_X = 128 * 128;        // up to 128 rows of X
constexpr int GN_SF = 2048;            // up to 4 scale atoms of 512 bytes, for W and for X
constexpr int GN_STAGE = GN_W + GN_X + 2 * GN_SF;
constexpr int GN_STAGING = 32 * 128 * 4;
constexpr int GN_SMEM = GN_STAGES * GN_STAGE + GN_STAGING + (int)sizeof(Groups) + 256 + 1024;
constexpr uint32_t GN_TMEM_COLS = 512;
constexpr uint32_t GN_TMEM_SF = 256;   // two 128-column accumulators, then 32 columns of scales per stage
static_assert(GN_TMEM_SF + 32 * GN_STAGES <= GN_TMEM_COLS, "TMEM budget");
static_assert(GN_SMEM <= 227 * 1024, "shared memory budget");
constexpr unsigned int kErrGrouped = 512u;

struct GroupedParams {
    CUtensorMap w, sfw, sfx, x[4];   // x[i]: boxes of 16 << i rows
    const int32_t *offsets;
    int n_groups, rows;
    const float *x_row_scale, *w_row_scale;   // INT8
    const float *x_ts, *w_ts;                 // NVFP4, FP8: X's scalar, one per expert
    void *y;
    int n, kbytes, num_k_tiles, s4, n_tiles, max_tiles, y_bf16, y_vec;
    unsigned int *err;
    unsigned long long wait_ns;
};

__device__ __forceinline__ void tma_load_2d(const CUtensorMap *map, void *dst, uint64_t *bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_cp(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
// One 512-byte scale atom for tcgen05.cp: no swizzle, 8-row core matrices 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_atom(const void *p) {
    return (uint64_t)((smem_u32(p) >> 4) & 0x3FFFu) | (8ull << 32) | (1ull << 46);
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int F>
__host__ __device__ constexpr int gn_atoms() { return F == kNVFP4 ? 4 : F == kMXFP4 ? 2 : F == kMXFP8 ? 1 : 0; }
template <int F>
__host__ __device__ constexpr int gn_threads() { return 192 + 32 * gn_atoms<F>(); }
template <int F>
__host__ __device__ constexpr uint32_t gn_idesc() {   // M = 128, K-major operands; N is or-ed in
    return (8u << 24) | (F == kNVFP4   ? (1u << 7) | (1u << 10)                 // E2M1, UE4M3 scales
                         : F == kMXFP4 ? (1u << 7) | (1u << 10) | (1u << 23)    // E2M1, UE8M0 scales
                         : F == kMXFP8 ? (1u << 23)                             // E4M3, UE8M0 scales
                         : F == kFP8Tensor ? (1u << 4)                          // E4M3 -> fp32
                                           : (2u << 4) | (1u << 7) | (1u << 10));   // s8 -> s32
}

// One 32-byte k-step; sf: the stage's scale columns (8 per atom: W's 4, X's 4).
template <int F>
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t sf, int ks) {
    if (F == kNVFP4) {
        const uint32_t s = sf + 8 * ks;
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(s), "r"(s + 4));
    } else if (F == kMXFP4) {   // an atom serves two k-steps: its scale columns 0-1, then 2-3
        const uint32_t s = sf + 8 * (ks >> 1), id = (uint32_t)((ks & 1) * 2);
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc | (id << 29) | (id << 4)), "r"(acc), "r"(s), "r"(s + 4));
    } else if (F == kMXFP8) {   // an atom serves four
        const uint32_t id = (uint32_t)ks;
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc | (id << 29) | (id << 4)), "r"(acc), "r"(sf), "r"(sf + 4));
    } else if (F == kFP8Tensor) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc));
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc));
    }
}

// An item: 128 features of an expert times up to 128 of its rows.
struct Item {
    int group, tile_n, row0, n_rows, sf_tile;
};
__device__ __forceinline__ Item item_at(const Groups &g, int n_groups, int n_tiles, int item) {
    const int key = item / n_tiles;   // the item's row block, counted over all groups
    int lo = 0, hi = n_groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (g.tile[mid] <= key) lo = mid;
        else hi = mid;
    }
    const int blocks = g.tile[lo + 1] - g.tile[lo], within = item - g.tile[lo] * n_tiles;
    Item it;
    it.group = lo;
    it.tile_n = within / blocks;
    const int block = within - it.tile_n * blocks;
    it.row0 = g.off[lo] + block * 128;
    const int left = g.off[lo + 1] - it.row0;
    it.n_rows = left < 128 ? left : 128;
    it.sf_tile = g.tile[lo] + block;
    return it;
}

template <int F>
__global__ void __launch_bounds__(gn_threads<F>(), 1) k_gemm_grouped_few(const __grid_constant__ GroupedParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint32_t *staging = reinterpret_cast<uint32_t *>(smem + GN_STAGES * GN_STAGE);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + GN_STAGES * GN_STAGE + GN_STAGING);
    uint64_t *empty = full + GN_STAGES;
    uint64_t *accf = empty + GN_STAGES;   // [2] accumulator stage full
    uint64_t *acce = accf + 2;            // [2] accumulator stage drained
    uint64_t *ready = acce + 2;           // partial sums of every CTA of the cluster in its staging
    uint64_t *freed = ready + 1;          // and read by all of them
    uint64_t *drain = freed + 1;
    uint64_t *sfready = drain + 1;        // [GN_STAGES] a stage's scales in TMEM
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sfready + GN_STAGES);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    Groups &groups = *reinterpret_cast<Groups *>(smem + GN_STAGES * GN_STAGE + GN_STAGING + 256);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t split;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    const uint32_t rank = cluster_rank();
    const int cid = (int)cluster_id(), ncl = (int)cluster_count();
    constexpr int NSF = gn_atoms<F>();

    if (warp == 0 && lane < 7) {
        const CUtensorMap *m = lane < 4 ? p.x + lane : lane == 4 ? &p.w : lane == 5 ? &p.sfw : &p.sfx;
        if (lane < 5 || NSF) asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < GN_STAGES; s++) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
            mbar_init(sfready + s, NSF ? NSF : 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(accf + i, 1);
            mbar_init(acce + i, 4);
        }
        mbar_init(ready, 4 * split);
        mbar_init(freed, 4 * split);
        mbar_init(drain, 1 + NSF);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(GN_TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    if (split > 1) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();
    load_groups(groups, p.offsets, p.n_groups, p.rows, blockIdx.x == 0 ? p.err : nullptr);

    const int tiles = groups.tile[p.n_groups];   // above max_tiles only for offsets out of order
    const int items = (tiles < p.max_tiles ? tiles : p.max_tiles) * p.n_tiles;
    const int kt0 = (int)((int64_t)p.num_k_tiles * rank / split), kt1 = (int)((int64_t)p.num_k_tiles * (rank + 1) / split);

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (int item = cid; item < items && !*abort_flag; item += ncl) {
                const Item w = item_at(groups, p.n_groups, p.n_tiles, item);
                const int box = w.n_rows <= 16 ? 0 : w.n_rows <= 32 ? 1 : w.n_rows <= 64 ? 2 : 3;
                const uint32_t bytes = GN_W + ((16u << box) * 128u) + NSF * 1024u;
                for (int kt = kt0; kt < kt1; kt++, it++) {
                    const int s = it % GN_STAGES;
                    if (!mbar_wait(empty + s, ((it / GN_STAGES) & 1) ^ 1, p.wait_ns)) {
                        atomicOr(p.err, kErrGrouped);
                        *abort_flag = 1;
                    }
                    if (*abort_flag) break;
                    uint8_t *sw = smem + s * GN_STAGE;
                    mbar_arrive_expect_tx(full + s, bytes);
                    tma_load_2d(&p.w, sw, full + s, kt * 128, w.group * p.n + w.tile_n * 128);
                    tma_load_2d(&p.x[box], sw + GN_W, full + s, kt * 128, w.row0);
                    if (NSF) {
                        tma_load_2d(&p.sfw, sw + GN_W + GN_X, full + s, 0, (w.group * p.n_tiles + w.tile_n) * p.s4 + kt * NSF);
                        tma_load_2d(&p.sfx, sw + GN_W + GN_X + GN_SF, full + s, 0, w.sf_tile * p.s4 + kt * NSF);
                    }
                }
            }
            if (*abort_flag)   // wait (bounded) for the loads that may still be in flight
                for (int i = (it > GN_STAGES ? it - GN_STAGES : 0); i < it; i++)
                    mbar_wait(full + (i % GN_STAGES), (i / GN_STAGES) & 1, p.wait_ns);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int it = 0, count = 0;
            const uint64_t ad0 = sdesc_sw128(smem), bd0 = sdesc_sw128(smem + GN_W);
            for (int item = cid; item < items && !*abort_flag; item += ncl, count++) {
                const Item w = item_at(groups, p.n_groups, p.n_tiles, item);
                const uint32_t idesc = gn_idesc<F>() | ((uint32_t)((w.n_rows + 15) >> 4) << 18);   // N / 8 at bit 17
                const int st = count & 1;
                const uint32_t acc = tmem + 128u * st;
                bool ok = mbar_wait_spin(acce + st, ((count >> 1) & 1) ^ 1, p.wait_ns);
                tc_fence_after();
                for (int kt = kt0; kt < kt1 && ok && !*abort_flag; kt++, it++) {
                    const int s = it % GN_STAGES;
                    ok = mbar_wait_spin(NSF ? sfready + s : full + s, (it / GN_STAGES) & 1, p.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sft = tmem + GN_TMEM_SF + 32u * s;
                    const int left = (p.kbytes - kt * 128) >> 5, nks = left < 4 ? left : 4;
                    const uint64_t off = (uint64_t)(s * (GN_STAGE >> 4));
#pragma unroll
                    for (int ks = 0; ks < 4; ks++)
                        if (ks < nks)
                            mma_step<F>(acc, ad0 + off + 2 * ks, bd0 + off + 2 * ks, idesc, kt > kt0 || ks > 0, sft, ks);
                    tc_commit(empty + s);
                }
                if (!ok) {
                    atomicOr(p.err, kErrGrouped);
                    *abort_flag = 1;
                }
                if (*abort_flag) break;
                tc_commit(accf + st);
            }
            if (*abort_flag) {   // what is in flight lands before the TMEM is freed
                tc_commit(drain);
                mbar_wait(drain, 0, p.wait_ns);
            }
        }
    } else if (warp >= 6) {
        const int atom = warp - 6;
        if (lane == 0) {
            int it = 0;
            for (int item = cid; item < items && !*abort_flag; item += ncl) {
                for (int kt = kt0; kt < kt1; kt++, it++) {
                    const int s = it % GN_STAGES;
                    if (!mbar_wait(full + s, (it / GN_STAGES) & 1, p.wait_ns)) {
                        atomicOr(p.err, kErrGrouped);
                        *abort_flag = 1;
                    }
                    if (*abort_flag) break;
                    tc_fence_after();
                    // atoms of 32-byte k-steps: 4 (NVFP4: one each), 2 or 1 a stage, fewer in the last
                    if (atom * (4 / (NSF ? NSF : 1)) * 32 < p.kbytes - kt * 128) {
                        const uint8_t *sf = smem + s * GN_STAGE + GN_W + GN_X + 512 * atom;
                        const uint32_t to = tmem + GN_TMEM_SF + 32u * s + 8u * atom;
                        tc_cp(to, sdesc_atom(sf));
                        tc_cp(to + 4, sdesc_atom(sf + GN_SF));
                    }
                    tc_commit(sfready + s);
                }
            }
            if (*abort_flag) {
                tc_commit(drain);
                mbar_wait(drain, 0, p.wait_ns);
            }
        }
    } else {
        const int q = warp & 3, feature = q * 32 + lane;   // TMEM lane quarter and lane
        const int et = threadIdx.x - 64;                   // 0 .. 127 among the epilogue threads
        int count = 0;
        uint32_t chunks = 0;   // staging rounds done
        bool ok = true;
        for (int item = cid; item < items; item += ncl, count++) {
            const Item w = item_at(groups, p.n_groups, p.n_tiles, item);
            const int st = count & 1;
            ok = ok && !*abort_flag && mbar_wait(accf + st, (count >> 1) & 1, p.wait_ns);
            // all 128 threads go on or none does: they meet at barriers below
            int all;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbar.red.and.pred q, 2, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
                : "=r"(all)
                : "r"((int)ok)
                : "memory");
            if (!all) {
                if (!ok && !*abort_flag) atomicOr(p.err, kErrGrouped);
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            float alpha = 1.0f;
            if (F == kNVFP4 || F == kFP8Tensor) alpha = __fmul_rn(__ldg(p.x_ts), __ldg(p.w_ts + w.group));
            const int n0 = w.tile_n * 128, n_chunks = (w.n_rows + 31) >> 5;
            for (int c = 0; c < n_chunks; c++, chunks++) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld_32x32b_x32(tmem + ((uint32_t)(q * 32) << 16) + 128u * st + 32u * c, r);
                if (c == n_chunks - 1) {   // the accumulator stage is drained
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_local_relaxed(acce + st);
                }
                // the staging of the round before has been read, here and by the cluster
                if (split == 1) epilogue_sync();
                else if (chunks > 0 && ok) ok = mbar_wait<true>(freed, (chunks - 1) & 1, p.wait_ns);
#pragma unroll
                for (int j = 0; j < 32; j++) staging[j * 128 + feature] = r[j];
                if (split == 1) {
                    epilogue_sync();
                } else {
                    __syncwarp();
                    if (lane < (int)split) mbar_arrive_remote(map_to_rank(ready, lane));
                    if (ok) ok = mbar_wait<true>(ready, chunks & 1, p.wait_ns);
                }
                // rows rank * 32 / split .. of the chunk, 8 features per thread
                const int per = 32 / (int)split, v8 = et & 15;
                for (int j = et >> 4; j < per && ok; j += 8) {
                    const int jr = (int)rank * per + j, row = w.row0 + c * 32 + jr;
                    if (c * 32 + jr >= w.n_rows) break;
                    const uint32_t *src = staging + jr * 128 + v8 * 8;
                    float v[8];
                    if (split == 1) {
                        const uint4 a = *reinterpret_cast<const uint4 *>(src), b = *reinterpret_cast<const uint4 *>(src + 4);
                        const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int i = 0; i < 8; i++) v[i] = F == kINT8Row ? (float)(int)u[i] : __uint_as_float(u[i]);
                    } else {
                        int vi[8] = {};
#pragma unroll
                        for (int i = 0; i < 8; i++) v[i] = 0.0f;
                        for (uint32_t s = 0; s < split; s++) {
                            const uint32_t at = map_to_rank(src, s);
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
                    }
                    const int col = n0 + v8 * 8;
                    if (F == kINT8Row) {
                        const float xs = __ldg(p.x_row_scale + row);
                        const float *ws = p.w_row_scale + (int64_t)w.group * p.n + col;
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            v[i] = __fmul_rn(__fmul_rn(v[i], xs), col + i < p.n ? __ldg(ws + i) : 0.0f);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; i++) v[i] = __fmul_rn(v[i], alpha);
                    }
                    const int64_t at = (int64_t)row * p.n + col;
                    if (p.y_bf16) {
                        __nv_bfloat16 *y = reinterpret_cast<__nv_bfloat16 *>(p.y) + at;
                        if (p.y_vec && col + 8 <= p.n) {
                            *reinterpret_cast<uint4 *>(y) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                       pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; i++)
                                if (col + i < p.n) y[i] = __float2bfloat16_rn(v[i]);
                        }
                    } else {
                        float *y = reinterpret_cast<float *>(p.y) + at;
                        if (p.y_vec && col + 8 <= p.n) {
                            reinterpret_cast<float4 *>(y)[0] = make_float4(v[0], v[1], v[2], v[3]);
                            reinterpret_cast<float4 *>(y)[1] = make_float4(v[4], v[5], v[6], v[7]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; i++)
                                if (col + i < p.n) y[i] = v[i];
                        }
                    }
                }
                if (split > 1) {
                    __syncwarp();
                    if (lane < (int)split) mbar_arrive_remote(map_to_rank(freed, lane));
                }
            }
            if (!ok) {
                if (!*abort_flag) atomicOr(p.err, kErrGrouped);
                *abort_flag = 1;
            }
        }
    }

    tc_fence_before();
    if (split > 1) cluster_sync();   // no CTA leaves while another may read its staging
    else __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(GN_TMEM_COLS));
    }
}

// ------------------------------------------------------------------ host

template <int F>
cudaError_t launch_few(const GroupedParams &p, int clusters, int split, cudaStream_t s) {
    static PerDeviceOnce smem_opt_in;
    cudaError_t e = smem_opt_in.run([] {
        return cudaFuncSetAttribute(k_gemm_grouped_few<F>, cudaFuncAttributeMaxDynamicSharedMemorySize, GN_SMEM);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * split), 1, 1);
    cfg.blockDim = dim3(gn_threads<F>(), 1, 1);
    cfg.dynamicSmemBytes = GN_SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2] = {pdl_attribute()};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_gemm_grouped_few<F>, p);
}

}  // namespace

static cudaError_t launch_qlinear_grouped_few(const GroupedOperands &op, cudaStream_t s) {
    GroupedParams p;
    memset(&p, 0, sizeof(p));
    const int64_t kbytes = fmt_is4(op.fmt) ? op.k / 2 : op.k;
    const auto SW128 = CU_TENSOR_MAP_SWIZZLE_128B, NOSW = CU_TENSOR_MAP_SWIZZLE_NONE;
    const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, U64 = CU_TENSOR_MAP_DATA_TYPE_UINT64;
    p.n_tiles = (int)((op.n + 127) / 128);
    p.max_tiles = (int)grouped_scale_tiles(op.rows, op.n_groups);
    if (!encode_2d(&p.w, U8, op.w_codes, kbytes, op.n * op.n_groups, kbytes, 128, 128, SW128)) return cudaErrorInvalidValue;
    for (int i = 0; i < 4; i++)
        if (!encode_2d(&p.x[i], U8, op.x_codes, kbytes, op.rows, kbytes, 128, 16u << i, SW128)) return cudaErrorInvalidValue;
    if (fmt_byte_scales(op.fmt)) {
        // scale atoms as rows of 64 x 8 bytes
        const int64_t s_pad = (op.k / fmt_block(op.fmt) + 15) / 16 * 16;
        p.s4 = (int)(s_pad / 4);
        const uint32_t atoms = op.fmt == kNVFP4 ? 4 : op.fmt == kMXFP4 ? 2 : 1;
        if (!encode_2d(&p.sfw, U64, op.w_scales, 64, (uint64_t)op.n_groups * p.n_tiles * p.s4, 512, 64, atoms, NOSW) ||
            !encode_2d(&p.sfx, U64, op.x_scales, 64, (uint64_t)p.max_tiles * p.s4, 512, 64, atoms, NOSW))
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
    p.y_vec = op.n % 8 == 0 && (reinterpret_cast<uintptr_t>(op.y) & 15u) == 0;
    p.wait_ns = 2000000000ull;   // 2 s
    cudaError_t e = error_word_address(&p.err);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    // K is split while the items at most (the host does not know the rows of each expert) leave SMs idle and every
    // CTA keeps at least two stages
    const int64_t items = (int64_t)p.max_tiles * p.n_tiles;
    int split = 1;
    while (split < 8 && items * split * 2 <= sms && p.num_k_tiles >= split * 4) split *= 2;
    const int clusters = (int)(items < sms / split ? items : sms / split);
    switch (op.fmt) {
    case kNVFP4: return launch_few<kNVFP4>(p, clusters, split, s);
    case kMXFP4: return launch_few<kMXFP4>(p, clusters, split, s);
    case kMXFP8: return launch_few<kMXFP8>(p, clusters, split, s);
    case kFP8Tensor: return launch_few<kFP8Tensor>(p, clusters, split, s);
    case kINT8Row: return launch_few<kINT8Row>(p, clusters, split, s);
    default: return cudaErrorInvalidValue;
    }
}

// The host knows the rows of all experts together, not of each: their mean
// decides.
cudaError_t launch_qlinear_grouped(const GroupedOperands &op, cudaStream_t s) {
    if (op.rows > 64 * (int64_t)op.n_groups) return launch_qlinear_grouped_many(op, s);
    return launch_qlinear_grouped_few(op, s);
}

}  // namespace mxq
