// experts.cu -- the steps on either side of a grouped product by expert
// (mixture-of-experts linears in the library's formats): the plan that gives
// every (token, choice) its row in expert order, the quantizer that writes
// tokens into that order, and the weighted sum that brings the products back
// to token order.
//
// Expert order: the rows of expert e are [offsets[e], offsets[e + 1]), the
// choices of one expert in token order.  slot[t][i] is the row of token t's
// i-th choice, negative for a dropped one.
#include <cuda_runtime.h>

#include "groups.cuh"
#include "mxq_formats.cuh"
#include "mxq_internal.h"
#include "tc_ptx.cuh"

namespace mxq {
namespace {

// ------------------------------------------------------------------ plan
//
// A stable counting sort without moving any data: slot = offsets[e] + the
// number of earlier choices of e.  A block counts its choices per warp in
// shared memory, turns the counts into starting rows (scan over experts, then
// over the block's warps), and walks its choices again: the choices of one
// expert among 32 consecutive ones are ranked by __match_any_sync, the
// warp's counter carries the rank on.  No atomic decides an order, so the
// plan is the same from run to run.  Up to kPlanOneBlock choices one block
// does it all (one launch); above that a first kernel writes each block's
// counts, and every block of the second sums those of the blocks before it.
// Bound: latency, both memory passes being a few MB.

constexpr int kPlanThreads = 512;   // >= kMaxGroups: a thread per expert in the scan
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanOneBlock = 4096;
constexpr int kPlanBlockRows = 1024;
constexpr int kPlanMaxBlocks = 74;   // half of a B200's 148 SMs (see plan_block_rows); a constant, since the workspace's
                                     // size is asked for without a device
static_assert(kPlanThreads >= kMaxGroups, "one thread per expert");

template <typename I>
__device__ __forceinline__ int expert_at(const I *ids, int64_t i, int64_t end, int n) {
    if (i >= end) return -1;
    const I v = ids[i];
    return v >= 0 && v < (I)n ? (int)v : -1;
}

// Counts of a block lie plan_stride(n) apart: whole 16-byte words.
__host__ __device__ __forceinline__ int plan_stride(int n) { return (n + 3) & ~3; }

template <typename I>
__global__ void __launch_bounds__(kPlanThreads) k_plan_count(const I *__restrict__ ids, int64_t rows, int n,
                                                             int64_t per_block, int32_t *__restrict__ counts) {
    __shared__ int hist[kMaxGroups];
    pdl_wait();
    pdl_launch_dependents();
    for (int e = threadIdx.x; e < n; e += kPlanThreads) hist[e] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * per_block;
    const int64_t end = begin + per_block < rows ? begin + per_block : rows;
    for (int64_t i0 = begin + threadIdx.x; i0 < end; i0 += 4 * kPlanThreads) {
        int e[4];
#pragma unroll
        for (int j = 0; j < 4; j++) e[j] = expert_at(ids, i0 + j * kPlanThreads, end, n);
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (e[j] >= 0) atomicAdd(hist + e[j], 1);
    }
    __syncthreads();
    const int stride = plan_stride(n);
    for (int e = threadIdx.x; e < stride; e += kPlanThreads) counts[(int64_t)blockIdx.x * stride + e] = e < n ? hist[e] : 0;
}

// counts: null with one block, else k_plan_count's.
template <typename I>
__global__ void __launch_bounds__(kPlanThreads)
    k_plan_place(const I *__restrict__ ids, int64_t rows, int n, int64_t per_block, const int32_t *__restrict__ counts,
                 int32_t *__restrict__ offsets, int32_t *__restrict__ slot) {
    __shared__ int at[kPlanWarps][kMaxGroups];   // counts, then the next row, of each warp's choices of each expert
    __shared__ int warp_sum[kPlanWarps];
    __shared__ int all[kMaxGroups], earlier[kMaxGroups];   // choices of each expert in all blocks, and in those before this
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // k_plan_count is the kernel before this one and lets it start only once
    // it has itself waited for the ids: they may be read before the wait
    if (!counts) pdl_wait();
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < kPlanWarps * kMaxGroups; i += kPlanThreads) (&at[0][0])[i] = 0;
    all[threadIdx.x] = earlier[threadIdx.x] = 0;
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * per_block;
    const int64_t end = begin + per_block < rows ? begin + per_block : rows;
    // contiguous choices per warp, whole groups of 32
    const int64_t per_warp = ((end - begin + kPlanThreads - 1) / kPlanThreads) * 32;
    const int64_t w_begin = begin + warp * per_warp;
    const int64_t w_end = w_begin + per_warp < end ? w_begin + per_warp : end;
    int keep[4] = {-1, -1, -1, -1};   // the first 128 choices, for the second walk
    for (int64_t i0 = w_begin; i0 < w_end; i0 += 128) {
        int e[4];
#pragma unroll
        for (int j = 0; j < 4; j++) e[j] = expert_at(ids, i0 + 32 * j + lane, w_end, n);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (e[j] >= 0) atomicAdd(&at[warp][e[j]], 1);   // a count: no order in it
            if (i0 == w_begin) keep[j] = e[j];
        }
    }
    if (counts) {
        pdl_wait();
        // a thread adds four experts' counts over every rows-th block, its loads eight at a time
        const int stride = plan_stride(n), groups = stride / 4, rows_of = kPlanThreads / groups;
        const int g = threadIdx.x % groups, start = threadIdx.x / groups, nb = (int)gridDim.x;
        int4 sum = make_int4(0, 0, 0, 0), pre = sum;
        if (start < rows_of) {
            for (int b0 = start; b0 < nb; b0 += 8 * rows_of) {
                int4 c[8];
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int b = b0 + j * rows_of;
                    c[j] = __ldcg(reinterpret_cast<const int4 *>(counts + (int64_t)(b < nb ? b : 0) * stride) + g);
                    if (b >= nb) c[j] = make_int4(0, 0, 0, 0);
                }
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    sum.x += c[j].x, sum.y += c[j].y, sum.z += c[j].z, sum.w += c[j].w;
                    if (b0 + j * rows_of < (int)blockIdx.x) pre.x += c[j].x, pre.y += c[j].y, pre.z += c[j].z, pre.w += c[j].w;
                }
            }
            atomicAdd(all + 4 * g, sum.x), atomicAdd(all + 4 * g + 1, sum.y);
            atomicAdd(all + 4 * g + 2, sum.z), atomicAdd(all + 4 * g + 3, sum.w);
            atomicAdd(earlier + 4 * g, pre.x), atomicAdd(earlier + 4 * g + 1, pre.y);
            atomicAdd(earlier + 4 * g + 2, pre.z), atomicAdd(earlier + 4 * g + 3, pre.w);
        }
    }
    __syncthreads();
    int own = 0, before = 0, total = 0;
    const int e = threadIdx.x;
    if (e < n) {
#pragma unroll
        for (int w = 0; w < kPlanWarps; w++) own += at[w][e];
        total = own;
        if (counts) {
            total = all[e];
            before = earlier[e];
        }
    }
    // exclusive scan of the totals over the experts
    int scan = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    int first = scan - total;
    for (int w = 0; w < warp; w++) first += warp_sum[w];
    if (e < n) {
        if (blockIdx.x == 0) {
            offsets[e] = first;
            if (e == n - 1) offsets[n] = first + total;
        }
        int next = first + before;
#pragma unroll
        for (int w = 0; w < kPlanWarps; w++) {
            const int c = at[w][e];
            at[w][e] = next;
            next += c;
        }
    }
    __syncthreads();
    const unsigned below = (1u << lane) - 1u, above = ~(below | (1u << lane));
    for (int64_t i0 = w_begin; i0 < w_end; i0 += 128) {
        int ex[4];
#pragma unroll
        for (int j = 0; j < 4; j++) ex[j] = i0 == w_begin ? keep[j] : expert_at(ids, i0 + 32 * j + lane, w_end, n);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const unsigned same = __match_any_sync(0xFFFFFFFFu, ex[j]);
            int r = -1;
            if (ex[j] >= 0) r = at[warp][ex[j]] + __popc(same & below);
            __syncwarp();
            if (ex[j] >= 0 && !(same & above)) at[warp][ex[j]] = r + 1;   // the last of them carries the rank on
            __syncwarp();
            const int64_t i = i0 + 32 * j + lane;
            if (i < w_end) slot[i] = r;
        }
    }
}

// ------------------------------------------------------------------ quantize in expert order
//
// A token is read and coded once and its codes written to the rows of all
// its choices: T K reads and T k K writes, against k times the reads of a
// gather.  A warp takes up to four spans of 32 consecutive 16-element chunks
// of a token (the chunk mapping of k_quantize, so blocks and Hadamard blocks
// lie in aligned lanes); lane i looks up choice i's row and its place in the
// grouped scale layout once for all of them, and the next span's load is in
// flight while one is coded.  Four block scales are gathered into the 4-byte
// word they share in a scale atom.  Bound: HBM.

constexpr int kGqThreads = 256;
constexpr int kGqWarps = kGqThreads / 32;
constexpr uint32_t kGqSpans = 4;
constexpr int kGqMaxCtas = 960;   // per-CTA maxima of the tensor-amax pass

struct GroupedQuantArgs {
    int64_t x_rows, cols, rows;   // rows: capacity of codes and scales
    FastDiv segs;                 // warps' work per token
    uint32_t n_segs, units;       // units = x_rows * n_segs
    uint32_t spans;               // spans of 32 chunks that a unit holds at most
    const int32_t *slot;          // null: token t is row t
    int topk;
    const int32_t *offsets;
    int n_groups;
    int hadamard_b;
    uint32_t s_pad4, scale_tiles;   // padded scale columns / 4, 128-row tiles the scales buffer holds
    uint8_t *codes;
    uint8_t *scales;
    float *tensor_scale;
    float *amax_slots;
    int n_slots;
    unsigned int *err;
};

// Row of choice `lane` of token t (lanes below topk; -1 elsewhere); the other
// form: -1 also for rows outside [first, last).
__device__ __forceinline__ int choice_row(const GroupedQuantArgs &a, uint32_t t, int lane) {
    return lane >= a.topk ? -1 : a.slot ? a.slot[(int64_t)t * a.topk + lane] : (int)t;
}
__device__ __forceinline__ int choice_row(const GroupedQuantArgs &a, uint32_t t, int lane, int first, int last) {
    const int r = choice_row(a, t, lane);
    return r >= first && r < last ? r : -1;
}

template <typename T>
__device__ __forceinline__ void load_or_zero(const T *p, bool valid, float v[16]) {
    if (valid) load16(p, v);
    else {
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] = 0.0f;
    }
}

__device__ __forceinline__ void unpack16(const uint4 (&k)[2], float (&v)[16]) {   // bf16
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t w[4] = {k[i].x, k[i].y, k[i].z, k[i].w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ void unpack16(const uint4 (&k)[4], float (&v)[16]) {   // fp32
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[4 * i] = __uint_as_float(k[i].x);
        v[4 * i + 1] = __uint_as_float(k[i].y);
        v[4 * i + 2] = __uint_as_float(k[i].z);
        v[4 * i + 3] = __uint_as_float(k[i].w);
    }
}

// A chunk as loaded, zeros where there is none.
template <typename T>
struct RawWords {
    uint4 q[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void load_words(RawWords<T> &r, const T *p, bool valid) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); i++)
        r.q[i] = valid ? __ldg(reinterpret_cast<const uint4 *>(p) + i) : make_uint4(0, 0, 0, 0);
}

// max |x| over the tokens that have a row, one maximum per CTA.
template <typename T>
__global__ void __launch_bounds__(kGqThreads) k_amax_grouped(const T *__restrict__ x, GroupedQuantArgs a) {
    __shared__ float wm[kGqWarps];
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int first = clamp_row(a.offsets[0], a.rows), last = clamp_row(a.offsets[a.n_groups], a.rows);
    const float norm = a.hadamard_b ? __frsqrt_rn((float)a.hadamard_b) : 1.0f;
    const uint32_t cpr = (uint32_t)(a.cols >> 4);
    float m = 0.0f;
    for (uint32_t u = blockIdx.x * kGqWarps + (threadIdx.x >> 5); u < a.units; u += gridDim.x * kGqWarps) {
        const uint32_t t = fdiv(u, a.segs), c0 = (u - t * a.n_segs) * a.spans * 32 + lane;
        const int r = choice_row(a, t, lane, first, last);
        if (!__any_sync(0xFFFFFFFFu, r >= 0)) continue;
#pragma unroll
        for (uint32_t j = 0; j < kGqSpans; j++) {
            if (j >= a.spans) break;
            const uint32_t c = c0 + 32 * j;
            float v[16];
            load_or_zero(x + (int64_t)t * a.cols + (int64_t)c * 16, c < cpr, v);
            if (a.hadamard_b) hadamard_chunk_n(v, a.hadamard_b, lane, norm);
            m = fmaxf(m, amax16(v));
        }
    }
    m = group_max<32>(m);
    if (lane == 0) wm[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kGqWarps; w++) m = fmaxf(m, wm[w]);
        a.amax_slots[blockIdx.x] = m;
    }
}

// Formats with byte scales, and FP8 per tensor.
template <typename T, int F>
__global__ void __launch_bounds__(kGqThreads, 4) k_quantize_grouped(const T *__restrict__ x, GroupedQuantArgs a) {
    __shared__ Groups groups;
    __shared__ float wm[kGqWarps];
    const int lane = threadIdx.x & 31;
    constexpr bool kByte = fmt_byte_scales(F);
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t cpr = (uint32_t)(a.cols >> 4);
    const uint32_t step = gridDim.x * kGqWarps, spans_t = (cpr + 31) >> 5;
    uint32_t u = blockIdx.x * kGqWarps + (threadIdx.x >> 5);
    // the span being coded: token t, chunk c of this lane, `left` more spans in the unit
    uint32_t t, c, left;
    auto unit = [&](uint32_t w, uint32_t &wt, uint32_t &wc, uint32_t &wleft) {
        wt = fdiv(w, a.segs);
        const uint32_t s0 = (w - wt * a.n_segs) * a.spans;
        wc = s0 * 32 + lane;
        wleft = (spans_t - s0 < a.spans ? spans_t - s0 : a.spans) - 1;
    };
    // the first span's loads go out before the table is built
    unit(u, t, c, left);
    RawWords<T> next;
    load_words(next, x + (int64_t)t * a.cols + (int64_t)c * 16, u < a.units && c < cpr);
    int next_r = u < a.units ? choice_row(a, t, lane) : -1;
    load_groups(groups, a.offsets, a.n_groups, a.rows, blockIdx.x == 0 ? a.err : nullptr);
    const int first = groups.off[0], last = groups.off[a.n_groups];
    TensorRecip tr;
    Recip rt;
    if (fmt_tensor_scaled(F)) {
        float m = 0.0f;
        for (int i = threadIdx.x; i < a.n_slots; i += kGqThreads) m = fmaxf(m, a.amax_slots[i]);
        m = group_max<32>(m);
        if (lane == 0) wm[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kGqWarps; w++) m = fmaxf(m, wm[w]);
        const float s = F == kNVFP4 ? nvfp4_tensor_scale(m) : fp8_tensor_scale(m);
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.tensor_scale = s;
        if (F == kNVFP4) tr = tensor_recip_of(s);
        else rt = recip_of(s);
    }
    const float norm = a.hadamard_b ? __frsqrt_rn((float)a.hadamard_b) : 1.0f;
    if (u >= a.units) return;
    int r = -1;
    uint32_t sword = 0;      // lane i: the row's first word among the scales
    unsigned any = 0;
    bool fresh = true;       // a new token: look its choices up
    while (true) {
        const bool valid = c < cpr;
        const uint32_t cur = c;
        float v[16];
        unpack16(next.q, v);
        if (fresh) {
            r = next_r >= first && next_r < last ? next_r : -1;
            if (kByte && r >= 0) {   // its group's first tile, then its rank in the group
                const int g = group_of_row(groups, a.n_groups, r);
                const uint32_t sr = g >= 0 ? (uint32_t)(128 * groups.tile[g] + r - groups.off[g]) : 0u;
                if (g < 0 || (sr >> 7) >= a.scale_tiles) r = -1;   // offsets that do not fit the buffers
                sword = (sr >> 7) * a.s_pad4 * 128 + (sr & 31) * 4 + ((sr >> 5) & 3);
            }
            any = __ballot_sync(0xFFFFFFFFu, r >= 0);
        }
        // the next span's load
        fresh = left == 0;
        bool more = true;
        if (!fresh) {
            c += 32;
            left--;
        } else {
            u += step;
            more = u < a.units;
            if (more) {
                unit(u, t, c, left);
                next_r = choice_row(a, t, lane);
            }
        }
        if (more) load_words(next, x + (int64_t)t * a.cols + (int64_t)c * 16, c < cpr);
        if (!any) {
            if (!more) break;
            continue;
        }
        if (a.hadamard_b) hadamard_chunk_n(v, a.hadamard_b, lane, norm);
        uint32_t w[4];        // codes: 16 bytes (8-bit elements) or 8
        uint32_t scale = 0;   // this lane's block scale
        float amax = amax16(v);
        if (F == kMXFP8 || F == kMXFP4) {
            amax = group_max<2>(amax);
            const bool zero = !(amax > 0.0f);
            float inv = 0.0f, q[16];
            scale = zero ? 127u : mx_scale(amax, F == kMXFP8 ? 8 : 2, inv);
            mul8(v, inv, q);   // a power of two: exact
            mul8(v + 8, inv, q + 8);
            if (F == kMXFP8) {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    w[i] = zero ? 0u : cvt_e4m3x4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < 2; i++)
                    w[i] = zero ? 0u : cvt_e2m1x8(q[8 * i], q[8 * i + 1], q[8 * i + 2], q[8 * i + 3], q[8 * i + 4],
                                                  q[8 * i + 5], q[8 * i + 6], q[8 * i + 7]);
            }
        } else if (F == kNVFP4) {
            float d;
            scale = nvfp4_block_scale_fast(amax, tr, d);
            w[0] = w[1] = 0u;
            if (scale) {
                const Recip rd = recip_of(d);
                w[0] = e2m1x8_quot(v, rd);
                w[1] = e2m1x8_quot(v + 8, rd);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) w[i] = e4m3x4_quot(v + 4 * i, rt);
        }
        uint32_t word = 0, col = 0;   // the four scales of an atom's 4-byte word, held by its first lane
        bool leader = false;
        if (kByte) {
            constexpr int L = F == kNVFP4 ? 1 : 2;   // lanes per block
            if (!valid) scale = 0u;
            word = scale | (__shfl_down_sync(0xFFFFFFFFu, scale, L) << 8) |
                   (__shfl_down_sync(0xFFFFFFFFu, scale, 2 * L) << 16) |
                   (__shfl_down_sync(0xFFFFFFFFu, scale, 3 * L) << 24);
            leader = valid && (lane & (4 * L - 1)) == 0;
            col = cur / L;
        }
        uint8_t *codes = a.codes + (int64_t)cur * (fmt_is4(F) ? 8 : 16);
        uint32_t *scales = reinterpret_cast<uint32_t *>(a.scales) + (col >> 2) * 128u;
        const int64_t pitch = (int64_t)cpr * (fmt_is4(F) ? 8 : 16);
        for (unsigned rest = any; rest; rest &= rest - 1) {
            const int i = __ffs(rest) - 1;
            const int row = __shfl_sync(0xFFFFFFFFu, r, i);
            const uint32_t word_at = kByte ? __shfl_sync(0xFFFFFFFFu, sword, i) : 0u;
            if (valid) {
                if (fmt_is4(F)) *reinterpret_cast<uint2 *>(codes + row * pitch) = make_uint2(w[0], w[1]);
                else *reinterpret_cast<uint4 *>(codes + row * pitch) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (kByte && leader) scales[word_at] = word;
        }
        if (!more) break;
    }
}

// INT8 per row: a warp per token; the first 8 chunks of a lane in bf16, 4 in
// fp32 (rows up to 4096 and 2048 elements), stay in registers between the row
// maximum and the codes, what is behind them is read twice.
template <typename T>
__global__ void __launch_bounds__(kGqThreads) k_quantize_grouped_int8(const T *__restrict__ x, GroupedQuantArgs a) {
    constexpr int kKeep = sizeof(T) == 2 ? 8 : 4;
    constexpr int kWords = sizeof(T) * 16 / 16;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int first = clamp_row(a.offsets[0], a.rows), last = clamp_row(a.offsets[a.n_groups], a.rows);
    if (blockIdx.x == 0)   // no scale needs a row's group here: the offsets between are only checked
        for (int i = threadIdx.x; i <= a.n_groups; i += kGqThreads)
            if (offset_wrong(a.offsets, i, a.rows)) latch_index_error(a.err);
    const float norm = a.hadamard_b ? __frsqrt_rn((float)a.hadamard_b) : 1.0f;
    const uint32_t cpr = (uint32_t)(a.cols >> 4), steps = (cpr + 31) / 32;
    for (uint32_t t = blockIdx.x * kGqWarps + (threadIdx.x >> 5); t < (uint32_t)a.x_rows; t += gridDim.x * kGqWarps) {
        const T *xr = x + (int64_t)t * a.cols;
        uint4 keep[kKeep][kWords];
#pragma unroll
        for (int j = 0; j < kKeep; j++) {
            const uint32_t c = j * 32 + lane;
#pragma unroll
            for (int q = 0; q < kWords; q++)
                keep[j][q] = c < cpr ? __ldg(reinterpret_cast<const uint4 *>(xr + (int64_t)c * 16) + q) : make_uint4(0, 0, 0, 0);
        }
        const int r = choice_row(a, t, lane, first, last);
        const unsigned any = __ballot_sync(0xFFFFFFFFu, r >= 0);
        if (!any) continue;
        auto values = [&](uint32_t j, float (&v)[16]) {   // chunk j * 32 + lane, rotated
            const uint32_t c = j * 32 + lane;
            load_or_zero(xr + (int64_t)c * 16, c < cpr, v);
            if (a.hadamard_b) hadamard_chunk_n(v, a.hadamard_b, lane, norm);
        };
        auto kept = [&](const uint4 (&k)[kWords], float (&v)[16]) {
            unpack16(k, v);
            if (a.hadamard_b) hadamard_chunk_n(v, a.hadamard_b, lane, norm);
        };
        float m = 0.0f, v[16];
#pragma unroll
        for (int j = 0; j < kKeep; j++)
            if ((uint32_t)j < steps) {
                kept(keep[j], v);
                m = fmaxf(m, amax16(v));
            }
        for (uint32_t j = kKeep; j < steps; j++) {
            values(j, v);
            m = fmaxf(m, amax16(v));
        }
        m = group_max<32>(m);
        const float s = __fdiv_rn(m, 127.0f);
        const Recip rs = recip_of(s);
        auto store = [&](uint32_t j, const float (&u)[16]) {
            const uint32_t c = j * 32 + lane;
            const uint4 w = make_uint4(int_x4_quot(u, rs, 127), int_x4_quot(u + 4, rs, 127), int_x4_quot(u + 8, rs, 127),
                                       int_x4_quot(u + 12, rs, 127));
            for (unsigned left = any; left; left &= left - 1) {
                const int row = __shfl_sync(0xFFFFFFFFu, r, __ffs(left) - 1);
                if (c < cpr) *reinterpret_cast<uint4 *>(a.codes + ((int64_t)row * cpr + c) * 16) = w;
            }
        };
#pragma unroll
        for (int j = 0; j < kKeep; j++)
            if ((uint32_t)j < steps) {
                kept(keep[j], v);
                store(j, v);
            }
        for (uint32_t j = kKeep; j < steps; j++) {
            values(j, v);
            store(j, v);
        }
        if (r >= 0) reinterpret_cast<float *>(a.scales)[r] = s;
    }
}

// ------------------------------------------------------------------ combine
//
// out[t] = sum over i of weights[t][i] y[slot[t][i]], fp32 FMAs in the order
// of i.  A warp owns up to 1024 neighbouring columns of a token (with few
// tokens 256); lane i reads choice i's row and weight once, and a lane has eight
// 16-byte loads in flight, four vectors of two rows or one of eight.
// Bound: HBM (16,384 tokens x 4 x 4096 in bf16: 98 us, 6.7 TB/s; two rows of
// eight columns a thread, addressed one by one, took 142).

struct CombineArgs {
    int64_t rows, n;
    FastDiv segs;             // warps' worth of columns per token
    uint32_t n_segs, units, n_vec;   // units = tokens * n_segs; n_vec: vectors per token
    const int32_t *slot;
    const float *weights;
    int topk;
    unsigned int *err;
};
template <typename T, int V>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> {
    uint4 q;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { q = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
};
template <>
struct Vec<float, 8> {
    float4 q[2];
    __device__ __forceinline__ void load(const float *p) {
        q[0] = __ldg(reinterpret_cast<const float4 *>(p));
        q[1] = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int j = 0; j < 2; j++) {
            v[4 * j] = q[j].x;
            v[4 * j + 1] = q[j].y;
            v[4 * j + 2] = q[j].z;
            v[4 * j + 3] = q[j].w;
        }
    }
};
template <typename T>
struct Vec<T, 1> {
    T q;
    __device__ __forceinline__ void load(const T *p) { q = __ldg(p); }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = (float)q; }
};
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                               pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store_vec(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float (&v)[1]) { *p = __float2bfloat16_rn(v[0]); }
__device__ __forceinline__ void store_vec(float *p, const float (&v)[1]) { *p = v[0]; }

// STEPS vectors of a lane (a warp takes 32 STEPS neighbouring ones of a token),
// ROWS choices at a time: all their loads before any use.
template <typename T, typename O, int V, int STEPS, int ROWS>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) k_expert_combine(const T *__restrict__ y, O *__restrict__ out, CombineArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    for (uint32_t u = blockIdx.x * 8 + (threadIdx.x >> 5); u < a.units; u += gridDim.x * 8) {
        const uint32_t t = fdiv(u, a.segs), c0 = (u - t * a.n_segs) * (32 * STEPS) + lane;
        int row = -1;   // lane i: choice i's row and weight
        float weight = 1.0f;
        if (lane < a.topk) {
            row = a.slot[(int64_t)t * a.topk + lane];
            if (a.weights) weight = a.weights[(int64_t)t * a.topk + lane];
            if (row >= a.rows) {
                latch_index_error(a.err);
                row = -1;
            }
        }
        unsigned left = __ballot_sync(0xFFFFFFFFu, row >= 0);
        float acc[STEPS][V] = {};
        while (left) {
            Vec<T, V> q[ROWS][STEPS];
            float w[ROWS];
            bool on[ROWS];
#pragma unroll
            for (int i = 0; i < ROWS; i++) {
                on[i] = left != 0;
                const int choice = on[i] ? __ffs(left) - 1 : 0;
                left &= left - 1;
                w[i] = __shfl_sync(0xFFFFFFFFu, weight, choice);
                const T *from = y + (int64_t)__shfl_sync(0xFFFFFFFFu, row, choice) * a.n;
#pragma unroll
                for (int k = 0; k < STEPS; k++)
                    if (on[i] && c0 + 32 * k < a.n_vec) q[i][k].load(from + (int64_t)(c0 + 32 * k) * V);
            }
#pragma unroll
            for (int i = 0; i < ROWS; i++)
#pragma unroll
                for (int k = 0; k < STEPS; k++)
                    if (on[i] && c0 + 32 * k < a.n_vec) {
                        float v[V];
                        q[i][k].get(v);
#pragma unroll
                        for (int j = 0; j < V; j++) acc[k][j] = __fmaf_rn(w[i], v[j], acc[k][j]);
                    }
        }
#pragma unroll
        for (int k = 0; k < STEPS; k++)
            if (c0 + 32 * k < a.n_vec) store_vec(out + (int64_t)t * a.n + (int64_t)(c0 + 32 * k) * V, acc[k]);
    }
}

// ------------------------------------------------------------------ host

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*k)(KArgs...), int64_t grid, int threads, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

// Choices per block of the plan's kernels: all of them up to kPlanOneBlock,
// else kPlanBlockRows, or as many as kPlanMaxBlocks blocks need, in whole
// rounds of the block's warps (128 choices each).  The second kernel's blocks
// start under the first one's; with at most half the SMs for each kernel they
// find free ones, with more they crowd on those that are left (262,144 choices
// over 256 experts: 64 blocks 9.3 us, 80 14.1, 128 11.2; 4 M: 74 blocks 83 us,
// 128 111).
int64_t plan_block_rows(int64_t rows) {
    if (rows <= kPlanOneBlock) return rows;
    const int64_t per = (rows + kPlanMaxBlocks - 1) / kPlanMaxBlocks, round = kPlanWarps * 128;
    return per <= kPlanBlockRows ? kPlanBlockRows : (per + round - 1) / round * round;
}
int plan_blocks(int64_t rows) { return rows <= kPlanOneBlock ? 1 : (int)((rows + plan_block_rows(rows) - 1) / plan_block_rows(rows)); }

template <typename I>
cudaError_t plan(const I *ids, int64_t rows, int n, int32_t *offsets, int32_t *slot, int32_t *counts, cudaStream_t s) {
    const int nb = plan_blocks(rows);
    const int64_t per = plan_block_rows(rows);
    if (nb > 1) {
        const cudaError_t e = launch_pdl(k_plan_count<I>, nb, kPlanThreads, s, ids, rows, n, per, counts);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(k_plan_place<I>, nb, kPlanThreads, s, ids, rows, n, per, (const int32_t *)(nb > 1 ? counts : nullptr),
                      offsets, slot);
}

template <typename T>
cudaError_t quantize_grouped(const T *x, int fmt, GroupedQuantArgs a, cudaStream_t s) {
    const int64_t warps = fmt == kINT8Row ? a.x_rows : (int64_t)a.units;
    int64_t ctas = (warps + kGqWarps - 1) / kGqWarps;
    const int64_t cap = (int64_t)sm_count() * 16;   // blocks build the table of groups each (8 per SM: 39.7 us, 16 39.0, 64 39.0)
    if (ctas > cap) ctas = cap;
    if (ctas < 1) ctas = 1;   // no tokens: the tensor scale is still written
    if (fmt == kINT8Row) return launch_pdl(k_quantize_grouped_int8<T>, ctas, kGqThreads, s, x, a);
    if (fmt_tensor_scaled(fmt)) {
        a.n_slots = (int)(ctas < kGqMaxCtas ? ctas : kGqMaxCtas);
        const cudaError_t e = launch_pdl(k_amax_grouped<T>, a.n_slots, kGqThreads, s, x, a);
        if (e != cudaSuccess) return e;
    }
    switch (fmt) {
    case kMXFP8: return launch_pdl(k_quantize_grouped<T, kMXFP8>, ctas, kGqThreads, s, x, a);
    case kMXFP4: return launch_pdl(k_quantize_grouped<T, kMXFP4>, ctas, kGqThreads, s, x, a);
    case kNVFP4: return launch_pdl(k_quantize_grouped<T, kNVFP4>, ctas, kGqThreads, s, x, a);
    default: return launch_pdl(k_quantize_grouped<T, kFP8Tensor>, ctas, kGqThreads, s, x, a);
    }
}

template <typename T, typename O, int V>
cudaError_t combine(const void *y, void *out, CombineArgs a, int64_t tokens, cudaStream_t s) {
    // four vectors a lane where that still gives every SM 16 warps, else one
    // (32 tokens x 8 x 4096: 4.8 us with four, 2.1 with one)
    const int64_t wide = (a.n_vec + 127) / 128, sms = sm_count();
    const bool few = tokens * wide < sms * 16;
    const int64_t segs = few ? (a.n_vec + 31) / 32 : wide;
    a.segs = make_fastdiv((uint32_t)segs);
    a.n_segs = (uint32_t)segs;
    a.units = (uint32_t)(tokens * segs);
    int64_t ctas = ((int64_t)a.units + 7) / 8;
    if (ctas > sms * 64) ctas = sms * 64;
    if (few) return launch_pdl(k_expert_combine<T, O, V, 1, 8>, ctas, 256, s, (const T *)y, (O *)out, a);
    return launch_pdl(k_expert_combine<T, O, V, 4, 2>, ctas, 256, s, (const T *)y, (O *)out, a);
}

}  // namespace

size_t plan_workspace_bytes(int64_t rows, int n_experts) {
    const int nb = plan_blocks(rows);
    return nb > 1 ? (size_t)nb * plan_stride(n_experts) * 4 : 0;
}

cudaError_t launch_expert_plan(const void *ids, bool ids64, int64_t rows, int n_experts, int32_t *offsets, int32_t *slot,
                               int32_t *counts, cudaStream_t s) {
    return ids64 ? plan((const int64_t *)ids, rows, n_experts, offsets, slot, counts, s)
                 : plan((const int32_t *)ids, rows, n_experts, offsets, slot, counts, s);
}

cudaError_t launch_quantize_grouped(const void *x, bool bf16, int64_t x_rows, int64_t cols, int fmt, int hadamard_b,
                                    const int32_t *offsets, int n_groups, const int32_t *slot, int topk, int64_t rows,
                                    void *codes, void *scales, float *tensor_scale, float *amax_slots, cudaStream_t s) {
    GroupedQuantArgs a = {};
    // a warp takes four spans of a token where that still gives every SM 32 warps, else one
    const int64_t spans_t = (cols / 16 + 31) / 32;
    a.spans = x_rows * ((spans_t + kGqSpans - 1) / kGqSpans) >= (int64_t)sm_count() * 32 ? kGqSpans : 1;
    const int64_t segs = (spans_t + a.spans - 1) / a.spans;
    a.x_rows = x_rows;
    a.cols = cols;
    a.rows = rows;
    a.segs = make_fastdiv((uint32_t)segs);
    a.n_segs = (uint32_t)segs;
    a.units = (uint32_t)(x_rows * segs);
    a.slot = slot;
    a.topk = topk;
    a.offsets = offsets;
    a.n_groups = n_groups;
    a.hadamard_b = hadamard_b;
    const int blk = fmt_block(fmt);
    if (fmt_byte_scales(fmt)) a.s_pad4 = (uint32_t)((cols / blk + 15) / 16 * 4);
    a.scale_tiles = (uint32_t)grouped_scale_tiles(rows, n_groups);
    a.codes = (uint8_t *)codes;
    a.scales = (uint8_t *)scales;
    a.tensor_scale = tensor_scale;
    a.amax_slots = amax_slots;
    const cudaError_t e = error_word_address(&a.err);
    if (e != cudaSuccess) return e;
    return bf16 ? quantize_grouped((const __nv_bfloat16 *)x, fmt, a, s) : quantize_grouped((const float *)x, fmt, a, s);
}

cudaError_t launch_expert_combine(const void *y, bool y_bf16, int64_t rows, int64_t n, const int32_t *slot,
                                  const float *weights, int64_t tokens, int topk, void *out, bool out_bf16,
                                  cudaStream_t s) {
    CombineArgs a = {};
    // 8 columns a thread where every row starts on a 16-byte boundary, else one
    const bool vec = n % 8 == 0 && ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
    const int64_t per_row = vec ? n / 8 : n;
    a.rows = rows;
    a.n = n;
    a.n_vec = (uint32_t)per_row;
    a.slot = slot;
    a.weights = weights;
    a.topk = topk;
    const cudaError_t e = error_word_address(&a.err);
    if (e != cudaSuccess) return e;
    using bf = __nv_bfloat16;
    if (y_bf16) {
        if (out_bf16) return vec ? combine<bf, bf, 8>(y, out, a, tokens, s) : combine<bf, bf, 1>(y, out, a, tokens, s);
        return vec ? combine<bf, float, 8>(y, out, a, tokens, s) : combine<bf, float, 1>(y, out, a, tokens, s);
    }
    if (out_bf16) return vec ? combine<float, bf, 8>(y, out, a, tokens, s) : combine<float, bf, 1>(y, out, a, tokens, s);
    return vec ? combine<float, float, 8>(y, out, a, tokens, s) : combine<float, float, 1>(y, out, a, tokens, s);
}

}  // namespace mxq
