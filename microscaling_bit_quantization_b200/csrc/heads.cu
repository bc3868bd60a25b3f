// heads.cu -- norm of every query and key head with the position rotation in
// the same pass: the step between a block's q/k/v linear and its attention,
// written back in 16 or 32 bits, or rotated by a Hadamard matrix and quantized
// for a low-bit cache.
//
// Per head x of D elements: v = (x - mean) r w with r = 1/sqrt(mean square +
// eps) (the mean taken off only for MXQ_NORM_LAYER), then the pairs (a, b) of
// the first `rot` elements become (a c - b s, b c + a s) with the cosine and
// sine of the token's position, in fp32, rounded once on output.
//
// Work mapping.  A lane holds 8 elements of a head, chosen so that it holds
// both ends of its pairs: 8 consecutive ones when pairs are neighbours
// (interleaved) or lie behind `rot`, else 4 of the first and the 4 partners of
// the second half.  A head takes U = D / 8 neighbouring lanes, a warp
// floor(32 / U) heads at a time, all of one token, so a lane's four angles
// are loaded once and serve every head it meets (they would otherwise be
// read twice as often as the data).  Sums run over the U lanes by a shuffle
// tree.  Bound: HBM; the next heads' loads are in flight while the present
// ones are normed.
#include <cuda_runtime.h>

#include "groups.cuh"
#include "mxq_formats.cuh"
#include "mxq_internal.h"
#include "tc_ptx.cuh"

namespace mxq {
namespace {

constexpr int kHeadThreads = 128;
constexpr int kHeadWarps = kHeadThreads / 32;

struct HeadKernelArgs {
    HeadArgs h;
    int units;              // lanes per head
    int per_pass;           // heads a warp takes at a time
    int passes, per_item;   // passes over a token's heads, and how many of them one warp does
    int items;              // warps per token
    unsigned int *err;
};

// Sum over the `units` lanes of a head; `u` is this lane's place among them
// (lanes past the last head have u >= units and take no part).
__device__ __forceinline__ float head_sum(float x, int u, int units, int lane) {
    for (int o = units > 16 ? 16 : units > 8 ? 8 : units > 4 ? 4 : units > 2 ? 2 : 1; o > 0; o >>= 1) {
        const float y = __shfl_down_sync(0xFFFFFFFFu, x, o);
        if (u < o && u + o < units) x += y;
    }
    return __shfl_sync(0xFFFFFFFFu, x, lane - u);
}

struct Raw4 {   // four elements as loaded
    uint4 w;
};
__device__ __forceinline__ void load4(Raw4 &r, const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    r.w.x = v.x;
    r.w.y = v.y;
}
__device__ __forceinline__ void load4(Raw4 &r, const float *p) { r.w = *reinterpret_cast<const uint4 *>(p); }
template <typename T>
__device__ __forceinline__ void unpack4(const Raw4 &r, float *v) {
    if (sizeof(T) == 2) {
        v[0] = __uint_as_float(r.w.x << 16);
        v[1] = __uint_as_float(r.w.x & 0xFFFF0000u);
        v[2] = __uint_as_float(r.w.y << 16);
        v[3] = __uint_as_float(r.w.y & 0xFFFF0000u);
    } else {
        v[0] = __uint_as_float(r.w.x);
        v[1] = __uint_as_float(r.w.y);
        v[2] = __uint_as_float(r.w.z);
        v[3] = __uint_as_float(r.w.w);
    }
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float *v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void store4(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Where a lane's two groups of four elements lie in its head, and its angles.
struct LanePlace {
    int p0, p1;
    bool turned;
    float c[4], s[4];
};
__device__ __forceinline__ LanePlace place_of(const HeadArgs &h, int u, int64_t pos) {
    LanePlace q;
    q.turned = 8 * u < h.rot;
    const bool split = q.turned && !h.interleaved;
    q.p0 = split ? 4 * u : 8 * u;
    q.p1 = split ? h.rot / 2 + 4 * u : 8 * u + 4;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        q.c[i] = 1.0f;
        q.s[i] = 0.0f;
    }
    if (q.turned) {
        const int64_t at = pos * (h.rot / 2) + 4 * u;
        const float4 c = __ldg(reinterpret_cast<const float4 *>(h.cos_t + at));
        const float4 s = __ldg(reinterpret_cast<const float4 *>(h.sin_t + at));
        q.c[0] = c.x; q.c[1] = c.y; q.c[2] = c.z; q.c[3] = c.w;
        q.s[0] = s.x; q.s[1] = s.y; q.s[2] = s.z; q.s[3] = s.w;
    }
    return q;
}

__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float x = a, y = b;
    a = fmaf(x, c, -(y * s));
    b = fmaf(y, c, x * s);
}

// Norm and rotation of a lane's 8 elements v (group 0 then group 1).
__device__ __forceinline__ void norm_rotate(float (&v)[8], const HeadArgs &h, const LanePlace &q, const float *w, int u,
                                            int units, int lane, bool on) {
    const float inv_d = 1.0f / (float)h.head_dim;
    if (h.norm == 1) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) sum += v[i];
        const float mean = head_sum(sum, u, units, lane) * inv_d;
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] -= mean;
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) sq = fmaf(v[i], v[i], sq);
    const float r = rsqrtf(fmaf(head_sum(sq, u, units, lane), inv_d, h.eps));
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] *= r;
    if (w && on) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(w + q.p0)), b = __ldg(reinterpret_cast<const float4 *>(w + q.p1));
        v[0] *= a.x; v[1] *= a.y; v[2] *= a.z; v[3] *= a.w;
        v[4] *= b.x; v[5] *= b.y; v[6] *= b.z; v[7] *= b.w;
    }
    if (q.turned) {
        if (h.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; i++) turn(v[2 * i], v[2 * i + 1], q.c[i], q.s[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) turn(v[i], v[i + 4], q.c[i], q.s[i]);
        }
    }
}

// The position of token t, or -1 (reported) for one outside the tables.
__device__ __forceinline__ int64_t position_of(const HeadArgs &h, int64_t t, unsigned int *err) {
    const int64_t pos = !h.positions ? t
                        : h.pos64    ? static_cast<const int64_t *>(h.positions)[t]
                                     : (int64_t)static_cast<const int32_t *>(h.positions)[t];
    if (h.rot == 0 || (pos >= 0 && pos < h.n_pos)) return pos;
    latch_index_error(err);
    return -1;
}

template <typename T>
__global__ void __launch_bounds__(kHeadThreads) k_qk_norm_rope(HeadKernelArgs a) {
    const HeadArgs &h = a.h;
    const int lane = threadIdx.x & 31;
    const int u = lane % a.units, sub = lane / a.units;   // place in the head, head of the pass
    const bool in_pass = sub < a.per_pass;
    const int heads = h.q_heads + h.k_heads;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t total = h.tokens * a.items;
    for (int64_t it = (int64_t)blockIdx.x * kHeadWarps + (threadIdx.x >> 5); it < total;
         it += (int64_t)gridDim.x * kHeadWarps) {
        const int64_t t = it / a.items;
        const int pass0 = (int)(it - t * a.items) * a.per_item;
        const int pass1 = pass0 + a.per_item < a.passes ? pass0 + a.per_item : a.passes;
        auto source = [&](int head) {   // start of the head
            return head < h.q_heads ? (const T *)h.q + t * h.q_stride + (int64_t)head * h.head_dim
                                    : (const T *)h.k + t * h.k_stride + (int64_t)(head - h.q_heads) * h.head_dim;
        };
        const int64_t pos = position_of(h, t, a.err);
        LanePlace q = place_of(h, in_pass ? u : 0, pos < 0 ? 0 : pos);
        Raw4 next[2] = {};
        int head = pass0 * a.per_pass + sub;
        bool on = in_pass && head < heads;
        if (on) {
            const T *x = source(head);
            load4(next[0], x + q.p0);
            load4(next[1], x + q.p1);
        }
        for (int pass = pass0; pass < pass1; pass++) {
            float v[8] = {};
            if (on) {
                unpack4<T>(next[0], v);
                unpack4<T>(next[1], v + 4);
            }
            const int this_head = head;
            const bool this_on = on;
            head += a.per_pass;
            on = in_pass && head < heads && pass + 1 < pass1;
            if (on) {
                const T *x = source(head);
                load4(next[0], x + q.p0);
                load4(next[1], x + q.p1);
            }
            const bool is_q = this_head < h.q_heads;
            norm_rotate(v, h, q, is_q ? h.q_weight : h.k_weight, in_pass ? u : 32, a.units, lane, this_on);
            if (pos < 0) {
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] = __int_as_float(0x7FC00000);
            }
            if (this_on) {
                // a lane stores the elements it loaded and no others: q_out = q and k_out = k are allowed
                T *y = is_q ? (T *)h.q_out + t * h.q_out_stride + (int64_t)this_head * h.head_dim
                            : (T *)h.k_out + t * h.k_out_stride + (int64_t)(this_head - h.q_heads) * h.head_dim;
                store4(y + q.p0, v);
                store4(y + q.p1, v + 4);
            }
        }
    }
}

// The same, then an optional Hadamard rotation and the codes of every head.
// Two passes' heads go through shared memory (fp32, at most 2 KB per warp) to
// the 16-element chunks of the quantizers, one chunk per lane, so that a
// quantization or Hadamard block lies in aligned neighbouring lanes.
template <typename T, int F>
__global__ void __launch_bounds__(kHeadThreads) k_qk_norm_rope_quantize(HeadKernelArgs a) {
    __shared__ __align__(16) float buf[kHeadWarps][512];
    const HeadArgs &h = a.h;
    const int lane = threadIdx.x & 31;
    float *b = buf[threadIdx.x >> 5];
    const int u = lane % a.units, sub = lane / a.units;
    const bool in_pass = sub < a.per_pass;
    const int heads = h.q_heads + h.k_heads;
    const int chunks = h.head_dim / 16;                     // lanes per head when coding
    const int chead = lane / chunks, cc = lane % chunks;    // head among the two passes', chunk of it
    const float norm = h.hadamard_b ? __frsqrt_rn((float)h.hadamard_b) : 1.0f;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t total = h.tokens * a.items;
    for (int64_t it = (int64_t)blockIdx.x * kHeadWarps + (threadIdx.x >> 5); it < total;
         it += (int64_t)gridDim.x * kHeadWarps) {
        const int64_t t = it / a.items;
        const int pass0 = (int)(it - t * a.items) * a.per_item;
        const int pass1 = pass0 + a.per_item < a.passes ? pass0 + a.per_item : a.passes;
        const int64_t pos = position_of(h, t, a.err);
        const LanePlace q = place_of(h, in_pass ? u : 0, pos < 0 ? 0 : pos);
        auto load = [&](int head, Raw4 (&r)[2]) {
            if (!in_pass || head >= heads) return;
            const T *x = head < h.q_heads ? (const T *)h.q + t * h.q_stride + (int64_t)head * h.head_dim
                                          : (const T *)h.k + t * h.k_stride + (int64_t)(head - h.q_heads) * h.head_dim;
            load4(r[0], x + q.p0);
            load4(r[1], x + q.p1);
        };
        Raw4 next[2][2] = {};
        int first = pass0 * a.per_pass;   // first head of the pair of passes
        load(first + sub, next[0]);
        if (pass0 + 1 < pass1) load(first + a.per_pass + sub, next[1]);
        for (int pass = pass0; pass < pass1; pass += 2, first += 2 * a.per_pass) {
            float v[2][8] = {};
#pragma unroll
            for (int p = 0; p < 2; p++) {
                unpack4<T>(next[p][0], v[p]);
                unpack4<T>(next[p][1], v[p] + 4);
            }
            if (pass + 2 < pass1) load(first + 2 * a.per_pass + sub, next[0]);
            if (pass + 3 < pass1) load(first + 3 * a.per_pass + sub, next[1]);
            __syncwarp();
#pragma unroll
            for (int p = 0; p < 2; p++) {
                const int head = first + p * a.per_pass + sub;
                const bool on = in_pass && head < heads && pass + p < pass1;
                norm_rotate(v[p], h, q, head < h.q_heads ? h.q_weight : h.k_weight, in_pass ? u : 32, a.units, lane, on);
                if (on) {
                    float *o = b + (p * a.per_pass + sub) * h.head_dim;
                    *reinterpret_cast<float4 *>(o + q.p0) = make_float4(v[p][0], v[p][1], v[p][2], v[p][3]);
                    *reinterpret_cast<float4 *>(o + q.p1) = make_float4(v[p][4], v[p][5], v[p][6], v[p][7]);
                }
            }
            __syncwarp();
            const int n_here = (pass + 1 < pass1 ? 2 : 1) * a.per_pass;
            const int head = first + chead;
            const bool valid = chead < n_here && head < heads;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; i++) x[i] = 0.0f;
            if (valid) {
                const float4 *src = reinterpret_cast<const float4 *>(b + lane * 16);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float4 f = src[i];
                    x[4 * i] = f.x; x[4 * i + 1] = f.y; x[4 * i + 2] = f.z; x[4 * i + 3] = f.w;
                }
            }
            if (h.hadamard_b) hadamard_chunk_n(x, h.hadamard_b, lane, norm);
            float amax = amax16(x);
            const bool is_q = head < h.q_heads;
            const int64_t row = is_q ? t * h.q_heads + head : t * h.k_heads + (head - h.q_heads);
            uint8_t *codes = (uint8_t *)(is_q ? h.q_out : h.k_out);
            void *scales = is_q ? h.q_scales : h.k_scales;
            if (F == kINT8Row) {
                for (int o = 16; o > 0; o >>= 1) {   // maximum over the head's lanes
                    const float y = __shfl_down_sync(0xFFFFFFFFu, amax, o);
                    if (cc < o && cc + o < chunks) amax = fmaxf(amax, y);
                }
                amax = __shfl_sync(0xFFFFFFFFu, amax, (lane - cc) & 31);
                const float s = pos < 0 ? __int_as_float(0x7FC00000) : __fdiv_rn(amax, 127.0f);
                const Recip rs = recip_of(s);
                if (valid) {
                    uint4 w = make_uint4(int_x4_quot(x, rs, 127), int_x4_quot(x + 4, rs, 127), int_x4_quot(x + 8, rs, 127),
                                         int_x4_quot(x + 12, rs, 127));
                    if (pos < 0) w = make_uint4(0x01010101u, 0x01010101u, 0x01010101u, 0x01010101u);   // 1 x NaN
                    *reinterpret_cast<uint4 *>(codes + (row * chunks + cc) * 16) = w;
                    if (cc == 0) reinterpret_cast<float *>(scales)[row] = s;
                }
            } else {
                amax = group_max<2>(amax);
                const bool zero = !(amax > 0.0f);
                float inv = 0.0f, z[16];
                uint32_t sb = zero ? 127u : mx_scale(amax, F == kMXFP8 ? 8 : 2, inv);
                if (pos < 0) sb = 255u;   // the NaN scale
                mul8(x, inv, z);
                mul8(x + 8, inv, z + 8);
                if (valid) {
                    if (F == kMXFP8) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            w[i] = zero ? 0u : cvt_e4m3x4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
                        *reinterpret_cast<uint4 *>(codes + (row * chunks + cc) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
                        uint32_t w[2];
#pragma unroll
                        for (int i = 0; i < 2; i++)
                            w[i] = zero ? 0u : cvt_e2m1x8(z[8 * i], z[8 * i + 1], z[8 * i + 2], z[8 * i + 3], z[8 * i + 4],
                                                          z[8 * i + 5], z[8 * i + 6], z[8 * i + 7]);
                        *reinterpret_cast<uint2 *>(codes + (row * chunks + cc) * 8) = make_uint2(w[0], w[1]);
                    }
                    if (!(cc & 1)) reinterpret_cast<uint8_t *>(scales)[row * (chunks / 2) + cc / 2] = (uint8_t)sb;
                }
            }
            __syncwarp();
        }
    }
}

template <typename F>
cudaError_t launch_heads(F *k, const HeadKernelArgs &a, cudaStream_t s) {
    const int64_t warps = a.h.tokens * a.items;
    int64_t ctas = (warps + kHeadWarps - 1) / kHeadWarps;
    const int64_t cap = (int64_t)sm_count() * 64;
    if (ctas > cap) ctas = cap;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(kHeadThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const HeadArgs &h, cudaStream_t s) {
    HeadKernelArgs a = {};
    a.h = h;
    a.units = h.head_dim / 8;
    a.per_pass = 32 / a.units;
    a.passes = (h.q_heads + h.k_heads + a.per_pass - 1) / a.per_pass;
    // Few tokens: spread a token's heads over warps, in steps of the two
    // passes that the quantizing kernel takes together, down to one step a
    // warp; many: a warp does up to 16 passes and reads its angles once.
    const int64_t want = (int64_t)sm_count() * 16;   // warps that fill the device
    int64_t per = h.tokens * a.passes / want;
    per = per < 2 ? 2 : per > 16 ? 16 : per / 2 * 2;
    if (h.fmt < 0 && h.tokens * a.passes < want) per = 1;
    a.per_item = (int)per;
    a.items = (a.passes + a.per_item - 1) / a.per_item;
    const cudaError_t e = error_word_address(&a.err);
    if (e != cudaSuccess) return e;
    if (h.fmt < 0) return h.bf16 ? launch_heads(k_qk_norm_rope<__nv_bfloat16>, a, s) : launch_heads(k_qk_norm_rope<float>, a, s);
    switch (h.fmt) {
    case kMXFP8:
        return h.bf16 ? launch_heads(k_qk_norm_rope_quantize<__nv_bfloat16, kMXFP8>, a, s)
                      : launch_heads(k_qk_norm_rope_quantize<float, kMXFP8>, a, s);
    case kMXFP4:
        return h.bf16 ? launch_heads(k_qk_norm_rope_quantize<__nv_bfloat16, kMXFP4>, a, s)
                      : launch_heads(k_qk_norm_rope_quantize<float, kMXFP4>, a, s);
    default:
        return h.bf16 ? launch_heads(k_qk_norm_rope_quantize<__nv_bfloat16, kINT8Row>, a, s)
                      : launch_heads(k_qk_norm_rope_quantize<float, kINT8Row>, a, s);
    }
}

}  // namespace mxq
