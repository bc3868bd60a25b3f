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
// floor(32 / U) heads at a time (a pass).  A warp's work is an item: up to
// 16 passes over the q heads, or the k heads, of one token, so that a lane's
// weights and angles, joined to one linear map, serve them all and pointers
// only step; the items of all q come before those of all k, so that the warps
// of a block, and the last blocks, have equal ones.  Sums run over the U lanes
// by shuffles: butterflies where U is a power of two, else a tree.
// Bound: instruction issue and latency together (8192 tokens x 40 heads x 128
// in bf16: 30.5 us, 5.6 TB/s, some 125 instructions per pass of 256 elements, 67% of
// issue slots used; items of up to 8 passes 32.5 us: a short one waits for its
// angles as long as a long one).  Lane counts that are no power of two pay idle
// lanes and the tree: 72 wide 25.5 us (58% of the copy rate), 64 wide 18.7 (70%).
#include <cuda_runtime.h>

#include "groups.cuh"
#include "mxq_formats.cuh"
#include "mxq_internal.h"
#include "tc_ptx.cuh"

namespace mxq {
namespace {

constexpr int kHeadThreads = 128;
constexpr int kHeadWarps = kHeadThreads / 32;
constexpr int kHeadPasses = 16;   // of an item, at most

struct HeadKernelArgs {
    HeadArgs h;
    int units;          // lanes per head
    int per_pass;       // heads a warp takes at a time
    // An item, a warp's work, is a run of passes over one side (q or k) of a token; first the items of all
    // tokens' q, then of their k, so that the warps of a block, and the last blocks, have equal ones
    int per_item[2];    // passes of an item (q, k)
    FastDiv items[2];   // items of a token
    uint32_t q_total, total;
    // 1 / head_dim; for the sum of squares that and eps times the Hadamard size b (exact, a power of two), so that the
    // head's factor carries 1/sqrt(b)
    float inv_d, scale, eps;
    unsigned int *err;
};

// Sum over the lanes of a head: UNITS neighbouring lanes, a power of two, or
// (UNITS = 0) any number, `u` being this lane's place among them (lanes past
// the last head have u >= units and take no part).
template <int UNITS>
__device__ __forceinline__ float head_sum(float x, int u, int units, int lane) {
    if constexpr (UNITS > 0) {
#pragma unroll
        for (int o = 1; o < UNITS; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
        return x;
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float y = __shfl_down_sync(0xFFFFFFFFu, x, o);
            if (u < o && u + o < units) x += y;
        }
        return __shfl_sync(0xFFFFFFFFu, x, lane - u);
    }
}

// A lane's eight elements as the firsts a[0..3] and the seconds b[0..3] of
// four pairs, two-wide for packed arithmetic.
struct Pairs {
    float2 a[2], b[2];
};
template <typename T>
struct Raw {
    uint4 w[sizeof(T) / 2];
};
template <bool IL>
__device__ __forceinline__ void load_raw(Raw<__nv_bfloat16> &r, const __nv_bfloat16 *x, int apart) {   // x: the first group
    if (IL) {
        r.w[0] = *reinterpret_cast<const uint4 *>(x);
    } else {
        const uint2 a = *reinterpret_cast<const uint2 *>(x), b = *reinterpret_cast<const uint2 *>(x + apart);
        r.w[0] = make_uint4(a.x, a.y, b.x, b.y);
    }
}
template <bool IL>
__device__ __forceinline__ void load_raw(Raw<float> &r, const float *x, int apart) {
    r.w[0] = *reinterpret_cast<const uint4 *>(x);
    r.w[1] = *reinterpret_cast<const uint4 *>(x + apart);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
template <bool IL>
__device__ __forceinline__ Pairs unpack(const Raw<__nv_bfloat16> &r) {
    const uint4 w = r.w[0];
    Pairs v;
    if (IL) {
        v.a[0] = make_float2(bf_lo(w.x), bf_lo(w.y));
        v.a[1] = make_float2(bf_lo(w.z), bf_lo(w.w));
        v.b[0] = make_float2(bf_hi(w.x), bf_hi(w.y));
        v.b[1] = make_float2(bf_hi(w.z), bf_hi(w.w));
    } else {
        v.a[0] = make_float2(bf_lo(w.x), bf_hi(w.x));
        v.a[1] = make_float2(bf_lo(w.y), bf_hi(w.y));
        v.b[0] = make_float2(bf_lo(w.z), bf_hi(w.z));
        v.b[1] = make_float2(bf_lo(w.w), bf_hi(w.w));
    }
    return v;
}
template <bool IL>
__device__ __forceinline__ Pairs unpack(const Raw<float> &r) {
    const uint4 x = r.w[0], y = r.w[1];
    auto f = [](uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); };
    Pairs v;
    if (IL) {
        v.a[0] = f(x.x, x.z);
        v.b[0] = f(x.y, x.w);
        v.a[1] = f(y.x, y.z);
        v.b[1] = f(y.y, y.w);
    } else {
        v.a[0] = f(x.x, x.y);
        v.a[1] = f(x.z, x.w);
        v.b[0] = f(y.x, y.y);
        v.b[1] = f(y.z, y.w);
    }
    return v;
}
// The elements at p0 .. p0 + 3 and p1 .. p1 + 3.
template <bool IL>
__device__ __forceinline__ void in_order(const Pairs &v, float4 &x, float4 &y) {
    if (IL) {
        x = make_float4(v.a[0].x, v.b[0].x, v.a[0].y, v.b[0].y);
        y = make_float4(v.a[1].x, v.b[1].x, v.a[1].y, v.b[1].y);
    } else {
        x = make_float4(v.a[0].x, v.a[0].y, v.a[1].x, v.a[1].y);
        y = make_float4(v.b[0].x, v.b[0].y, v.b[1].x, v.b[1].y);
    }
}
template <bool IL>
__device__ __forceinline__ void store_raw(__nv_bfloat16 *o, int apart, const Pairs &v) {
    float4 x, y;
    in_order<IL>(v, x, y);
    const uint2 a = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
    const uint2 b = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    if (IL) {
        *reinterpret_cast<uint4 *>(o) = make_uint4(a.x, a.y, b.x, b.y);
    } else {
        *reinterpret_cast<uint2 *>(o) = a;
        *reinterpret_cast<uint2 *>(o + apart) = b;
    }
}
template <bool IL>
__device__ __forceinline__ void store_raw(float *o, int apart, const Pairs &v) {
    float4 x, y;
    in_order<IL>(v, x, y);
    *reinterpret_cast<float4 *>(o) = x;
    *reinterpret_cast<float4 *>(o + apart) = y;
}

// Weight and rotation of a lane's pairs as one linear map:
// a' = aa a + ab b, b' = bb b + ba a with aa = w_a c, ab = -w_b s, bb = w_b c,
// ba = w_a s; for elements behind rot_dim a' = w_a a, b' = w_b b.  One serves
// an item.
struct Turn {
    float2 aa[2], ab[2], bb[2], ba[2];
};
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
// A lane's cosines and sines of position pos.
struct Angles {
    float4 c, s;
};
__device__ __forceinline__ Angles angles_of(const HeadArgs &h, int u, bool turned, int64_t pos) {
    Angles a = {};
    if (turned) {
        const int64_t at = pos * (h.rot / 2) + 4 * u;
        a.c = __ldg(reinterpret_cast<const float4 *>(h.cos_t + at));
        a.s = __ldg(reinterpret_cast<const float4 *>(h.sin_t + at));
    }
    return a;
}
// (The angles are asked for before the weights: they hang on the position's
// load and come from further away; in the other order the same heads to MXFP8
// behind a Hadamard rotation take 48.4 us, not 47.7, in bf16 30.6, not 30.5.)
template <bool IL>
__device__ __forceinline__ Turn turn_of(const float *w, int p0, int p1, bool turned, const Angles &angles) {
    float4 x = make_float4(1.0f, 1.0f, 1.0f, 1.0f), y = x;
    if (w) {
        x = __ldg(reinterpret_cast<const float4 *>(w + p0));
        y = __ldg(reinterpret_cast<const float4 *>(w + p1));
    }
    Turn t;
    if (IL) {
        t.aa[0] = make_float2(x.x, x.z);
        t.bb[0] = make_float2(x.y, x.w);
        t.aa[1] = make_float2(y.x, y.z);
        t.bb[1] = make_float2(y.y, y.w);
    } else {
        t.aa[0] = make_float2(x.x, x.y);
        t.aa[1] = make_float2(x.z, x.w);
        t.bb[0] = make_float2(y.x, y.y);
        t.bb[1] = make_float2(y.z, y.w);
    }
    if (turned) {
        const float4 c = angles.c, s = angles.s;
        const float2 cc[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
        const float2 ss[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
        const float2 minus = make_float2(-1.0f, -1.0f);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            t.ab[i] = mul2(mul2(t.bb[i], minus), ss[i]);
            t.ba[i] = mul2(t.aa[i], ss[i]);
            t.aa[i] = mul2(t.aa[i], cc[i]);
            t.bb[i] = mul2(t.bb[i], cc[i]);
        }
    }
    return t;
}

// Norm of the heads in a pass: v becomes its weighted and turned elements
// before the head's factor r = 1/sqrt(mean square + eps), which is returned
// (the map is linear: one multiplication less, and none waits for the sum).
template <int UNITS>
__device__ __forceinline__ float norm_turn(Pairs &v, const HeadKernelArgs &k, const Turn &t, bool turned, int u, int lane) {
    if (k.h.norm == 1) {
        const float2 s2 = __fadd2_rn(__fadd2_rn(v.a[0], v.a[1]), __fadd2_rn(v.b[0], v.b[1]));
        const float m = -head_sum<UNITS>(s2.x + s2.y, u, k.units, lane) * k.inv_d;
        const float2 mm = make_float2(m, m);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            v.a[i] = __fadd2_rn(v.a[i], mm);
            v.b[i] = __fadd2_rn(v.b[i], mm);
        }
    }
    const float2 q2 = fma2(v.b[1], v.b[1], fma2(v.b[0], v.b[0], fma2(v.a[1], v.a[1], mul2(v.a[0], v.a[0]))));
    const float r = rsqrtf(fmaf(head_sum<UNITS>(q2.x + q2.y, u, k.units, lane), k.scale, k.eps));
#pragma unroll
    for (int i = 0; i < 2; i++) {
        float2 a = mul2(t.aa[i], v.a[i]), b = mul2(t.bb[i], v.b[i]);
        if (turned) {
            a = fma2(t.ab[i], v.b[i], a);
            b = fma2(t.ba[i], v.a[i], b);
        }
        v.a[i] = a;
        v.b[i] = b;
    }
    return r;
}

// The larger of two magnitudes, NaN if either is one (fmaxf drops a NaN).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// Over aligned groups of G lanes (G a power of two).
template <int G>
__device__ __forceinline__ float group_max_nan(float a) {
#pragma unroll
    for (int o = 1; o < G; o <<= 1) a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    return a;
}

// The position of token t, or -1 (reported) for one outside the tables.
__device__ __forceinline__ int64_t position_of(const HeadArgs &h, int64_t t, unsigned int *err) {
    if (h.rot == 0) return 0;
    const int64_t pos = !h.positions ? t
                        : h.pos64    ? static_cast<const int64_t *>(h.positions)[t]
                                     : (int64_t)static_cast<const int32_t *>(h.positions)[t];
    if (pos >= 0 && pos < h.n_pos) return pos;
    latch_index_error(err);
    return -1;
}

// What a lane does in every head: its place and its two groups of elements.
template <int UNITS, bool IL>
struct LanePlace {
    int u, sub, p0, p1;
    bool in_pass, turned;
    __device__ __forceinline__ LanePlace(const HeadKernelArgs &a, int lane) {
        const int units = UNITS ? UNITS : a.units;
        u = lane % units;
        sub = lane / units;
        in_pass = UNITS ? true : sub < a.per_pass;
        turned = in_pass && 8 * u < a.h.rot;
        p0 = turned && !IL ? 4 * u : 8 * u;
        p1 = turned && !IL ? a.h.rot / 2 + 4 * u : 8 * u + 4;
        if (!in_pass) {   // a lane past the last head: no part in a sum, and its weights are read from the first ones
            u = 32;
            p0 = 0;
            p1 = 4;
        }
    }
};

// An item: a run of neighbouring heads of one token, all q or all k.
template <typename T>
struct HeadItem {
    bool is_k;
    int64_t t, pos;
    int head, end, passes;   // this lane's first head, the side's number of heads, passes of the item
    const T *x;              // this lane's elements of that head
    __device__ __forceinline__ HeadItem(const HeadKernelArgs &a, uint32_t item, int sub, bool in_pass, int p0) {
        is_k = item >= a.q_total;
        if (is_k) item -= a.q_total;
        const FastDiv items = is_k ? a.items[1] : a.items[0];
        const int per_item = is_k ? a.per_item[1] : a.per_item[0];
        const uint32_t token = fdiv(item, items);
        t = token;
        end = is_k ? a.h.k_heads : a.h.q_heads;
        const int first = (int)(item - token * items.d) * per_item * a.per_pass;
        const int left = (end - first + a.per_pass - 1) / a.per_pass;
        passes = left < per_item ? left : per_item;
        head = first + sub;
        if (!in_pass) end = 0;   // lanes past the last head have none
        x = (is_k ? (const T *)a.h.k + t * a.h.k_stride : (const T *)a.h.q + t * a.h.q_stride) + (int64_t)head * a.h.head_dim + p0;
    }
};

template <typename T, int UNITS, bool IL>
__global__ void __launch_bounds__(kHeadThreads, 8) k_qk_norm_rope(HeadKernelArgs a) {
    // passes whose loads are in flight (8192 x 40 heads x 128 bf16: 4 30.5 us, 2 32.0, 8 40.7; 72 wide 2 25.5, 4 26.2;
    // 128 wide fp32 2 54.4, 4 66.9)
    constexpr int kDepth = sizeof(T) == 2 && UNITS > 0 ? 4 : 2;
    const HeadArgs &h = a.h;
    const int lane = threadIdx.x & 31;
    const LanePlace<UNITS, IL> q(a, lane);
    const int step = a.per_pass * h.head_dim, apart = q.p1 - q.p0;
    pdl_wait();
    pdl_launch_dependents();
    for (uint32_t item = blockIdx.x * kHeadWarps + (threadIdx.x >> 5); item < a.total; item += gridDim.x * kHeadWarps) {
        HeadItem<T> in(a, item, q.sub, q.in_pass, q.p0);
        Raw<T> raw[kDepth] = {};
        int ahead = in.head;
        auto fetch = [&](Raw<T> &r) {
            if (ahead < in.end) load_raw<IL>(r, in.x, apart);
            ahead += a.per_pass;
            in.x += step;
        };
#pragma unroll
        for (int j = 0; j < kDepth; j++)
            if (j < in.passes) fetch(raw[j]);
        const int64_t pos = position_of(h, in.t, a.err);
        const Turn turn = turn_of<IL>(in.is_k ? h.k_weight : h.q_weight, q.p0, q.p1, q.turned,
                                      angles_of(h, q.u, q.turned, pos < 0 ? 0 : pos));
        T *y = (in.is_k ? (T *)h.k_out + in.t * h.k_out_stride : (T *)h.q_out + in.t * h.q_out_stride) +
               (int64_t)in.head * h.head_dim + q.p0;
#pragma unroll 1
        for (int pass = 0; pass < in.passes; pass += kDepth) {
#pragma unroll
            for (int j = 0; j < kDepth; j++) {
                if (pass + j < in.passes) {
                    Pairs v = unpack<IL>(raw[j]);
                    if (pass + j + kDepth < in.passes) fetch(raw[j]);
                    float r = norm_turn<UNITS>(v, a, turn, q.turned, q.u, lane);
                    if (pos < 0) r = __int_as_float(0x7FC00000);
                    if (in.head < in.end) {
                        // a lane stores the elements it loaded and no others: q_out = q and k_out = k are allowed
                        const float2 rr = make_float2(r, r);
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            v.a[i] = mul2(v.a[i], rr);
                            v.b[i] = mul2(v.b[i], rr);
                        }
                        store_raw<IL>(y, apart, v);
                    }
                    in.head += a.per_pass;
                    y += step;
                }
            }
        }
    }
}

// Block-diagonal Hadamard rotation of the heads in a pass without its factor
// 1/sqrt(b): lane u of a head holds its elements 8u .. 8u + 7, the even ones in
// v.a and the odd ones in v.b.  Stages 1, 2 and 4 lie in the lane, stage 8 l
// pairs lanes that differ in bit l: a lane's elements stay or change sign and
// the partner's are added, one packed FMA for two.
template <int UNITS>
__device__ __forceinline__ void hadamard_heads(Pairs &v, int b, int lane) {
    const float2 minus = make_float2(-1.0f, -1.0f);
    auto both = [&](float2 &x, float2 &y) {   // (x + y, x - y)
        const float2 s = __fadd2_rn(x, y);
        y = fma2(y, minus, x);
        x = s;
    };
    both(v.a[0], v.b[0]);
    both(v.a[1], v.b[1]);
    if (b > 2) {
        auto inside = [](float2 &x) { x = make_float2(__fadd_rn(x.x, x.y), __fsub_rn(x.x, x.y)); };
        inside(v.a[0]);
        inside(v.a[1]);
        inside(v.b[0]);
        inside(v.b[1]);
    }
    if (b > 4) {
        both(v.a[0], v.a[1]);
        both(v.b[0], v.b[1]);
    }
#pragma unroll
    for (int l = 1; l < (UNITS ? UNITS : 32); l <<= 1) {
        if (8 * l < b) {
            const float sign = (lane & l) ? -1.0f : 1.0f;
            const float2 sg = make_float2(sign, sign);
            auto cross = [&](float2 &x) {
                x = fma2(sg, x, make_float2(__shfl_xor_sync(0xFFFFFFFFu, x.x, l), __shfl_xor_sync(0xFFFFFFFFu, x.y, l)));
            };
            cross(v.a[0]);
            cross(v.a[1]);
            cross(v.b[0]);
            cross(v.b[1]);
        }
    }
}

// The same, then an optional Hadamard rotation and the codes of every head.
// Codes want a lane to hold 8 neighbouring elements.  Interleaved pairs have
// them so; pairs of halves go through shared memory (1 KB per warp), stored so
// that both 16-byte reads give even and odd elements apart.  The head's factor
// (with 1/sqrt(b) in it) is applied where the codes are formed.  Bound: instruction
// issue (the same heads to MXFP8: 35.5 us, with a Hadamard rotation of 128 47.7,
// pairs of halves 37.0 and 56.8; some 270 instructions per pass with the rotation
// and 80% of issue slots used; two passes unrolled 48.9 us and pairs of halves
// 55.1, the cross-lane stages as a loop 56.4 and 58.9: the instructions have to
// fit the fetch and be few).
template <typename T, int F, int UNITS, bool IL>
__global__ void __launch_bounds__(kHeadThreads, 7) k_qk_norm_rope_quantize(HeadKernelArgs a) {
    __shared__ __align__(16) float buf[IL ? 1 : kHeadWarps][IL ? 4 : 256];
    const HeadArgs &h = a.h;
    const int lane = threadIdx.x & 31;
    float *b = buf[IL ? 0 : threadIdx.x >> 5];
    const LanePlace<UNITS, IL> q(a, lane);
    const int d = h.head_dim, step = a.per_pass * d, apart = q.p1 - q.p0;
    constexpr int kPerByte = F == kMXFP4 ? 2 : 1;
    const int code_step = step / kPerByte, scale_step = a.per_pass * (F == kINT8Row ? 4 : d / 32);
    pdl_wait();
    pdl_launch_dependents();
    for (uint32_t item = blockIdx.x * kHeadWarps + (threadIdx.x >> 5); item < a.total; item += gridDim.x * kHeadWarps) {
        HeadItem<T> in(a, item, q.sub, q.in_pass, q.p0);
        const int64_t pos = position_of(h, in.t, a.err);
        Raw<T> raw = {};
        if (in.head < in.end) load_raw<IL>(raw, in.x, apart);
        const Turn turn = turn_of<IL>(in.is_k ? h.k_weight : h.q_weight, q.p0, q.p1, q.turned,
                                      angles_of(h, q.u, q.turned, pos < 0 ? 0 : pos));
        const int64_t row = in.t * (in.is_k ? h.k_heads : h.q_heads) + in.head;
        uint8_t *codes = (uint8_t *)(in.is_k ? h.k_out : h.q_out) + (row * d + 8 * q.u) / kPerByte;
        uint8_t *scales = (uint8_t *)(in.is_k ? h.k_scales : h.q_scales) + (F == kINT8Row ? row * 4 : row * (d / 32) + q.u / 4);
#pragma unroll 1
        for (int pass = 0; pass < in.passes; pass++) {
            Pairs v = unpack<IL>(raw);
            const bool valid = in.head < in.end;
            in.head += a.per_pass;
            in.x += step;
            if (in.head < in.end && pass + 1 < in.passes) load_raw<IL>(raw, in.x, apart);
            float f = norm_turn<UNITS>(v, a, turn, q.turned, q.u, lane);
            if (pos < 0) f = __int_as_float(0x7FC00000);
            if (!IL) {
                __syncwarp();   // the pass before has been read
                if (q.in_pass) {
                    *reinterpret_cast<float4 *>(b + q.sub * d + q.p0) = make_float4(v.a[0].x, v.a[1].x, v.a[0].y, v.a[1].y);
                    *reinterpret_cast<float4 *>(b + q.sub * d + q.p1) = make_float4(v.b[0].x, v.b[1].x, v.b[0].y, v.b[1].y);
                }
                __syncwarp();
                if (q.in_pass) {
                    const float4 x = *reinterpret_cast<const float4 *>(b + q.sub * d + 8 * q.u);
                    const float4 y = *reinterpret_cast<const float4 *>(b + q.sub * d + 8 * q.u + 4);
                    v.a[0] = make_float2(x.x, x.y);
                    v.b[0] = make_float2(x.z, x.w);
                    v.a[1] = make_float2(y.x, y.y);
                    v.b[1] = make_float2(y.z, y.w);
                }
            }
            if (h.hadamard_b) hadamard_heads<UNITS>(v, h.hadamard_b, lane);
            float amax = max_nan(max_nan(max_nan(fabsf(v.a[0].x), fabsf(v.a[0].y)), max_nan(fabsf(v.a[1].x), fabsf(v.a[1].y))),
                                 max_nan(max_nan(fabsf(v.b[0].x), fabsf(v.b[0].y)), max_nan(fabsf(v.b[1].x), fabsf(v.b[1].y))));
            // the largest |v f| is the largest |v| times f: rounding keeps the order, and a NaN anywhere stays one
            // (as an infinite v does where the mean square is infinite, f zero)
            amax = __fmul_rn(amax, f);
            if (F == kINT8Row) {
                if (UNITS) {
                    amax = group_max_nan<(UNITS ? UNITS : 1)>(amax);
                } else {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        const float y = __shfl_down_sync(0xFFFFFFFFu, amax, o);
                        if (q.u < o && q.u + o < a.units) amax = max_nan(amax, y);
                    }
                    amax = __shfl_sync(0xFFFFFFFFu, amax, lane - q.u);
                }
                const float s = __fdiv_rn(amax, 127.0f);
                const Recip rs = recip_of(s);
                if (valid) {
                    const float2 ff = make_float2(f, f);
                    const float2 a0 = mul2(v.a[0], ff), a1 = mul2(v.a[1], ff), b0 = mul2(v.b[0], ff), b1 = mul2(v.b[1], ff);
                    const float x[8] = {a0.x, b0.x, a0.y, b0.y, a1.x, b1.x, a1.y, b1.y};
                    *reinterpret_cast<uint2 *>(codes) = make_uint2(int_x4_quot(x, rs, 127), int_x4_quot(x + 4, rs, 127));
                    if (q.u == 0) *reinterpret_cast<float *>(scales) = s;
                }
            } else {
                amax = group_max_nan<4>(amax);
                constexpr int kEmax = F == kMXFP8 ? 8 : 2;
                uint32_t sb;
                float inv;
                const bool mid = mx_scale_mid(amax, kEmax, sb, inv);
                // (v f) 2^-e rounded once, as v (f 2^-e) where that factor is finite and normal
                float m = __fmul_rn(f, inv);
                if (!(mid && m >= 1e-30f && m <= 1e30f)) {
                    inv = 0.0f;
                    const bool zero = !(amax > 0.0f);
                    sb = amax != amax ? 255u : zero ? 127u : mx_scale(amax, kEmax, inv);   // 255: the NaN scale
                    m = __fmul_rn(f, inv);
                    if (zero) {
                        v = Pairs{};
                        m = 0.0f;
                    } else if (!(m >= 1e-30f && m <= 1e30f)) {
                        m = inv;
                        const float2 ff = make_float2(f, f);
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            v.a[i] = mul2(v.a[i], ff);
                            v.b[i] = mul2(v.b[i], ff);
                        }
                    }
                }
                if (valid) {
                    const float2 mm = make_float2(m, m);
                    const float2 a0 = mul2(v.a[0], mm), a1 = mul2(v.a[1], mm), b0 = mul2(v.b[0], mm), b1 = mul2(v.b[1], mm);
                    if (F == kMXFP8)
                        *reinterpret_cast<uint2 *>(codes) =
                            make_uint2(cvt_e4m3x4(a0.x, b0.x, a0.y, b0.y), cvt_e4m3x4(a1.x, b1.x, a1.y, b1.y));
                    else
                        *reinterpret_cast<uint32_t *>(codes) = cvt_e2m1x8(a0.x, b0.x, a0.y, b0.y, a1.x, b1.x, a1.y, b1.y);
                    if (!(q.u & 3)) *scales = (uint8_t)sb;
                }
            }
            codes += code_step;
            scales += scale_step;
        }
    }
}

cudaError_t launch_heads(void (*k)(HeadKernelArgs), const HeadKernelArgs &a, cudaStream_t s) {
    int64_t ctas = ((int64_t)a.total + kHeadWarps - 1) / kHeadWarps;
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

// The instance for a head's lanes (a power of two of them in registers'
// butterflies, any other number by the shuffle tree) and its way of pairing.
template <typename T, int UNITS, bool IL>
cudaError_t pick_format(const HeadKernelArgs &a, cudaStream_t s) {
    switch (a.h.fmt) {
    case kMXFP8: return launch_heads(k_qk_norm_rope_quantize<T, kMXFP8, UNITS, IL>, a, s);
    case kMXFP4: return launch_heads(k_qk_norm_rope_quantize<T, kMXFP4, UNITS, IL>, a, s);
    case kINT8Row: return launch_heads(k_qk_norm_rope_quantize<T, kINT8Row, UNITS, IL>, a, s);
    default: return launch_heads(k_qk_norm_rope<T, UNITS, IL>, a, s);
    }
}
template <typename T, bool IL>
cudaError_t pick_units(const HeadKernelArgs &a, cudaStream_t s) {
    switch (a.units) {
    case 8: return pick_format<T, 8, IL>(a, s);
    case 16: return pick_format<T, 16, IL>(a, s);
    case 32: return pick_format<T, 32, IL>(a, s);
    default: return pick_format<T, 0, IL>(a, s);
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const HeadArgs &h, cudaStream_t s) {
    HeadKernelArgs a = {};
    a.h = h;
    a.units = h.head_dim / 8;
    const float b = h.hadamard_b ? (float)h.hadamard_b : 1.0f;
    a.inv_d = 1.0f / (float)h.head_dim;
    a.scale = a.inv_d * b;
    a.eps = h.eps * b;
    a.per_pass = 32 / a.units;
    // Few tokens: a token's heads are spread over warps, down to one pass each;
    // many: a warp does up to kHeadPasses passes and reads its angles once.
    const int64_t passes[2] = {(h.q_heads + a.per_pass - 1) / a.per_pass, (h.k_heads + a.per_pass - 1) / a.per_pass};
    int64_t most = h.tokens * (passes[0] + passes[1]) / ((int64_t)sm_count() * 16);
    most = most < 1 ? 1 : most > kHeadPasses ? kHeadPasses : most;
    auto items = [&](int side) { return (passes[side] + most - 1) / most; };
    while (h.tokens * (items(0) + items(1)) >= ((int64_t)1 << 31)) most *= 2;   // items are counted in 31 bits (tokens in 30: two items of a token fit)
    for (int side = 0; side < 2; side++) {
        const int64_t n = items(side) ? items(side) : 1;
        a.per_item[side] = (int)((passes[side] + n - 1) / n);   // equal shares
        a.items[side] = make_fastdiv((uint32_t)n);
    }
    a.q_total = (uint32_t)(h.tokens * items(0));
    a.total = a.q_total + (uint32_t)(h.tokens * items(1));
    const cudaError_t e = error_word_address(&a.err);
    if (e != cudaSuccess) return e;
    if (h.bf16) return h.interleaved ? pick_units<__nv_bfloat16, true>(a, s) : pick_units<__nv_bfloat16, false>(a, s);
    return h.interleaved ? pick_units<float, true>(a, s) : pick_units<float, false>(a, s);
}

}  // namespace mxq
