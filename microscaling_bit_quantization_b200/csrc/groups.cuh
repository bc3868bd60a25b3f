// groups.cuh -- rows in expert order: the group table that the grouped
// quantizer and the grouped products build from the device offsets, and the
// bounds they hold those offsets to.
#pragma once

#include <stdint.h>

#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr unsigned int kErrIndex = 256u;   // error word: an index in device data outside its range (mxq_check: MXQ_EINVAL)

__device__ __forceinline__ void latch_index_error(unsigned int *err) {
    if (err) atomicOr(err, kErrIndex);
}

// Offsets are device data the host cannot check: each is held to
// [0, rows], and a group whose end lies before its start is empty, so that
// no offset leads outside the buffers.
__device__ __forceinline__ int clamp_row(int o, int64_t rows) {
    return o < 0 ? 0 : (int64_t)o > rows ? (int)rows : o;
}

// Whether offsets[i] lies outside [0, rows] or before its predecessor.
__device__ __forceinline__ bool offset_wrong(const int32_t *offsets, int i, int64_t rows) {
    const int o = offsets[i];
    return o != clamp_row(o, rows) || (i > 0 && offsets[i - 1] > o);
}

struct Groups {
    int off[kMaxGroups + 1];
    int tile[kMaxGroups + 1];   // 128-row scale tiles before each group
    int wide[kMaxGroups + 1];   // blocks of 256 rows before each group
    int2 sum[kMaxGroups / 32];  // tiles and blocks of 32 groups
};

// Fills `g` (all threads of the block call this); a table that had to be
// clamped is reported to *err when err is given.
__device__ __forceinline__ void load_groups(Groups &g, const int32_t *offsets, int n, int64_t rows, unsigned int *err) {
    for (int i = threadIdx.x; i <= n; i += blockDim.x) {
        g.off[i] = clamp_row(offsets[i], rows);
        if (offset_wrong(offsets, i, rows)) latch_index_error(err);
    }
    __syncthreads();
    // a warp scans 32 groups; then each entry adds the sums of the warps before
    const int lane = threadIdx.x & 31;
    for (int b = threadIdx.x >> 5; 32 * b < n; b += blockDim.x >> 5) {
        const int e = 32 * b + lane;
        const int rows_e = e < n ? g.off[e + 1] - g.off[e] : 0;
        const int t = rows_e > 0 ? (rows_e + 127) >> 7 : 0, w = (t + 1) >> 1;
        int s = t, s2 = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, s, o), v2 = __shfl_up_sync(0xFFFFFFFFu, s2, o);
            if (lane >= o) {
                s += v;
                s2 += v2;
            }
        }
        if (e < n) {
            g.tile[e] = s - t;
            g.wide[e] = s2 - w;
        }
        if (lane == 31) g.sum[b] = make_int2(s, s2);
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= n; e += blockDim.x) {
        int2 before = make_int2(0, 0);
        for (int b = 0; 32 * b + 31 < e || (e == n && 32 * b < n); b++) {
            before.x += g.sum[b].x;
            before.y += g.sum[b].y;
        }
        g.tile[e] = before.x + (e < n ? g.tile[e] : 0);
        g.wide[e] = before.y + (e < n ? g.wide[e] : 0);
    }
    __syncthreads();
}

// The group that holds row r, or -1.
__device__ __forceinline__ int group_of_row(const Groups &g, int n, int r) {
    int lo = 0, hi = n;   // the last group that starts at or before r
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (g.off[mid] <= r) lo = mid;
        else hi = mid;
    }
    return r >= g.off[lo] && r < g.off[lo + 1] ? lo : -1;
}

}  // namespace
}  // namespace mxq
