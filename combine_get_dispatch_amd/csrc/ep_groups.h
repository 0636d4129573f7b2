// ep_groups.h -- the rows of every expert, as the experts' kernels see them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep.h"

namespace ep {

constexpr int kGroupsMaxExperts = 1024;

// Rows of expert e: packed layout (region_rows = 0): rows [start, start + n)
// with start = (e / epr) * cap_rows + offsets[e] and n = counts[e], cut at the
// rank's cap_rows. Low-latency layout: for each source s < R the rows
// e * R * region_rows + s * region_rows + [0, counts[e * R + s]). Counts and
// offsets come from the device and are cut to what lies inside the rank's
// (region's) rows, so no kernel leaves the row arrays whatever they hold.
struct GroupArgs {
    const int32_t *offsets, *counts;
    int E, R, epr;
    int64_t cap_rows;
    int region_rows;
};

// Host side (ep_rows.hip): the checked kernel arguments of a caller's groups,
// all rows of the receive array, the rows its groups are expected to hold, the
// current device's compute units, and the library's code for a HIP result.
int group_args(const ep_groups *g, GroupArgs *out);
int64_t group_rows(const ep_groups *g);
int64_t group_rows_expected(const ep_groups *g);
int device_cus(int *cus);
int hip_status(hipError_t e, const char *what);

// Host side: whether two arrays share bytes (NULL and empty ones none). Workgroups
// write results while others still read operands, so no output may.
inline bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && a_bytes > 0 && b_bytes > 0 && x < y + (uint64_t)b_bytes && y < x + (uint64_t)a_bytes;
}

__device__ __forceinline__ int group_region_count(const GroupArgs &g, int e, int s) {
    const int c = g.counts[(int64_t)e * g.R + s];
    return c < 0 ? 0 : c > g.region_rows ? g.region_rows : c;
}

// rows of expert e (all its regions together)
__device__ __forceinline__ int group_count(const GroupArgs &g, int e) {
    if (g.region_rows > 0) {
        int n = 0;
        for (int s = 0; s < g.R; ++s) n += group_region_count(g, e, s);
        return n;
    }
    const int off = g.offsets[e], c = g.counts[e];
    if (off < 0 || c <= 0 || off >= g.cap_rows) return 0;
    const int64_t room = g.cap_rows - off;
    return c > room ? (int)room : c;
}

// receive row of expert e's i-th row; i < group_count(g, e)
__device__ __forceinline__ int64_t group_row(const GroupArgs &g, int e, int i) {
    if (g.region_rows > 0) {
        const int64_t base = (int64_t)e * g.R * g.region_rows;
        for (int s = 0; s < g.R - 1; ++s) {
            const int c = group_region_count(g, e, s);
            if (i < c) return base + (int64_t)s * g.region_rows + i;
            i -= c;
        }
        return base + (int64_t)(g.R - 1) * g.region_rows + i;
    }
    return (int64_t)(e / g.epr) * g.cap_rows + g.offsets[e] + i;
}

// sum of two counts, held at the largest int (overlapping experts could pass it)
__device__ __forceinline__ int group_add(int a, int b) {
    const uint32_t s = (uint32_t)a + (uint32_t)b;
    return s > 0x7FFFFFFFu ? 0x7FFFFFFF : (int)s;
}

// In place: ends[e] = sum of ends[i], i <= e, by the workgroup's first wave.
// Between barriers of its own. E <= kGroupsMaxExperts entries in LDS.
__device__ __forceinline__ void group_prefix(int *ends, int E) {
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid < 64) {
        int carry = 0;
        for (int base = 0; base < E; base += 64) {
            const int e = base + tid;
            int v = e < E ? ends[e] : 0;
            for (int d = 1; d < 64; d <<= 1) {
                const int u = __shfl_up(v, d);
                if (tid >= d) v = group_add(v, u);
            }
            v = group_add(v, carry);
            if (e < E) ends[e] = v;
            carry = __shfl(v, 63);
        }
    }
    __syncthreads();
}

// ends[e] = rows of the experts <= e, by a workgroup of `threads` threads
// (whole waves). Returns all rows.
__device__ __forceinline__ int group_scan(const GroupArgs &g, int *ends, int threads) {
    for (int e = threadIdx.x; e < g.E; e += threads) ends[e] = group_count(g, e);
    group_prefix(ends, g.E);
    return ends[g.E - 1];
}

// first expert whose end is past t (t < ends[E - 1])
__device__ __forceinline__ int group_find(const int *ends, int E, int t) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

}  // namespace ep
