// ep_rows.hip -- the experts' row-wise operators over the received rows:
// SwiGLU and its gradient, MXFP4 quantization and back.
//
// All four read every value once and write every value once: they are bound
// by memory, SwiGLU to FP8 by its vector instructions (the SIMDs issue them in
// 97% of their cycles). A wave takes chunks of 512 channels of a row, 8 a lane
// (16 bytes of bf16, neighbouring lanes neighbouring addresses: 32 channels a
// lane, a whole scale group, took 2.3 times as long to write), a run of
// neighbouring chunks per wave, kUnroll chunks' loads in flight together. A
// scale group of 32 channels is four lanes, one of 128 sixteen.
//
// On MI355X: SwiGLU of 32768 rows x 2048 to bf16 68 us (403 MB, 5.95 TB/s), to
// FP8 72 us (338 MB, 4.7 TB/s), its gradient on 65536 rows 236 us (1.34 GB, 5.7
// TB/s), 16384 x 7168 values to MXFP4 55 us and back 64 us (297 MB each, 5.4 and
// 4.6 TB/s). Streams without arithmetic, of the same mixes of reads and writes:
// 6.7, 6.7, 6.3, 6.7 and 5.6 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cstdio>

#include "ep.h"
#include "ep_groups.h"

namespace {

using ep::GroupArgs;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

struct RowsArgs {
    GroupArgs g;
    int grouped;       // 0: rows [0, num_rows)
    int64_t num_rows;
    int64_t cols;      // channels of one output row (I of SwiGLU)
    const uint16_t *a; // gate_up, or the values to quantize
    const uint16_t *d; // SwiGLU's grad_out
    const uint8_t *q;  // dequantization
    const uint8_t *qs;
    void *out;
    void *scales;
};

__device__ __forceinline__ float lo16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi16(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// round to nearest even; NaN stays NaN
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// 1 / (1 + exp(-g)). exp(-g) = 2^(t + r) with t = -g log2(e) rounded and r what
// the rounding and log2(e)'s own fp32 form left out, |r| < 2^-16, so that the
// error stays near that of the hardware's exp2 and reciprocal (one step each)
// for large |g| too. A result below 2^-126 (g below -87) is 0: the hardware's
// reciprocal has no subnormal results, and silu that small is none to keep.
// r is left out for |t| >= 128, where exp2 is infinite or nothing beside 1:
// from |g| = 2.36e38 on t is infinite and r no number.
__device__ __forceinline__ float sigmoid(float g) {
    constexpr float kLog2e = 1.44269502162933349609375f, kRest = 1.92596299112661746887e-8f;
    const float t = -g * kLog2e;
    const float r = fmaf(-g, kLog2e, -t) - g * kRest;
    const float x = __builtin_amdgcn_exp2f(t);
    const float y = fabsf(t) < 128.0f ? fmaf(x, r * 0.693147180559945309f, x) : x;  // (NaN: x)
    return __builtin_amdgcn_rcpf(1.0f + y);
}

// A wave's place in the list of rows: receive rows of a run of list entries.
struct RowWalk {
    const GroupArgs *g;
    const int *ends;
    int e, start, end;
    int64_t base;

    __device__ __forceinline__ void enter(int expert) {
        e = __builtin_amdgcn_readfirstlane(expert);
        start = __builtin_amdgcn_readfirstlane(e ? ends[e - 1] : 0);
        end = __builtin_amdgcn_readfirstlane(ends[e]);
        base = g->region_rows > 0 ? 0 : (int64_t)(e / g->epr) * g->cap_rows + g->offsets[e];
    }
    // receive row of list entry i >= start, i < ends[E - 1]
    __device__ __forceinline__ int64_t row(int i) {
        if (i >= end) enter(ep::group_find(ends, g->E, i));
        return g->region_rows > 0 ? ep::group_row(*g, e, i - start) : base + (i - start);
    }
};

enum Op { kSwigluBf16, kSwigluFp8, kSwigluMx4, kSwigluGrad, kQuantize, kDequantize };

constexpr int kPer = 8;     // channels per lane and chunk
constexpr int kUnroll = 2;      // chunks whose loads are in flight together
// Workgroups per CU at most, eight of which are resident: with 8, whose waves
// share all chunks out among them, SwiGLU's gradient took 260 us and MXFP4
// there and back 129, with 64 (and the hardware dealing them out) 233 and 119.
constexpr int kBlocksPerCu = 64;

// 16-byte vectors that a lane loads
template <int OP>
constexpr int kVecs = OP == kSwigluGrad ? 3 : OP == kQuantize || OP == kDequantize ? 1 : 2;

__device__ __forceinline__ u32x4 load16(const void *p) { return __builtin_nontemporal_load((const u32x4 *)p); }
template <class T>
__device__ __forceinline__ void store(T v, void *p) {
    __builtin_nontemporal_store(v, (T *)p);
}

template <int CTRL>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float lane_max(float m) {
    return fmaxf(m, __uint_as_float(from_lane<CTRL>(__float_as_uint(m))));
}

// Eight MXFP4 codes of a lane and the scale byte of its four lanes' group.
__device__ __forceinline__ uint32_t mx4_codes(const float (&f)[8], uint8_t &scale) {
    uint32_t top = 0;  // the largest magnitude's bits: NaN and infinity keep the largest exponent
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    top = max(top, from_lane<0xB1>(top));
    top = max(top, from_lane<0x4E>(top));
    const int field = (int)(top >> 23);        // floor(log2) + 127 of a normal number
    const bool bad = field == 255;
    const int e = max(field - 2, 0);           // the scale byte; subnormals and zeros: 0, which is 2^-127
    scale = bad ? 255 : (uint8_t)e;
    const float s = __uint_as_float(e == 0 ? 0x00400000u : (uint32_t)e << 23);
    uint32_t v = 0;
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, f[0], f[1], s, 0);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, f[2], f[3], s, 1);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, f[4], f[5], s, 2);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, f[6], f[7], s, 3);
    return bad ? 0 : v;
}

template <int OP>
__device__ __forceinline__ void load_lane(const RowsArgs &a, int64_t row, int64_t c, u32x4 *v) {
    const int64_t at = row * a.cols + c;
    if constexpr (OP == kDequantize) {
        v[0].x = __builtin_nontemporal_load((const uint32_t *)(a.q + at / 2));
        v[0].y = a.qs[at / 32];
    } else if constexpr (OP == kQuantize) {
        v[0] = load16(a.a + at);
    } else {
        const uint16_t *p = a.a + row * 2 * a.cols + c;
        v[0] = load16(p);
        v[1] = load16(p + a.cols);
        if constexpr (OP == kSwigluGrad) v[2] = load16(a.d + at);
    }
}

template <int OP>
__device__ __forceinline__ void write_lane(const RowsArgs &a, int64_t row, int64_t c, const u32x4 *v) {
    const int64_t at = row * a.cols + c;
    if constexpr (OP == kDequantize) {
        // scale byte b as fp32 2^(b-127); 255: NaN, which its product with any code is
        const uint32_t b = v[0].y;
        const float s = __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
        u32x4 o;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // e2m1 as fp32: exponent and mantissa bits moved up, the bias (1 against 127) made up by 2^126
                const uint32_t code = v[0].x >> (8 * k + 4 * h);
                f[h] = __uint_as_float((code & 7) << 22 | (code & 8) << 28) * 0x1p126f * s;
            }
            o[k] = pack_bf16(f[0], f[1]);
        }
        store(o, (uint16_t *)a.out + at);
    } else if constexpr (OP == kSwigluGrad) {
        u32x4 og, ou;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float dg[2], du[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float g = h ? hi16(v[0][k]) : lo16(v[0][k]), u = h ? hi16(v[1][k]) : lo16(v[1][k]);
                const float d = h ? hi16(v[2][k]) : lo16(v[2][k]);
                const float s = sigmoid(g), gs = g * s;
                dg[h] = d * u * fmaf(gs, 1.0f - s, s);
                du[h] = d * gs;
            }
            og[k] = pack_bf16(dg[0], dg[1]);
            ou[k] = pack_bf16(du[0], du[1]);
        }
        uint16_t *o = (uint16_t *)a.out + row * 2 * a.cols + c;
        store(og, o);
        store(ou, o + a.cols);
    } else {
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float g = h ? hi16(v[0][k]) : lo16(v[0][k]);
                if constexpr (OP == kQuantize)
                    f[2 * k + h] = g;
                else
                    f[2 * k + h] = g * sigmoid(g) * (h ? hi16(v[1][k]) : lo16(v[1][k]));
            }
        if constexpr (OP == kSwigluBf16) {
            store(u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])},
                  (uint16_t *)a.out + at);
        } else if constexpr (OP == kSwigluMx4 || OP == kQuantize) {
            uint8_t s;
            const uint32_t w = mx4_codes(f, s);
            store(w, (uint8_t *)a.out + at / 2);
            if ((threadIdx.x & 3) == 0) ((uint8_t *)a.scales)[at / 32] = s;
        } else {
            float m = 0.0f, z = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m = fmaxf(m, fabsf(f[i]));
                z = fmaf(f[i], 0.0f, z);  // NaN if any value is NaN or infinite
            }
            if (z != z) m = __builtin_inff();
            m = lane_max<0xB1>(m);
            m = lane_max<0x4E>(m);
            m = lane_max<0x141>(m);
            m = lane_max<0x140>(m);
            const bool bad = m == __builtin_inff();
            const float am = fmaxf(m, 1e-4f);
            const float inv = 448.0f / am;
            uint32_t q[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = fminf(fmaxf(f[4 * i + k] * inv, -448.0f), 448.0f);
                int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
                w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
                q[i] = bad ? 0x7F7F7F7Fu : (uint32_t)w;
            }
            store(u32x2{q[0], q[1]}, (uint8_t *)a.out + at);
            if ((threadIdx.x & 15) == 0) ((float *)a.scales)[at / 128] = bad ? __builtin_nanf("") : am / 448.0f;
        }
    }
}

template <int OP>
__global__ __launch_bounds__(kThreads) void k_rows(RowsArgs a) {
    constexpr int U = kUnroll;
    __shared__ int ends[ep::kGroupsMaxExperts];
    const int64_t rows = a.grouped ? ep::group_scan(a.g, ends, kThreads) : a.num_rows;
    const int lane = threadIdx.x & 63;
    const int64_t waves = (int64_t)gridDim.x * (kThreads / 64);
    const int64_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
    const int64_t chunks = (a.cols + 64 * kPer - 1) / (64 * kPer);
    const int64_t items = rows * chunks, each = items / waves, more = items % waves;
    int64_t at = wave * each + (wave < more ? wave : more);
    const int64_t last = at + each + (wave < more ? 1 : 0);
    if (at >= last) return;
    int64_t entry = at / chunks, chunk = at - entry * chunks;
    RowWalk walk{&a.g, ends, 0, 0, 0, 0};
    int64_t row = a.grouped ? walk.row((int)entry) : entry;
    while (at < last) {
        u32x4 v[U][kVecs<OP>];
        int64_t rows_u[U], cols_u[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rows_u[u] = row;
            cols_u[u] = chunk * 64 * kPer + lane * kPer;
            on[u] = at < last && cols_u[u] < a.cols;
            if (on[u]) load_lane<OP>(a, row, cols_u[u], v[u]);
            if (++at < last && ++chunk == chunks) {
                chunk = 0;
                ++entry;
                row = a.grouped ? walk.row((int)entry) : entry;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (on[u]) write_lane<OP>(a, rows_u[u], cols_u[u], v[u]);
    }
}

template <int OP>
hipError_t launch_rows(const RowsArgs &a, int64_t rows, int cus, hipStream_t s) {
    const int64_t chunks = (a.cols + 64 * kPer - 1) / (64 * kPer);
    const int64_t blocks = (rows * chunks + kThreads / 64 - 1) / (kThreads / 64);
    const int64_t most = (int64_t)cus * kBlocksPerCu;
    k_rows<OP><<<(int)(blocks < 1 ? 1 : blocks < most ? blocks : most), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// common checks of the row-wise calls; EP_OK with *rows = 0: nothing to do
int rows_args(const ep_groups *groups, int64_t num_rows, int64_t cols, RowsArgs *a, int64_t *rows) {
    a->grouped = groups != nullptr;
    a->num_rows = num_rows;
    a->cols = cols;
    a->a = a->d = nullptr;
    a->q = a->qs = nullptr;
    a->out = a->scales = nullptr;
    a->g = GroupArgs{};
    *rows = num_rows;
    if (num_rows < 0 || num_rows >= ((int64_t)1 << 31)) return EP_ERR_ARG;
    if (groups) {
        if (int r = ep::group_args(groups, &a->g)) return r;
        if (ep::group_rows(groups) != num_rows) return EP_ERR_ARG;
        const int64_t n = ep::group_rows_expected(groups);
        *rows = num_rows == 0 ? 0 : n < 1 ? 1 : n;
    }
    return EP_OK;
}

}  // namespace

namespace ep {

int hip_status(hipError_t e, const char *what) {
    if (e == hipSuccess) return EP_OK;
    std::fprintf(stderr, "libep: %s failed: %s\n", what, hipGetErrorString(e));
    return EP_ERR_HIP;
}

int device_cus(int *cus) {
    static std::atomic<int> known[64];
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return EP_ERR_HIP;
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1)
            return EP_ERR_HIP;
        if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    }
    *cus = n;
    return EP_OK;
}

int group_args(const ep_groups *g, GroupArgs *out) {
    if (!g) return EP_ERR_ARG;
    if (g->num_experts < 1 || g->num_experts > kGroupsMaxExperts) return EP_ERR_ARG;
    if (g->num_ranks < 1 || g->num_ranks > 64 || g->num_experts % g->num_ranks) return EP_ERR_ARG;
    if (g->cap_rows < 0 || g->cap_rows >= ((int64_t)1 << 31) || g->num_ranks * g->cap_rows >= ((int64_t)1 << 31))
        return EP_ERR_ARG;
    if (g->region_rows < 0 || g->rows_hint < 0) return EP_ERR_ARG;
    if (!g->counts) return EP_ERR_ARG;
    if (g->region_rows > 0) {
        if (g->offsets || g->region_rows > g->cap_rows || g->cap_rows != g->num_experts * g->region_rows)
            return EP_ERR_ARG;
    } else if (!g->offsets) {
        return EP_ERR_ARG;
    }
    if (misaligned(g->counts, 4) || misaligned(g->offsets, 4)) return EP_ERR_ALIGN;
    out->offsets = g->offsets;
    out->counts = g->counts;
    out->E = g->num_experts;
    out->R = g->num_ranks;
    out->epr = g->num_experts / g->num_ranks;
    out->cap_rows = g->cap_rows;
    out->region_rows = (int)g->region_rows;
    return EP_OK;
}

int64_t group_rows(const ep_groups *g) { return g->num_ranks * g->cap_rows; }

int64_t group_rows_expected(const ep_groups *g) {
    const int64_t all = group_rows(g);
    return g->rows_hint > 0 && g->rows_hint < all ? g->rows_hint : all;
}

}  // namespace ep

extern "C" {

int ep_swiglu(const ep_groups *groups, const uint16_t *gate_up, int64_t num_rows, int I, int form, void *out,
              void *scales, ep_stream_t stream) {
    RowsArgs a;
    int64_t rows;
    int cus = 0;
    if (form != EP_FORM_BF16 && form != EP_FORM_FP8 && form != EP_FORM_MXFP4) return EP_ERR_ARG;
    if (I < 8 || I > 65536 || I % (form == EP_FORM_BF16 ? 8 : form == EP_FORM_FP8 ? 128 : 32)) return EP_ERR_ARG;
    if (int r = rows_args(groups, num_rows, I, &a, &rows)) return r;
    if (rows == 0) return EP_OK;
    if (!gate_up || !out || (form != EP_FORM_BF16) != (scales != nullptr)) return EP_ERR_ARG;
    if (misaligned(gate_up, 16) || misaligned(out, 16) || misaligned(scales, form == EP_FORM_FP8 ? 4 : 1))
        return EP_ERR_ALIGN;
    const int64_t n = num_rows * I, out_bytes = form == EP_FORM_BF16 ? n * 2 : form == EP_FORM_FP8 ? n : n / 2;
    const int64_t scale_bytes = form == EP_FORM_FP8 ? n / 128 * 4 : n / 32;
    if (ep::overlap(out, out_bytes, gate_up, n * 4) || ep::overlap(scales, scale_bytes, gate_up, n * 4) ||
        ep::overlap(out, out_bytes, scales, scale_bytes))
        return EP_ERR_ARG;
    if (int r = ep::device_cus(&cus)) return r;
    a.a = gate_up;
    a.out = out;
    a.scales = scales;
    const hipStream_t s = (hipStream_t)stream;
    return ep::hip_status(form == EP_FORM_BF16  ? launch_rows<kSwigluBf16>(a, rows, cus, s)
                          : form == EP_FORM_FP8 ? launch_rows<kSwigluFp8>(a, rows, cus, s)
                                                : launch_rows<kSwigluMx4>(a, rows, cus, s),
                          "ep_swiglu");
}

int ep_swiglu_backward(const ep_groups *groups, const uint16_t *grad_out, const uint16_t *gate_up, int64_t num_rows,
                       int I, uint16_t *grad_gate_up, ep_stream_t stream) {
    RowsArgs a;
    int64_t rows;
    int cus = 0;
    if (I < 8 || I > 65536 || I % 8) return EP_ERR_ARG;
    if (int r = rows_args(groups, num_rows, I, &a, &rows)) return r;
    if (rows == 0) return EP_OK;
    if (!grad_out || !gate_up || !grad_gate_up) return EP_ERR_ARG;
    if (misaligned(grad_out, 16) || misaligned(gate_up, 16) || misaligned(grad_gate_up, 16)) return EP_ERR_ALIGN;
    const int64_t n = num_rows * I;  // in place every lane writes what it read alone
    if (ep::overlap(grad_gate_up, n * 4, grad_out, n * 2) ||
        (grad_gate_up != gate_up && ep::overlap(grad_gate_up, n * 4, gate_up, n * 4)))
        return EP_ERR_ARG;
    if (int r = ep::device_cus(&cus)) return r;
    a.a = gate_up;
    a.d = grad_out;
    a.out = grad_gate_up;
    return ep::hip_status(launch_rows<kSwigluGrad>(a, rows, cus, (hipStream_t)stream), "ep_swiglu_backward");
}

int ep_quantize_mxfp4(const ep_groups *groups, const uint16_t *x, int64_t num_rows, int cols, uint8_t *q,
                      uint8_t *scales, ep_stream_t stream) {
    RowsArgs a;
    int64_t rows;
    int cus = 0;
    if (cols < 32 || cols > 65536 || cols % 32) return EP_ERR_ARG;
    if (int r = rows_args(groups, num_rows, cols, &a, &rows)) return r;
    if (rows == 0) return EP_OK;
    if (!x || !q || !scales) return EP_ERR_ARG;
    if (misaligned(x, 16) || misaligned(q, 16)) return EP_ERR_ALIGN;
    const int64_t n = num_rows * cols;
    if (ep::overlap(q, n / 2, x, n * 2) || ep::overlap(scales, n / 32, x, n * 2) || ep::overlap(q, n / 2, scales, n / 32))
        return EP_ERR_ARG;
    if (int r = ep::device_cus(&cus)) return r;
    if (!groups) {  // dense rows are one long one
        a.cols = num_rows * cols;
        a.num_rows = rows = 1;
    }
    a.a = x;
    a.out = q;
    a.scales = scales;
    return ep::hip_status(launch_rows<kQuantize>(a, rows, cus, (hipStream_t)stream), "ep_quantize_mxfp4");
}

int ep_dequantize_mxfp4(const ep_groups *groups, const uint8_t *q, const uint8_t *scales, int64_t num_rows, int cols,
                        uint16_t *x, ep_stream_t stream) {
    RowsArgs a;
    int64_t rows;
    int cus = 0;
    if (cols < 32 || cols > 65536 || cols % 32) return EP_ERR_ARG;
    if (int r = rows_args(groups, num_rows, cols, &a, &rows)) return r;
    if (rows == 0) return EP_OK;
    if (!x || !q || !scales) return EP_ERR_ARG;
    if (misaligned(x, 16) || misaligned(q, 16)) return EP_ERR_ALIGN;
    const int64_t n = num_rows * cols;
    if (ep::overlap(x, n * 2, q, n / 2) || ep::overlap(x, n * 2, scales, n / 32)) return EP_ERR_ARG;
    if (int r = ep::device_cus(&cus)) return r;
    if (!groups) {
        a.cols = num_rows * cols;
        a.num_rows = rows = 1;
    }
    a.q = q;
    a.qs = scales;
    a.out = x;
    return ep::hip_status(launch_rows<kDequantize>(a, rows, cus, (hipStream_t)stream), "ep_dequantize_mxfp4");
}

}  // extern "C"
