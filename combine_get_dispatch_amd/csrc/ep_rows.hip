// ep_rows.hip -- the experts' row-wise operators over the received rows:
// SwiGLU and its gradient, MXFP4 quantization and back; 8-bit integers with one
// scale per row, and checkpoints in MXINT8 (each with its figures below).
//
// All read every value once and write every value once (a row of 8-bit integers
// too long for a wave's registers: twice): they are bound by memory, SwiGLU to
// FP8 by its vector instructions (the SIMDs issue them in 97% of their cycles).
// The first four: a wave takes chunks of 512 channels of a row, 8 a lane
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
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

struct RowsArgs {
    GroupArgs g;
    int grouped;       // 0: rows [0, num_rows)
    int64_t num_rows;
    int64_t cols;      // channels of one output row (I of SwiGLU)
    const uint16_t *a; // gate_up, or the values to quantize
    const uint16_t *d; // SwiGLU's grad_out
    const uint8_t *q;  // dequantization, what SwiGLU kept
    const uint8_t *qs;
    void *out;
    void *scales;
    uint8_t *keep;     // what SwiGLU keeps (its scales: scales)
    uint16_t *again;   // SwiGLU of what was kept, or NULL
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

enum Op {
    kSwigluBf16, kSwigluFp8, kSwigluMx4, kSwigluGrad, kQuantize, kDequantize,
    kQuantizeMx8, kDequantizeMx8, kSwigluKeep, kSwigluKeptGrad
};

constexpr int kPer = 8;     // channels per lane and chunk
constexpr int kUnroll = 2;      // chunks whose loads are in flight together
// Workgroups per CU at most, eight of which are resident: with 8, whose waves
// share all chunks out among them, SwiGLU's gradient took 260 us and MXFP4
// there and back 129, with 64 (and the hardware dealing them out) 233 and 119.
constexpr int kBlocksPerCu = 64;

// 16-byte vectors that a lane loads
template <int OP>
constexpr int kVecs = OP == kSwigluGrad || OP == kSwigluKeptGrad                                       ? 3
                      : OP == kQuantize || OP == kDequantize || OP == kQuantizeMx8 || OP == kDequantizeMx8 ? 1
                                                                                                       : 2;

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

// Four whole numbers as bytes: of magnitudes up to 127, each added to 1.5 * 2^23,
// whose sum has the nearest whole number (ties to even) in its low bits.
constexpr float kWhole = 12582912.0f;
__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d) {
    const uint32_t ab = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x0C0C0400);
    const uint32_t cd = __builtin_amdgcn_perm(__float_as_uint(d), __float_as_uint(c), 0x04000C0C);
    return ab | cd;
}

// MXINT8 codes of a lane's eight bf16 values and the scale byte of its four lanes' group.
__device__ __forceinline__ u32x2 mx8_codes(u32x4 w, uint8_t &scale) {
    u16x2 m = {0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[k] & 0x7FFF7FFFu));
    uint32_t top = max(m.x, m.y);
    top = max(top, from_lane<0xB1>(top));
    top = max(top, from_lane<0x4E>(top));
    const int field = (int)(top >> 7);  // as in mx4_codes; a subnormal's group: 0, which is 2^-127
    const bool bad = field == 255;
    scale = (uint8_t)field;
    uint32_t q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float z[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // x / 2^(field - 133), exact
            const uint32_t u = w[2 * i + k / 2];
            const float y = __builtin_amdgcn_ldexpf(k % 2 ? hi16(u) : lo16(u), 133 - field);
            z[k] = __builtin_amdgcn_fmed3f(y, -127.0f, 127.0f) + kWhole;
        }
        q[i] = low_bytes(z[0], z[1], z[2], z[3]);
    }
    return bad ? u32x2{0, 0} : u32x2{q[0], q[1]};
}

// 2^(b - 133), what a code of 1 stands for under the scale byte b (255: NaN)
__device__ __forceinline__ float mx8_unit(uint32_t b) {
    return b == 255 ? __builtin_nanf("") : __uint_as_float(b > 6 ? (b - 6) << 23 : 1u << (16 + b));
}
__device__ __forceinline__ float mx8_code(uint32_t word, int i) { return (float)((int)(word << (24 - 8 * i)) >> 24); }

template <int OP>
__device__ __forceinline__ void load_lane(const RowsArgs &a, int64_t row, int64_t c, u32x4 *v) {
    const int64_t at = row * a.cols + c;
    if constexpr (OP == kDequantize) {
        v[0].x = __builtin_nontemporal_load((const uint32_t *)(a.q + at / 2));
        v[0].y = a.qs[at / 32];
    } else if constexpr (OP == kDequantizeMx8) {
        const u32x2 q = __builtin_nontemporal_load((const u32x2 *)(a.q + at));
        v[0] = u32x4{q.x, q.y, a.qs[at / 32], 0};
    } else if constexpr (OP == kSwigluKeptGrad) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // gate, up
            const int64_t from = row * 2 * a.cols + h * a.cols + c;
            const u32x2 q = __builtin_nontemporal_load((const u32x2 *)(a.q + from));
            v[h] = u32x4{q.x, q.y, a.qs[from / 32], 0};
        }
        v[2] = load16(a.d + at);
    } else if constexpr (OP == kQuantize || OP == kQuantizeMx8) {
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

// ---------------------------------------------------------------------------
// 8-bit checkpoints
// ---------------------------------------------------------------------------

// what a lane makes of its eight channels: bf16 results, codes and scales
struct Made {
    u32x4 wide[3];
    u32x2 codes[2];
    uint8_t scale[2];
};

template <int OP>
__device__ __forceinline__ void make(const u32x4 *v, Made &m) {
    if constexpr (OP == kQuantizeMx8) {
        m.codes[0] = mx8_codes(v[0], m.scale[0]);
    } else if constexpr (OP == kDequantizeMx8) {
        const float unit = mx8_unit(v[0].z);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            m.wide[0][k] =
                pack_bf16(mx8_code(v[0][k / 2], k % 2 * 2) * unit, mx8_code(v[0][k / 2], k % 2 * 2 + 1) * unit);
    } else if constexpr (OP == kSwigluKeep) {
#pragma unroll
        for (int i = 0; i < 2; ++i) m.codes[i] = mx8_codes(v[i], m.scale[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float g = h ? hi16(v[0][k]) : lo16(v[0][k]);
                f[h] = g * sigmoid(g) * (h ? hi16(v[1][k]) : lo16(v[1][k]));
            }
            m.wide[0][k] = pack_bf16(f[0], f[1]);
        }
    } else {
        const float gate = mx8_unit(v[0].z), up = mx8_unit(v[1].z);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float dg[2], du[2], y[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float g = mx8_code(v[0][k / 2], k % 2 * 2 + h) * gate;
                const float u = mx8_code(v[1][k / 2], k % 2 * 2 + h) * up;
                const float d = h ? hi16(v[2][k]) : lo16(v[2][k]);
                const float s = sigmoid(g), gs = g * s;
                dg[h] = d * u * fmaf(gs, 1.0f - s, s);
                du[h] = d * gs;
                y[h] = gs * u;
            }
            m.wide[0][k] = pack_bf16(dg[0], dg[1]);
            m.wide[1][k] = pack_bf16(du[0], du[1]);
            m.wide[2][k] = pack_bf16(y[0], y[1]);
        }
    }
}

template <int OP>
__device__ __forceinline__ void write_made(const RowsArgs &a, int64_t row, int64_t c, const Made &m) {
    const int64_t at = row * a.cols + c;
    if constexpr (OP == kQuantizeMx8) {
        store(m.codes[0], (uint8_t *)a.out + at);
    } else if constexpr (OP == kDequantizeMx8) {
        store(m.wide[0], (uint16_t *)a.out + at);
    } else if constexpr (OP == kSwigluKeep) {
        store(m.wide[0], (uint16_t *)a.out + at);
#pragma unroll
        for (int i = 0; i < 2; ++i) store(m.codes[i], a.keep + row * 2 * a.cols + i * a.cols + c);  // gate, up
    } else {
        uint16_t *o = (uint16_t *)a.out + row * 2 * a.cols + c;
        store(m.wide[0], o);
        store(m.wide[1], o + a.cols);
        if (a.again) store(m.wide[2], a.again + at);
    }
}

template <int OP>
__device__ __forceinline__ void write_scales(const RowsArgs &a, int64_t row, int64_t c, const Made &m) {
    if constexpr (OP == kQuantizeMx8) {
        ((uint8_t *)a.scales)[(row * a.cols + c) / 32] = m.scale[0];
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) ((uint8_t *)a.scales)[(row * 2 * a.cols + i * a.cols + c) / 32] = m.scale[i];
    }
}

// A wave takes segments of up to C chunks of a row: all their loads, then all
// results, then all stores, the single scale bytes last. (Stores between a
// wave's loads cost more than what they overlap with: quantization of 32768 rows
// x 7168, whole rows either way, 147 us in place of 116; SwiGLU that keeps its
// input, 65536 rows x 2048, 200 us chunk by chunk and 179 by fours.) On MI355X,
// memory bounds all four: that quantization 113 us (6.3 TB/s), of 16384 rows 55.5
// and back 56.6 us (6.4 and 6.3), SwiGLU that keeps 179 us (6.0), its gradient with
// the forward result 218 us (6.2; 232 with a fourth of the workgroups). C is the same
// for every width (dense rows are one long row): in groups, a segment past its row's
// end computes chunks that are not stored. TB/s of 134e6 values in rows of 2048, 1408,
// 768, 512 and 128 channels: quantization 5.6, 5.0, 3.6, 2.8, 1.0, back 6.2, 6.0, 4.5,
// 3.5, 1.5, SwiGLU that keeps 6.2, 5.9, 5.4, 5.1, 1.8, its gradient 6.2, 6.1, 6.1, 5.9,
// 2.3.
template <int OP, int C>
__global__ __launch_bounds__(kThreads) void k_segments(RowsArgs a) {
    __shared__ int ends[ep::kGroupsMaxExperts];
    const int64_t rows = a.grouped ? ep::group_scan(a.g, ends, kThreads) : a.num_rows;
    const int lane = threadIdx.x & 63;
    const int64_t waves = (int64_t)gridDim.x * (kThreads / 64);
    const int64_t segments = (a.cols + 512 * C - 1) / (512 * C), items = rows * segments;
    RowWalk walk{&a.g, ends, 0, 0, 0, 0};
    for (int64_t item = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6)); item < items;
         item += waves) {
        const int64_t entry = segments == 1 ? item : item / segments;
        const int64_t row = a.grouped ? walk.row((int)entry) : entry;
        const int64_t c = (item - entry * segments) * 512 * C + lane * kPer;
        u32x4 v[C][kVecs<OP>];
        Made m[C];
#pragma unroll
        for (int i = 0; i < C; ++i) load_lane<OP>(a, row, c + i * 512 < a.cols ? c + i * 512 : 0, v[i]);  // past the end: any
#pragma unroll
        for (int i = 0; i < C; ++i) make<OP>(v[i], m[i]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (c + i * 512 < a.cols) write_made<OP>(a, row, c + i * 512, m[i]);
        if constexpr (OP == kQuantizeMx8 || OP == kSwigluKeep) {
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (c + i * 512 < a.cols && (lane & 3) == 0) write_scales<OP>(a, row, c + i * 512, m[i]);
        }
    }
}

template <int OP, int C>
hipError_t launch_segments(const RowsArgs &a, int64_t rows, int cus, hipStream_t s) {
    const int64_t items = rows * ((a.cols + 512 * C - 1) / (512 * C)), blocks = (items + kThreads / 64 - 1) / (kThreads / 64);
    const int64_t most = (int64_t)cus * (OP == kSwigluKeptGrad ? 256 : 64);
    k_segments<OP, C><<<(int)(blocks < 1 ? 1 : blocks < most ? blocks : most), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// 8-bit integers with one scale per row
// ---------------------------------------------------------------------------

// A wave has a row, C chunks of 512 channels of it in registers (a longer row
// is read twice, C = 0): the scale needs the largest of all. SWIGLU: of
// silu(gate) up in place of the values. On MI355X: 32768 rows x 7168 113 us (705
// MB, 6.2 TB/s), SwiGLU of 32768 rows x 2048 60 us (336 MB, 5.6 TB/s; its vector
// instructions are issued in 86% of the SIMDs' cycles), 1024 rows in the
// low-latency layout 10.1 and 8.6 us, a launch and one row's way. (16 chunks a
// lane: registers for three waves a SIMD; left to the compiler 133 us in place of
// 113, for four 206.)
template <int C, bool SWIGLU>
__global__ __launch_bounds__(kThreads, C >= 16 ? 3 : 1) void k_row_int8(RowsArgs a) {
    __shared__ int ends[ep::kGroupsMaxExperts];
    const int64_t rows = a.grouped ? ep::group_scan(a.g, ends, kThreads) : a.num_rows;
    const int lane = threadIdx.x & 63;
    const int64_t waves = (int64_t)gridDim.x * (kThreads / 64);
    RowWalk walk{&a.g, ends, 0, 0, 0, 0};
    const int chunks = (int)((a.cols + 511) / 512);
    for (int64_t entry = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6)); entry < rows;
         entry += waves) {
        const int64_t row = a.grouped ? walk.row((int)entry) : entry;
        const uint16_t *p = a.a + row * a.cols * (SWIGLU ? 2 : 1);
        auto load = [&](int i, u32x4 (&v)[SWIGLU ? 2 : 1]) __attribute__((always_inline)) {
            const int c = i * 512 + lane * 8;
            const bool in = c < a.cols;
#pragma unroll
            for (int s = 0; s < (SWIGLU ? 2 : 1); ++s) v[s] = in ? load16(p + s * a.cols + c) : u32x4{0, 0, 0, 0};
        };
        auto values = [&](const u32x4 (&v)[SWIGLU ? 2 : 1], float (&f)[8]) __attribute__((always_inline)) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float g = h ? hi16(v[0][k]) : lo16(v[0][k]);
                    if constexpr (SWIGLU)
                        f[2 * k + h] = g * sigmoid(g) * (h ? hi16(v[1][k]) : lo16(v[1][k]));
                    else
                        f[2 * k + h] = g;
                }
        };
        float m = 0.0f, z = 0.0f;
        auto largest = [&](const float (&f)[8]) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m = fmaxf(m, fabsf(f[i]));
                z = fmaf(f[i], 0.0f, z);  // NaN if any value is NaN or infinite
            }
        };
        auto write = [&](int i, const float (&f)[8], float inv, bool bad) __attribute__((always_inline)) {
            const int c = i * 512 + lane * 8;
            uint32_t q[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                q[k] = low_bytes(f[4 * k] * inv + kWhole, f[4 * k + 1] * inv + kWhole, f[4 * k + 2] * inv + kWhole,
                                 f[4 * k + 3] * inv + kWhole);
            if (c < a.cols) store(bad ? u32x2{0, 0} : u32x2{q[0], q[1]}, (uint8_t *)a.out + row * a.cols + c);
        };
        // (silu(gate) up is kept; plain values are unpacked again, in half the registers)
        float f[SWIGLU && C > 0 ? C : 1][8];
        u32x4 v[C > 0 ? C : 1][SWIGLU ? 2 : 1];
        if constexpr (C > 0) {
#pragma unroll
            for (int i = 0; i < C; ++i) load(i, v[i]);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                values(v[i], f[SWIGLU ? i : 0]);
                largest(f[SWIGLU ? i : 0]);
            }
        } else {
            for (int i = 0; i < chunks; ++i) {
                load(i, v[0]);
                values(v[0], f[0]);
                largest(f[0]);
            }
        }
        if (z != z) m = __builtin_inff();
#pragma unroll
        for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
        const bool bad = m == __builtin_inff();
        const float am = fmaxf(m, 1e-30f), inv = 127.0f / am;
        if constexpr (C > 0) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (!SWIGLU) values(v[i], f[0]);
                write(i, f[SWIGLU ? i : 0], inv, bad);
            }
        } else {
            for (int i = 0; i < chunks; ++i) {
                load(i, v[0]);
                values(v[0], f[0]);
                write(i, f[0], inv, bad);
            }
        }
        if (lane == 0) ((float *)a.scales)[row] = bad ? __builtin_nanf("") : am / 127.0f;
    }
}

// The fewest chunks in registers that hold a row; beyond 16 (SwiGLU, whose values
// are kept in 32 bits: 8) it is read twice (32768 rows x 7168 so: 204 us in place of
// 113, 1024 rows 23 in place of 10; rows that need it: 16384 x 14336 203 us, 3.5 TB/s,
// SwiGLU of 16384 x 8192 213 us, 3.2 TB/s, computed twice).
template <bool SWIGLU>
hipError_t launch_row_int8(const RowsArgs &a, int64_t rows, int cus, hipStream_t s) {
    const int64_t blocks = (rows + kThreads / 64 - 1) / (kThreads / 64), most = (int64_t)cus * kBlocksPerCu;
    const int grid = (int)(blocks < 1 ? 1 : blocks < most ? blocks : most);
    const int64_t chunks = (a.cols + 511) / 512;
    if (chunks <= 2)
        k_row_int8<2, SWIGLU><<<grid, kThreads, 0, s>>>(a);
    else if (chunks <= 4)
        k_row_int8<4, SWIGLU><<<grid, kThreads, 0, s>>>(a);
    else if (chunks <= 8)
        k_row_int8<8, SWIGLU><<<grid, kThreads, 0, s>>>(a);
    else if (!SWIGLU && chunks <= 16)
        k_row_int8<SWIGLU ? 0 : 16, SWIGLU><<<grid, kThreads, 0, s>>>(a);
    else
        k_row_int8<0, SWIGLU><<<grid, kThreads, 0, s>>>(a);
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
    a->keep = nullptr;
    a->again = nullptr;
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
    if (form != EP_FORM_BF16 && form != EP_FORM_FP8 && form != EP_FORM_MXFP4 && form != EP_FORM_INT8) return EP_ERR_ARG;
    if (I < 8 || I > 65536 || I % (form == EP_FORM_BF16 ? 8 : form == EP_FORM_FP8 ? 128 : form == EP_FORM_INT8 ? 16 : 32))
        return EP_ERR_ARG;
    if (int r = rows_args(groups, num_rows, I, &a, &rows)) return r;
    if (rows == 0) return EP_OK;
    if (!gate_up || !out || (form != EP_FORM_BF16) != (scales != nullptr)) return EP_ERR_ARG;
    if (misaligned(gate_up, 16) || misaligned(out, 16) || misaligned(scales, form == EP_FORM_MXFP4 ? 1 : 4))
        return EP_ERR_ALIGN;
    const int64_t n = num_rows * I, out_bytes = form == EP_FORM_BF16 ? n * 2 : form == EP_FORM_MXFP4 ? n / 2 : n;
    const int64_t scale_bytes = form == EP_FORM_FP8 ? n / 128 * 4 : form == EP_FORM_INT8 ? num_rows * 4 : n / 32;
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
                          : form == EP_FORM_INT8 ? launch_row_int8<true>(a, rows, cus, s)
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

int ep_quantize_int8(const ep_groups *groups, const uint16_t *x, int64_t num_rows, int cols, int8_t *q, float *scales,
                     ep_stream_t stream) {
    RowsArgs a;
    int64_t rows;
    int cus = 0;
    if (cols < 16 || cols > 65536 || cols % 16) return EP_ERR_ARG;
    if (int r = rows_args(groups, num_rows, cols, &a, &rows)) return r;
    if (rows == 0) return EP_OK;
    if (!x || !q || !scales) return EP_ERR_ARG;
    if (misaligned(x, 16) || misaligned(q, 16) || misaligned(scales, 4)) return EP_ERR_ALIGN;
    const int64_t n = num_rows * cols;
    if (ep::overlap(q, n, x, n * 2) || ep::overlap(scales, num_rows * 4, x, n * 2) ||
        ep::overlap(q, n, scales, num_rows * 4))
        return EP_ERR_ARG;
    if (int r = ep::device_cus(&cus)) return r;
    a.a = x;
    a.out = q;
    a.scales = scales;
    return ep::hip_status(launch_row_int8<false>(a, rows, cus, (hipStream_t)stream), "ep_quantize_int8");
}

int ep_quantize_mxint8(const ep_groups *groups, const uint16_t *x, int64_t num_rows, int cols, int8_t *q,
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
    if (ep::overlap(q, n, x, n * 2) || ep::overlap(scales, n / 32, x, n * 2) || ep::overlap(q, n, scales, n / 32))
        return EP_ERR_ARG;
    if (int r = ep::device_cus(&cus)) return r;
    a.a = x;
    a.out = q;
    a.scales = scales;
    if (!groups) {  // dense rows are one long one
        a.cols = num_rows * cols;
        a.num_rows = rows = 1;
    }
    return ep::hip_status(launch_segments<kQuantizeMx8, 8>(a, rows, cus, (hipStream_t)stream), "ep_quantize_mxint8");
}

int ep_dequantize_mxint8(const ep_groups *groups, const int8_t *q, const uint8_t *scales, int64_t num_rows, int cols,
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
    if (ep::overlap(x, n * 2, q, n) || ep::overlap(x, n * 2, scales, n / 32)) return EP_ERR_ARG;
    if (int r = ep::device_cus(&cus)) return r;
    if (!groups) {
        a.cols = num_rows * cols;
        a.num_rows = rows = 1;
    }
    a.q = (const uint8_t *)q;
    a.qs = scales;
    a.out = x;
    return ep::hip_status(launch_segments<kDequantizeMx8, 4>(a, rows, cus, (hipStream_t)stream), "ep_dequantize_mxint8");
}

int ep_swiglu_checkpoint(const ep_groups *groups, const uint16_t *gate_up, int64_t num_rows, int I, uint16_t *out,
                         int8_t *q, uint8_t *scales, ep_stream_t stream) {
    RowsArgs a;
    int64_t rows;
    int cus = 0;
    if (I < 32 || I > 65536 || I % 32) return EP_ERR_ARG;
    if (int r = rows_args(groups, num_rows, I, &a, &rows)) return r;
    if (rows == 0) return EP_OK;
    if (!gate_up || !out || !q || !scales) return EP_ERR_ARG;
    if (misaligned(gate_up, 16) || misaligned(out, 16) || misaligned(q, 16)) return EP_ERR_ALIGN;
    const int64_t n = num_rows * I;
    if (ep::overlap(out, n * 2, gate_up, n * 4) || ep::overlap(q, n * 2, gate_up, n * 4) ||
        ep::overlap(scales, n / 16, gate_up, n * 4) || ep::overlap(out, n * 2, q, n * 2) ||
        ep::overlap(out, n * 2, scales, n / 16) || ep::overlap(q, n * 2, scales, n / 16))
        return EP_ERR_ARG;
    if (int r = ep::device_cus(&cus)) return r;
    a.a = gate_up;
    a.out = out;
    a.keep = (uint8_t *)q;
    a.scales = scales;
    return ep::hip_status(launch_segments<kSwigluKeep, 4>(a, rows, cus, (hipStream_t)stream), "ep_swiglu_checkpoint");
}

int ep_swiglu_checkpoint_backward(const ep_groups *groups, const uint16_t *grad_out, const int8_t *q,
                                  const uint8_t *scales, int64_t num_rows, int I, uint16_t *grad_gate_up, uint16_t *out,
                                  ep_stream_t stream) {
    RowsArgs a;
    int64_t rows;
    int cus = 0;
    if (I < 32 || I > 65536 || I % 32) return EP_ERR_ARG;
    if (int r = rows_args(groups, num_rows, I, &a, &rows)) return r;
    if (rows == 0) return EP_OK;
    if (!grad_out || !q || !scales || !grad_gate_up) return EP_ERR_ARG;
    if (misaligned(grad_out, 16) || misaligned(q, 16) || misaligned(grad_gate_up, 16) || misaligned(out, 16))
        return EP_ERR_ALIGN;
    const int64_t n = num_rows * I;
    if (ep::overlap(grad_gate_up, n * 4, grad_out, n * 2) || ep::overlap(grad_gate_up, n * 4, q, n * 2) ||
        ep::overlap(grad_gate_up, n * 4, scales, n / 16) || ep::overlap(out, n * 2, grad_out, n * 2) ||
        ep::overlap(out, n * 2, q, n * 2) || ep::overlap(out, n * 2, scales, n / 16) ||
        ep::overlap(out, n * 2, grad_gate_up, n * 4))
        return EP_ERR_ARG;
    if (int r = ep::device_cus(&cus)) return r;
    a.q = (const uint8_t *)q;
    a.qs = scales;
    a.d = grad_out;
    a.out = grad_gate_up;
    a.again = out;
    return ep::hip_status(launch_segments<kSwigluKeptGrad, 2>(a, rows, cus, (hipStream_t)stream),
                          "ep_swiglu_checkpoint_backward");
}

}  // extern "C"
