// ep_experts.hip -- the experts' matrix products over the received rows.
//
//   product   out[p][n]    = sum_k W[e][n][k] x[p][k]          (rows p of expert e)
//   dgrad     grad_x[p][k] = sum_n grad[p][n] W[e][n][k]
//   wgrad     grad_W[e][n][k] = sum_p grad[p][n] x[p][k]
//
// One tile algorithm for all three. A workgroup computes a BM x BN tile of one
// expert; the reduction runs in steps of 128 bytes per row (64 bf16, 128 e4m3
// or 256 e2m1 values), each step's operand tiles copied from memory to LDS by
// the copy engine path of the load unit (16 bytes per lane, no registers) into
// a ring of STAGES buffers. The matrix instruction's first operand is the
// weights' side and its second the rows' side, so that a lane's four results
// are neighbours along the output row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep.h"
#include "ep_groups.h"

namespace {

using ep::GroupArgs;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

// read through the scalar cache: the kernels never write it
typedef const __attribute__((address_space(4))) float *constant_f32;

enum Form { kBf16 = EP_FORM_BF16, kFp8 = EP_FORM_FP8, kMx4 = EP_FORM_MXFP4 };

constexpr int kStepBytes = 128;  // of a row, per reduction step

// lanes whose chunk lies past the end of a row copy this one instead
__device__ const uint4 k_zero_chunk = {0, 0, 0, 0};

struct ProductArgs {
    GroupArgs g;
    const uint8_t *x;        // rows, x_bytes each
    const uint8_t *w;        // [E][w_rows][w_bytes]
    const uint8_t *x_scales; // FP8: fp32 [rows][K/128]; MX4: bytes [rows][K/32]
    const uint8_t *w_scales; // FP8: fp32 [E][ceil(N/128)][K/128]; MX4: bytes [E][N][K/32]
    uint16_t *out;           // [rows][N] bf16
    int K, N;                // reduction length and output channels
    int steps;               // reduction steps
};

// ---------------------------------------------------------------------------
// copies to LDS and waits
// ---------------------------------------------------------------------------

// Copy 16 (4) bytes per lane from `src` to LDS at `lds` + 16 (4) * lane; `lds`
// is the same in every lane. Written as asm because the compiler, which
// cannot tell the ring's buffers apart, otherwise waits for all copies in
// flight before every LDS read; the instruction has no result register, and
// the waits are wait_copies() below. M0 holds the LDS address and needs one
// wait state before its use.
__device__ __forceinline__ void copy16(const void *src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "memory");
}
__device__ __forceinline__ void copy4(const void *src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(lds) : "memory");
}

// Wait until at most `N` of this wave's copies are in flight and its LDS
// reads have returned, then meet the workgroup's other waves.
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

__device__ __forceinline__ i32x4 read16(uint32_t a) {
    return *(const __attribute__((address_space(3))) i32x4 *)(uintptr_t)a;
}

__device__ __forceinline__ uint16_t bf16_of(float f) {
    // round to nearest even; the hardware's conversion keeps NaN a NaN
    const __bf16 b = (__bf16)f;
    return __builtin_bit_cast(uint16_t, b);
}

// ---------------------------------------------------------------------------
// operand tiles in LDS
// ---------------------------------------------------------------------------

// Reduction-contiguous operand: ROWS rows of 128 bytes. Chunk c (16 bytes) of
// row r is at slot c ^ (r & 7), so that eight neighbouring rows' same chunk
// fall on different banks. A wave copies 8 rows per instruction, lane l taking
// slot l & 7 of row l >> 3.
//
// Reduction-strided operand (TR): 64 reduction rows of COLS bf16. The 32-byte
// unit u of row r is at u ^ f(r), f = (r & 3) | (r >> 3 & 1) << 2: the sixteen
// rows one transposing read touches spread over all banks.
__device__ __forceinline__ int tr_swizzle(int r) { return (r & 3) | ((r >> 1) & 4); }

// bf16 fragment (8 reduction values of one column) of column tile `ct` and
// 32-value step s from a TR tile of COLS columns
template <int COLS>
__device__ __forceinline__ i32x4 read_tr(uint32_t tile, int ct, int s) {
    const int l = threadIdx.x & 63;
    const int r = s * 32 + (l >> 4) * 8 + ((l >> 2) & 3);
    const int f = ((l >> 2) & 3) | ((l >> 2) & 4);
    const uint32_t a = tile + r * (COLS * 2) + ((ct ^ f) << 5) + (l & 3) * 8;
    typedef __attribute__((address_space(3))) s16x4 *lp;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(uintptr_t)a);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(uintptr_t)(a + 4 * COLS * 2));
    struct {
        s16x4 a, b;
    } both = {lo, hi};
    return __builtin_bit_cast(i32x4, both);
}

__device__ __forceinline__ f32x4 mfma_bf16(i32x4 a, i32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

__device__ __forceinline__ i32x8 join(i32x4 a, i32x4 b) {
    return i32x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// ---------------------------------------------------------------------------
// product and dgrad
// ---------------------------------------------------------------------------

template <int FORM, bool WTR, int BM, int BN, int WM, int WN, int STAGES>
struct Product {
    static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    static constexpr int MT = BM / 16 / WM, NT = BN / 16 / WN;  // 16 x 16 tiles per wave
    static constexpr int kXBytes = BM * kStepBytes, kWBytes = BN * kStepBytes;
    // scales of one step in LDS: FP8 one float per row; MX4 eight bytes per row of both sides
    static constexpr int kXScale = FORM == kFp8 ? (BM < 64 ? 64 : BM) * 4 : FORM == kMx4 ? (BM < 32 ? 32 : BM) * 8 : 0;
    static constexpr int kWScale = FORM == kMx4 ? BN * 8 : 0;
    static constexpr int kStage = kXBytes + kWBytes + kXScale + kWScale;
    // copies per wave and step: a multiple for all waves, so that one count of copies in flight holds for each
    static constexpr int kXIns = kXBytes / 1024, kWIns = kWBytes / 1024;
    static constexpr int kXPer = (kXIns + kWaves - 1) / kWaves, kWPer = (kWIns + kWaves - 1) / kWaves;
    static constexpr int kXsIns = kXScale / 256, kWsIns = kWScale / 256;
    static constexpr int kXsPer = (kXsIns + kWaves - 1) / kWaves, kWsPer = (kWsIns + kWaves - 1) / kWaves;
    static constexpr int kPer = kXPer + kWPer + kXsPer + kWsPer;
    static_assert(MT >= 1 && NT >= 1 && STAGES >= 2, "tile");
    static_assert(!WTR || FORM == kBf16, "only bf16 has a transposing read");

    struct Shared {
        uint8_t ring[STAGES][kStage];
        int ends[ep::kGroupsMaxExperts];
        int row[BM];
    };

    // this wave's sources: kXPer + kWPer chunks per lane, advanced by the step
    struct Sources {
        const uint8_t *x[kXPer], *w[kWPer];
        const uint8_t *xs[kXsPer > 0 ? kXsPer : 1], *ws[kWsPer > 0 ? kWsPer : 1];
    };

    static __device__ __forceinline__ int x_ins(int wave, int i) { return (wave + i * kWaves) % kXIns; }
    static __device__ __forceinline__ int w_ins(int wave, int i) { return (wave + i * kWaves) % kWIns; }

    static __device__ __forceinline__ void copy_step(const ProductArgs &a, const Sources &src, uint32_t stage, int step,
                                                     int wave, int lane, int n0) {
        const int64_t rowbytes = FORM == kBf16 ? (int64_t)a.K * 2 : FORM == kFp8 ? a.K : a.K / 2;
        const int64_t at = (int64_t)step * kStepBytes;
        const bool whole = at + kStepBytes <= rowbytes;
        const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;  // of a reduction-contiguous tile: row & 7 == lane >> 3
        const bool in = whole || at + chunk < rowbytes;
#pragma unroll
        for (int i = 0; i < kXPer; ++i)
            copy16(in ? (const void *)(src.x[i] + at) : (const void *)&k_zero_chunk, stage + x_ins(wave, i) * 1024);
#pragma unroll
        for (int i = 0; i < kWPer; ++i) {
            const int ins = w_ins(wave, i);
            const uint8_t *p;
            if (WTR) {  // 64 reduction rows of BN columns: the step's rows past the end are zeros
                const int r = (ins * 64 + lane) / (BN / 8);
                const bool ok = step * 64 + r < a.K;
                p = ok ? src.w[i] + (int64_t)step * 64 * a.N * 2 : (const uint8_t *)&k_zero_chunk;
            } else {
                p = in ? src.w[i] + at : (const uint8_t *)&k_zero_chunk;
            }
            copy16(p, stage + kXBytes + ins * 1024);
        }
        if constexpr (FORM == kFp8) {
#pragma unroll
            for (int i = 0; i < kXsPer; ++i)
                copy4(src.xs[i] + step * 4, stage + kXBytes + kWBytes + ((wave + i * kWaves) % kXsIns) * 256);
        }
        if constexpr (FORM == kMx4) {
            // two words of four scales per row and step; the last step may have one
            const bool ok = step * 8 + (lane & 1) * 4 < a.K / 32;
#pragma unroll
            for (int i = 0; i < kXsPer; ++i)
                copy4(ok ? src.xs[i] + step * 8 : (const uint8_t *)&k_zero_chunk,
                      stage + kXBytes + kWBytes + ((wave + i * kWaves) % kXsIns) * 256);
#pragma unroll
            for (int i = 0; i < kWsPer; ++i)
                copy4(ok ? src.ws[i] + step * 8 : (const uint8_t *)&k_zero_chunk,
                      stage + kXBytes + kWBytes + kXScale + ((wave + i * kWaves) % kWsIns) * 256);
        }
    }

    // one step's products of the wave's first ACT row tiles
    template <int ACT>
    static __device__ __forceinline__ void multiply(uint32_t stage, float w_scale, int wm, int wn, int lane,
                                                    f32x4 (&acc)[MT][NT]) {
        const int g = lane >> 4, r = lane & 15;
        const uint32_t xt = stage + r * kStepBytes, wt = stage + kXBytes + r * kStepBytes;
        if constexpr (FORM == kFp8) {
            const uint32_t lo = (g ^ (r & 7)) * 16, hi = ((g + 4) ^ (r & 7)) * 16;
            i32x8 wf[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint32_t t = wt + (wn * NT + j) * 16 * kStepBytes;
                wf[j] = join(read16(t + lo), read16(t + hi));
            }
#pragma unroll
            for (int i = 0; i < ACT; ++i) {
                const uint32_t t = xt + (wm + i * WM) * 16 * kStepBytes;
                const i32x8 xf = join(read16(t + lo), read16(t + hi));
                const float s = w_scale * *(const __attribute__((address_space(3))) float *)(uintptr_t)(
                                              stage + kXBytes + kWBytes + ((wm + i * WM) * 16 + r) * 4);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[j], xf, f32x4{0, 0, 0, 0}, 0, 0,
                                                                                     0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[i][j][q] = fmaf(p[q], s, acc[i][j][q]);
                }
            }
        } else {
            int wsc[NT], xsc[ACT];
            if constexpr (FORM == kMx4) {
                const uint32_t st = stage + kXBytes + kWBytes;
#pragma unroll
                for (int i = 0; i < ACT; ++i)
                    xsc[i] = *(const __attribute__((address_space(3))) uint16_t *)(uintptr_t)(
                        st + ((wm + i * WM) * 16 + r) * 8 + g * 2);
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    wsc[j] = *(const __attribute__((address_space(3))) uint16_t *)(uintptr_t)(
                        st + kXScale + ((wn * NT + j) * 16 + r) * 8 + g * 2);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                // MX4: a lane's two chunks are neighbours, as are their scales in one 16-bit word
                const uint32_t c = ((FORM == kMx4 ? 2 * g + s : 4 * s + g) ^ (r & 7)) * 16;
                i32x4 wf[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    wf[j] = WTR ? read_tr<BN>(stage + kXBytes, wn * NT + j, s)
                                : read16(wt + (wn * NT + j) * 16 * kStepBytes + c);
#pragma unroll
                for (int i = 0; i < ACT; ++i) {
                    const i32x4 xf = read16(xt + (wm + i * WM) * 16 * kStepBytes + c);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        if constexpr (FORM == kBf16) {
                            acc[i][j] = mfma_bf16(wf[j], xf, acc[i][j]);
                        } else {
                            const i32x4 z = {0, 0, 0, 0};
                            if (s == 0)
                                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                    join(wf[j], z), join(xf, z), acc[i][j], 4, 4, 0, wsc[j], 0, xsc[i]);
                            else
                                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                    join(wf[j], z), join(xf, z), acc[i][j], 4, 4, 1, wsc[j], 1, xsc[i]);
                        }
                    }
                }
            }
        }
    }

    template <int ACT>
    static __device__ __forceinline__ void reduce(const ProductArgs &a, const Sources &src, uint32_t ring, int wave,
                                                  int lane, int n0, constant_f32 w_scale_row, f32x4 (&acc)[MT][NT]) {
        const int wm = wave / WN, wn = wave % WN;
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i)
            if (i < a.steps) copy_step(a, src, ring + i * kStage, i, wave, lane, n0);
        int slot = 0, fill = STAGES - 1;
        float next_scale = FORM == kFp8 ? w_scale_row[0] : 1.0f;
        for (int step = 0; step < a.steps; ++step) {
            if (STAGES > 2 && step + STAGES - 2 < a.steps)
                wait_copies<(STAGES - 2) * kPer>();
            else
                wait_copies<0>();
            if (step + STAGES - 1 < a.steps)
                copy_step(a, src, ring + fill * kStage, step + STAGES - 1, wave, lane, n0);
            const float w_scale = next_scale;
            if constexpr (FORM == kFp8) next_scale = w_scale_row[step + 1 < a.steps ? step + 1 : step];
            multiply<ACT>(ring + slot * kStage, w_scale, wm, wn, lane, acc);
            slot = slot + 1 == STAGES ? 0 : slot + 1;
            fill = fill + 1 == STAGES ? 0 : fill + 1;
        }
    }

    static __device__ __forceinline__ void body(const ProductArgs &a, Shared &sh) {
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const uint32_t ring = lds_address(&sh.ring[0][0]);
        const int ntiles = (a.N + BN - 1) / BN;
        const int mtiles = ep::group_scan(a.g, BM, sh.ends, kThreads);
        const int64_t tiles = (int64_t)mtiles * ntiles;
        // workgroups of one XCD (block index mod 8) take neighbouring tiles: they share rows and weights in its L2
        const int grid = gridDim.x;
        const int first = grid % 8 == 0 ? (blockIdx.x % 8) * (grid / 8) + blockIdx.x / 8 : blockIdx.x;
        for (int64_t t = first; t < tiles; t += grid) {
            // expert, then groups of up to 8 row tiles, within one the row tiles first
            const int e = __builtin_amdgcn_readfirstlane(ep::group_find(sh.ends, a.g.E, (int)(t / ntiles)));
            const int et0 = __builtin_amdgcn_readfirstlane(e ? sh.ends[e - 1] : 0);
            const int em = __builtin_amdgcn_readfirstlane(sh.ends[e]) - et0;
            const int64_t lt = t - (int64_t)et0 * ntiles;
            const int band = (int)(lt / (8 * ntiles));
            const int inb = (int)(lt - (int64_t)band * 8 * ntiles);
            const int bm = min(8, em - band * 8);
            const int m0 = (band * 8 + inb % bm) * BM, n0 = inb / bm * BN;
            const int rows = __builtin_amdgcn_readfirstlane(ep::group_count(a.g, e)) - m0;  // > 0 unless the counts overflowed the scan
            if (rows <= 0) continue;
            __syncthreads();  // the last tile's reads of the ring and the row list are done
            for (int i = tid; i < BM; i += kThreads)
                sh.row[i] = (int)ep::group_row(a.g, e, m0 + (i < rows ? i : rows - 1));
            __syncthreads();

            Sources src;
            const int64_t xb = FORM == kBf16 ? (int64_t)a.K * 2 : FORM == kFp8 ? a.K : a.K / 2;
            const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
            for (int i = 0; i < kXPer; ++i) src.x[i] = a.x + sh.row[x_ins(wave, i) * 8 + (lane >> 3)] * xb + chunk;
#pragma unroll
            for (int i = 0; i < kWPer; ++i) {
                if (WTR) {  // W[e] is [K reduction rows][N columns]; columns past the end repeat the last chunk
                    const int at = w_ins(wave, i) * 64 + lane, r = at / (BN / 8), pc = at % (BN / 8);
                    const int n = n0 + ((((pc >> 1) ^ tr_swizzle(r)) << 1) | (pc & 1)) * 8;
                    src.w[i] = a.w + (((int64_t)e * a.K + r) * a.N + min(n, a.N - 8)) * 2;
                } else {  // rows past the end repeat the last one
                    const int n = min(n0 + w_ins(wave, i) * 8 + (lane >> 3), a.N - 1);
                    src.w[i] = a.w + ((int64_t)e * a.N + n) * xb + chunk;
                }
            }
            if constexpr (FORM == kFp8) {
#pragma unroll
                for (int i = 0; i < kXsPer; ++i)
                    src.xs[i] = a.x_scales +
                                (int64_t)sh.row[min(((wave + i * kWaves) % kXsIns) * 64 + lane, BM - 1)] * (a.K / 128) * 4;
            }
            if constexpr (FORM == kMx4) {
#pragma unroll
                for (int i = 0; i < kXsPer; ++i)
                    src.xs[i] = a.x_scales +
                                (int64_t)sh.row[min(((wave + i * kWaves) % kXsIns) * 32 + (lane >> 1), BM - 1)] * (a.K / 32) +
                                (lane & 1) * 4;
#pragma unroll
                for (int i = 0; i < kWsPer; ++i) {
                    const int n = min(n0 + ((wave + i * kWaves) % kWsIns) * 32 + (lane >> 1), a.N - 1);
                    src.ws[i] = a.w_scales + ((int64_t)e * a.N + n) * (a.K / 32) + (lane & 1) * 4;
                }
            }
            constant_f32 w_scale_row = nullptr;
            if constexpr (FORM == kFp8) {
                static_assert(FORM != kFp8 || 128 % (NT * 16) == 0, "a wave's channels share one weight scale");
                const int nb = min(n0 + wn * NT * 16, a.N - 1) / 128;
                w_scale_row = (constant_f32)(uintptr_t)a.w_scales + ((int64_t)e * ((a.N + 127) / 128) + nb) * (a.K / 128);
            }

            f32x4 acc[MT][NT];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
            // row tiles are dealt to the waves in turn: a tile with few rows costs each of them less
            const int act = (min(rows, BM) + 16 * WM - 1) / (16 * WM);
            if (MT >= 4 && act <= MT / 4)
                reduce<MT / 4 ? MT / 4 : 1>(a, src, ring, wave, lane, n0, w_scale_row, acc);
            else if (MT >= 2 && act <= MT / 2)
                reduce<MT / 2 ? MT / 2 : 1>(a, src, ring, wave, lane, n0, w_scale_row, acc);
            else
                reduce<MT>(a, src, ring, wave, lane, n0, w_scale_row, acc);

#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int m = (wm + i * WM) * 16 + (lane & 15);
                if (m >= rows) continue;
                uint16_t *o = a.out + (int64_t)sh.row[m] * a.N;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int n = n0 + (wn * NT + j) * 16 + (lane >> 4) * 4;
                    if (n < a.N)
                        *(u16x4 *)(o + n) = u16x4{bf16_of(acc[i][j].x), bf16_of(acc[i][j].y), bf16_of(acc[i][j].z),
                                                  bf16_of(acc[i][j].w)};
                }
            }
        }
    }
};

template <int FORM, bool WTR, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM *WN * 64) void k_product(ProductArgs a) {
    using P = Product<FORM, WTR, BM, BN, WM, WN, STAGES>;
    __shared__ typename P::Shared sh;
    P::body(a, sh);
}


// ---------------------------------------------------------------------------
// wgrad
// ---------------------------------------------------------------------------

struct WgradArgs {
    GroupArgs g;
    const uint8_t *x;     // rows [..][K] bf16
    const uint8_t *grad;  // rows [..][N] bf16
    void *out;            // [E][N][K] fp32 or bf16
    int K, N;
    int out_f32, accumulate;
};

// grad_W[e][n][k] = sum over e's rows: both operands are reduction-strided and
// read through the transposing read. A BM (n) x BN (k) tile, 64 rows a step;
// rows past the expert's last are zeros on both sides, so that whatever the
// unused receive rows hold (NaN included) does not enter a sum.
template <int BM, int BN, int WM, int WN, int STAGES>
struct Wgrad {
    static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    static constexpr int MT = BM / 16 / WM, NT = BN / 16 / WN;
    static constexpr int kGBytes = 64 * BM * 2, kXBytes = 64 * BN * 2, kStage = kGBytes + kXBytes;
    static constexpr int kGPer = kGBytes / 1024 / kWaves, kXPer = kXBytes / 1024 / kWaves, kPer = kGPer + kXPer;
    static_assert(kGPer * kWaves * 1024 == kGBytes && kXPer * kWaves * 1024 == kXBytes, "whole copies per wave");

    struct Shared {
        uint8_t ring[STAGES][kStage];
    };

    template <int COLS, int PER>
    static __device__ __forceinline__ void copy_side(const WgradArgs &a, const uint8_t *rows, int width, int c0, int e,
                                                     int64_t base, int count, int step, uint32_t tile, int wave,
                                                     int lane) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int ins = wave + i * kWaves;
            const int at = ins * 64 + lane, r = at / (COLS / 8), pc = at % (COLS / 8);
            const int c = min(c0 + ((((pc >> 1) ^ tr_swizzle(r)) << 1) | (pc & 1)) * 8, width - 8);
            const int m = step * 64 + r;
            const uint8_t *p = (const uint8_t *)&k_zero_chunk;
            if (m < count) p = rows + ((a.g.region_rows > 0 ? ep::group_row(a.g, e, m) : base + m) * width + c) * 2;
            copy16(p, tile + ins * 1024);
        }
    }

    static __device__ __forceinline__ void body(const WgradArgs &a, Shared &sh) {
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const uint32_t ring = lds_address(&sh.ring[0][0]);
        const int nt = (a.N + BM - 1) / BM, kt = (a.K + BN - 1) / BN;
        const int64_t tiles = (int64_t)a.g.E * nt * kt;
        const int grid = gridDim.x;
        const int first = grid % 8 == 0 ? (blockIdx.x % 8) * (grid / 8) + blockIdx.x / 8 : blockIdx.x;
        for (int64_t t = first; t < tiles; t += grid) {
            const int e = __builtin_amdgcn_readfirstlane((int)(t / (nt * kt)));
            const int lt = __builtin_amdgcn_readfirstlane((int)(t - (int64_t)e * nt * kt));
            const int band = lt / (8 * kt), inb = lt - band * 8 * kt, bm = min(8, nt - band * 8);
            const int n0 = (band * 8 + inb % bm) * BM, k0 = inb / bm * BN;
            const int count = __builtin_amdgcn_readfirstlane(ep::group_count(a.g, e));
            const int64_t base = a.g.region_rows > 0 || count == 0
                                     ? 0
                                     : (int64_t)(e / a.g.epr) * a.g.cap_rows + a.g.offsets[e];
            const int steps = (count + 63) / 64;
            __syncthreads();  // the last tile's reads of the ring are done

            f32x4 acc[MT][NT];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
            auto copy_step = [&](int step, int slot) {
                const uint32_t st = ring + slot * kStage;
                copy_side<BM, kGPer>(a, a.grad, a.N, n0, e, base, count, step, st, wave, lane);
                copy_side<BN, kXPer>(a, a.x, a.K, k0, e, base, count, step, st + kGBytes, wave, lane);
            };
#pragma unroll
            for (int i = 0; i < STAGES - 1; ++i)
                if (i < steps) copy_step(i, i);
            int slot = 0, fill = STAGES - 1;
            for (int step = 0; step < steps; ++step) {
                if (STAGES > 2 && step + STAGES - 2 < steps)
                    wait_copies<(STAGES - 2) * kPer>();
                else
                    wait_copies<0>();
                if (step + STAGES - 1 < steps) copy_step(step + STAGES - 1, fill);
                const uint32_t st = ring + slot * kStage;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    i32x4 xf[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) xf[j] = read_tr<BN>(st + kGBytes, wn * NT + j, s);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const i32x4 gf = read_tr<BM>(st, wm + i * WM, s);
#pragma unroll
                        for (int j = 0; j < NT; ++j) acc[i][j] = mfma_bf16(xf[j], gf, acc[i][j]);
                    }
                }
                slot = slot + 1 == STAGES ? 0 : slot + 1;
                fill = fill + 1 == STAGES ? 0 : fill + 1;
            }

#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int n = n0 + (wm + i * WM) * 16 + (lane & 15);
                if (n >= a.N) continue;
                const int64_t row = ((int64_t)e * a.N + n) * a.K;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int k = k0 + (wn * NT + j) * 16 + (lane >> 4) * 4;
                    if (k >= a.K) continue;
                    if (a.out_f32) {
                        f32x4 *o = (f32x4 *)((float *)a.out + row + k);
                        *o = a.accumulate ? *o + acc[i][j] : acc[i][j];
                    } else {
                        *(u16x4 *)((uint16_t *)a.out + row + k) = u16x4{bf16_of(acc[i][j].x), bf16_of(acc[i][j].y),
                                                                       bf16_of(acc[i][j].z), bf16_of(acc[i][j].w)};
                    }
                }
            }
        }
    }
};

template <int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM *WN * 64) void k_wgrad(WgradArgs a) {
    using P = Wgrad<BM, BN, WM, WN, STAGES>;
    __shared__ typename P::Shared sh;
    P::body(a, sh);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// A launch fills the chip with as many workgroups as it holds at once (they
// loop over the tiles), or fewer where there cannot be that many tiles.
template <int FORM, bool WTR, int BM, int BN, int WM, int WN, int STAGES>
hipError_t launch_product(const ProductArgs &a, int64_t rows, int cus, hipStream_t s) {
    using P = Product<FORM, WTR, BM, BN, WM, WN, STAGES>;
    constexpr int kPerCu = sizeof(typename P::Shared) * 2 <= 160 * 1024 ? 2 : 1;
    const int64_t tiles = (rows / BM + a.g.E) * ((a.N + BN - 1) / BN);
    const int grid = (int)(tiles < (int64_t)cus * kPerCu ? tiles : (int64_t)cus * kPerCu);
    k_product<FORM, WTR, BM, BN, WM, WN, STAGES><<<grid, P::kThreads, 0, s>>>(a);
    return hipGetLastError();
}

// Row tiles by the rows an expert has on average, rounded up well past it: an
// expert's weights are read once per row tile, and a row tile with few rows
// costs only the matrix instructions of the rows it has (in quarters).
template <int FORM, bool WTR>
hipError_t launch_product_form(const ProductArgs &a, int64_t rows, int cus, hipStream_t s) {
    const int64_t per = rows / a.g.E;
    if (per <= 8) return launch_product<FORM, WTR, 16, 128, 1, 4, 4>(a, rows, cus, s);
    if (per <= 48) return launch_product<FORM, WTR, 64, 128, 1, 4, 3>(a, rows, cus, s);
    return launch_product<FORM, WTR, 256, 256, 2, 4, 2>(a, rows, cus, s);
}

template <int BM, int BN, int WM, int WN, int STAGES>
hipError_t launch_wgrad(const WgradArgs &a, int cus, hipStream_t s) {
    using P = Wgrad<BM, BN, WM, WN, STAGES>;
    constexpr int kPerCu = sizeof(typename P::Shared) * 2 <= 160 * 1024 ? 2 : 1;
    const int64_t tiles = (int64_t)a.g.E * ((a.N + BM - 1) / BM) * ((a.K + BN - 1) / BN);
    const int grid = (int)(tiles < (int64_t)cus * kPerCu ? tiles : (int64_t)cus * kPerCu);
    k_wgrad<BM, BN, WM, WN, STAGES><<<grid, P::kThreads, 0, s>>>(a);
    return hipGetLastError();
}

bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

bool bad_channels(int n) { return n < 8 || n > 65536 || n % 8; }

}  // namespace

extern "C" {

int ep_expert_gemm(const ep_groups *groups, int form, const void *rows, const void *row_scales, const void *weights,
                   const void *weight_scales, int K, int N, uint16_t *out, ep_stream_t stream) {
    ProductArgs a;
    if (int r = ep::group_args(groups, &a.g)) return r;
    if (form != EP_FORM_BF16 && form != EP_FORM_FP8 && form != EP_FORM_MXFP4) return EP_ERR_ARG;
    if (bad_channels(K) || bad_channels(N)) return EP_ERR_ARG;
    if (form != EP_FORM_BF16 && K % 128) return EP_ERR_ARG;
    if (ep::group_rows(groups) == 0) return EP_OK;
    if (!rows || !weights || !out) return EP_ERR_ARG;
    if ((form != EP_FORM_BF16) != (row_scales != nullptr) || (form != EP_FORM_BF16) != (weight_scales != nullptr))
        return EP_ERR_ARG;
    if (misaligned(rows, 16) || misaligned(weights, 16) || misaligned(out, 16) || misaligned(row_scales, 4) ||
        misaligned(weight_scales, 4))
        return EP_ERR_ALIGN;
    int cus;
    if (int r = ep::device_cus(&cus)) return r;
    a.x = (const uint8_t *)rows;
    a.w = (const uint8_t *)weights;
    a.x_scales = (const uint8_t *)row_scales;
    a.w_scales = (const uint8_t *)weight_scales;
    a.out = out;
    a.K = K;
    a.N = N;
    const int64_t n = ep::group_rows_expected(groups);
    if (form == EP_FORM_BF16) {
        a.steps = (K + 63) / 64;
        return ep::hip_status(launch_product_form<kBf16, false>(a, n, cus, (hipStream_t)stream), "ep_expert_gemm");
    }
    if (form == EP_FORM_FP8) {
        a.steps = K / 128;
        return ep::hip_status(launch_product_form<kFp8, false>(a, n, cus, (hipStream_t)stream), "ep_expert_gemm");
    }
    a.steps = (K + 255) / 256;
    return ep::hip_status(launch_product_form<kMx4, false>(a, n, cus, (hipStream_t)stream), "ep_expert_gemm");
}

int ep_expert_gemm_dgrad(const ep_groups *groups, const uint16_t *grad_out, const uint16_t *weights, int K, int N,
                         uint16_t *grad_rows, ep_stream_t stream) {
    ProductArgs a;
    if (int r = ep::group_args(groups, &a.g)) return r;
    if (bad_channels(K) || bad_channels(N)) return EP_ERR_ARG;
    if (ep::group_rows(groups) == 0) return EP_OK;
    if (!grad_out || !weights || !grad_rows) return EP_ERR_ARG;
    if (misaligned(grad_out, 16) || misaligned(weights, 16) || misaligned(grad_rows, 16)) return EP_ERR_ALIGN;
    int cus;
    if (int r = ep::device_cus(&cus)) return r;
    a.x = (const uint8_t *)grad_out;
    a.w = (const uint8_t *)weights;
    a.x_scales = a.w_scales = nullptr;
    a.out = grad_rows;
    a.K = N;  // the reduction runs over the product's output channels
    a.N = K;
    a.steps = (N + 63) / 64;
    return ep::hip_status(launch_product_form<kBf16, true>(a, ep::group_rows_expected(groups), cus, (hipStream_t)stream),
                          "ep_expert_gemm_dgrad");
}

int ep_expert_gemm_wgrad(const ep_groups *groups, const uint16_t *grad_out, const uint16_t *rows, int K, int N,
                         void *grad_weights, int out_f32, int accumulate, ep_stream_t stream) {
    WgradArgs a;
    if (int r = ep::group_args(groups, &a.g)) return r;
    if (bad_channels(K) || bad_channels(N)) return EP_ERR_ARG;
    if (accumulate && !out_f32) return EP_ERR_ARG;
    if (!grad_weights) return EP_ERR_ARG;
    if (ep::group_rows(groups) > 0 && (!grad_out || !rows)) return EP_ERR_ARG;
    if (misaligned(grad_out, 16) || misaligned(rows, 16) || misaligned(grad_weights, 16)) return EP_ERR_ALIGN;
    int cus;
    if (int r = ep::device_cus(&cus)) return r;
    a.x = (const uint8_t *)rows;
    a.grad = (const uint8_t *)grad_out;
    a.out = grad_weights;
    a.K = K;
    a.N = N;
    a.out_f32 = out_f32 != 0;
    a.accumulate = accumulate != 0;
    const int64_t big = (int64_t)a.g.E * ((N + 255) / 256) * ((K + 255) / 256);
    const hipError_t e = big >= cus ? launch_wgrad<256, 256, 2, 4, 2>(a, cus, (hipStream_t)stream)
                                    : launch_wgrad<128, 128, 2, 2, 2>(a, cus, (hipStream_t)stream);
    return ep::hip_status(e, "ep_expert_gemm_wgrad");
}

}  // extern "C"
