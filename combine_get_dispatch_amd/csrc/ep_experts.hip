// ep_experts.hip -- the experts' matrix products over the received rows.
//
//   product   out[p][n]    = sum_k W[e][n][k] x[p][k]          (rows p of expert e)
//   dgrad     grad_x[p][k] = sum_n grad[p][n] W[e][n][k]
//   wgrad     grad_W[e][n][k] = sum_p grad[p][n] x[p][k]
//
// One tile algorithm for all three. A workgroup computes a tile of one expert;
// the reduction runs in steps of 128 bytes per row (64 bf16, 128 e4m3 or 256
// e2m1 values), each step's operand tiles copied from memory to LDS without
// passing registers (16 bytes a lane) into a ring of two to four buffers. The
// matrix instruction's first operand is the weights' side and its second the
// rows' side, so that a lane's four results are neighbours along the output
// row.
//
// Two shapes. 256 rows x 256 channels, one workgroup per CU: four waves of 128
// x 128 results, the fewest LDS bytes per product that the registers allow
// (FP8, whose sums pass through vector registers to be scaled: eight waves of
// 128 x 64). 128 x 128, two workgroups per CU, where an expert has few rows
// and the weights' bytes are the time. On MI355X: gradients of 32768 rows, 8
// experts of 4096 x 7168: 1.27 PFLOP/s (a library product of that size 1.52);
// FP8, 32768 rows on 8 experts of the same size: 2.25 PFLOP/s (2.94), on 64,
// ragged, 1.76; MXFP4, 16384 rows: 3.8 PFLOP/s; 1024 rows on 256 experts, 7.4 GB
// of FP8 weights: 1090 us, 6.8 TB/s. What bounds the large ones: bf16 the clock
// under matrix instructions; FP8 no one thing (the matrix unit works 57% of the
// time, beside it 148 vector instructions a step and wave, most of them scale
// additions); MXFP4 the ring's filling and the results' writes around 28 steps,
// and LDS bank conflicts (17% of the cycles).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ep.h"
#include "ep_groups.h"

namespace {

using ep::GroupArgs;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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

// a pointer that is the same in every lane, in scalar registers as the copies' base has to be
__device__ __forceinline__ const uint8_t *uniform(const uint8_t *p) {
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const uint8_t *)((uint64_t)hi << 32 | lo);
}

// Copy 16 (4) bytes per lane from base + off to LDS at `lds` + 16 (4) * lane;
// base and lds are the same in every lane. Written as asm because the
// compiler, which cannot tell the ring's buffers apart, otherwise waits for
// all copies in flight before every LDS read; the instruction has no result
// register, and the waits are wait_copies() below. M0 holds the LDS address
// and needs one wait state before its use. The compiler reserves M0 (its
// register allocation never uses it, and it takes no clobber by that name);
// no other instruction of the kernels writes or reads it. A base that a vector
// instruction wrote needs five wait states. A test reads both in the compiled
// kernels.
__device__ __forceinline__ void copy16(const uint8_t *base, uint32_t off, uint32_t lds) {
    base = uniform(base);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base),
                 "s"(__builtin_amdgcn_readfirstlane(lds))
                 : "memory");
}
// the same for bytes that nothing reads again: they take no other line's place in the caches
__device__ __forceinline__ void copy16_once(const uint8_t *base, uint32_t off, uint32_t lds) {
    base = uniform(base);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(off), "s"(base),
                 "s"(__builtin_amdgcn_readfirstlane(lds))
                 : "memory");
}
__device__ __forceinline__ void copy4(const uint8_t *base, uint32_t off, uint32_t lds) {
    base = uniform(base);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base),
                 "s"(__builtin_amdgcn_readfirstlane(lds))
                 : "memory");
}
// the same with an address per lane
__device__ __forceinline__ void copy16(const uint8_t *src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src),
                 "s"(__builtin_amdgcn_readfirstlane(lds))
                 : "memory");
}
__device__ __forceinline__ void copy4(const uint8_t *src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src),
                 "s"(__builtin_amdgcn_readfirstlane(lds))
                 : "memory");
}

// Wait until at most `N` of this wave's copies are in flight and its LDS
// reads have returned, then meet the workgroup's other waves.
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Keep the compiler from moving instructions across.
__device__ __forceinline__ void pin() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

template <class T>
__device__ __forceinline__ T lds_read(uint32_t a) {
    return *(const __attribute__((address_space(3))) T *)(uintptr_t)a;
}

__device__ __forceinline__ uint16_t bf16_of(float f) {
    // round to nearest even; the hardware's conversion keeps NaN a NaN
    const __bf16 b = (__bf16)f;
    return __builtin_bit_cast(uint16_t, b);
}

// A row of 16 x 16 results as bf16: `c` four neighbouring 16-channel tiles of
// a lane (row l & 15, channels 4 (l >> 4) + [0, 4) of each). Lanes exchange
// them, 4 x 4 among the groups of 16, so that a lane holds its row's 16
// channels of tile l >> 4: 32 bytes, 128 of a row with its neighbours' (four
// times fewer memory lines a store than straight from the accumulators).
__device__ __forceinline__ void to_row(const f32x4 *c, u32x4 (&out)[2]) {
    uint32_t d[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        d[j][0] = bf16_of(c[j].x) | (uint32_t)bf16_of(c[j].y) << 16;
        d[j][1] = bf16_of(c[j].z) | (uint32_t)bf16_of(c[j].w) << 16;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        u32x2 s;
        // halves of the wave between tiles 0, 2 and 1, 3, then neighbouring groups between 0, 1 and 2, 3
#define EP_SWAP(fn, i, j) s = fn(d[i][k], d[j][k], false, false), d[i][k] = s.x, d[j][k] = s.y
        EP_SWAP(__builtin_amdgcn_permlane32_swap, 0, 2);
        EP_SWAP(__builtin_amdgcn_permlane32_swap, 1, 3);
        EP_SWAP(__builtin_amdgcn_permlane16_swap, 0, 1);
        EP_SWAP(__builtin_amdgcn_permlane16_swap, 2, 3);
#undef EP_SWAP
    }
    out[0] = u32x4{d[0][0], d[0][1], d[1][0], d[1][1]};
    out[1] = u32x4{d[2][0], d[2][1], d[3][0], d[3][1]};
}

// ---------------------------------------------------------------------------
// operand tiles in LDS
// ---------------------------------------------------------------------------

// Reduction-contiguous operand: rows of 128 bytes. Chunk c (16 bytes) of row r
// is at slot c ^ (r & 7), so that eight neighbouring rows' same chunk fall on
// different banks. A wave copies 8 rows per instruction, lane l taking slot
// l & 7 of row l >> 3.
//
// Reduction-strided operand (TR): 64 reduction rows of COLS bf16. The 32-byte
// unit u of row r is at u ^ f(r), f = (r & 3) | (r >> 3 & 1) << 2: the sixteen
// rows one transposing read touches spread over all banks.
__device__ __forceinline__ int tr_swizzle(int r) { return (r & 3) | ((r >> 1) & 4); }

// the column (of COLS) and row that lane `lane` of copy `ins` of a TR tile takes
template <int COLS>
__device__ __forceinline__ void tr_place(int ins, int lane, int &row, int &col) {
    const int at = ins * 64 + lane, pc = at % (COLS / 8);
    row = at / (COLS / 8);
    col = ((((pc >> 1) ^ tr_swizzle(row)) << 1) | (pc & 1)) * 8;
}

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

__device__ __forceinline__ i32x8 join(i32x4 a, i32x4 b) {
    return i32x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// the host pass parses device code, and knows another register of this name
#if defined(__HIP_DEVICE_COMPILE__)
#define EP_ACC "+a"
#else
#define EP_ACC "+m"
#endif

// c += a b. ACC: the accumulators of a wave that has a SIMD to itself live in
// its accumulation registers and everything else in the others, which the
// compiler does not manage by itself for so many (it moves them about within
// the loop). Written as asm, the instructions are outside the compiler's
// hazard tracking: their operands come from LDS reads alone (which it does
// track), and settle() ends every step that can be a tile's last.
template <bool ACC>
__device__ __forceinline__ void mfma_bf16(i32x4 a, i32x4 b, f32x4 &c) {
    if constexpr (ACC)
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : EP_ACC(c) : "v"(a), "v"(b));
    else
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                    0, 0);
}

// as: the scale byte of the lane's 32 values of a, in the word's low byte
template <bool ACC>
__device__ __forceinline__ void mfma_mx4(i32x4 a, i32x4 b, f32x4 &c, int as, int bs) {
    if constexpr (ACC) {
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                     : EP_ACC(c)
                     : "v"(a), "v"(b), "v"(as), "v"(bs));
    } else {
        const i32x4 z = {0, 0, 0, 0};
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(a, z), join(b, z), c, 4, 4, 0, as, 0, bs);
    }
}

// the last matrix instructions' results have reached the registers (at most 16 passes of 4 cycles)
__device__ __forceinline__ void settle() {
    pin();
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    pin();
}

// ---------------------------------------------------------------------------
// the reduction
// ---------------------------------------------------------------------------

// Copies first..last of a step into its buffer: a whole step's, or one's with
// chunks past the end.
template <class P>
__device__ __forceinline__ void copy_step(const P &p, uint32_t stage, int step, int whole, int first, int last) {
    if (step < whole) {
#pragma unroll
        for (int c = 0; c < P::kPer; ++c)
            if (c >= first && c < last) p.template copy<true>(step, stage, c);
    } else if (!P::kRuns) {  // with runs of scales all steps are whole
#pragma unroll
        for (int c = 0; c < P::kPer; ++c)
            if (c >= first && c < last) p.template copy<false>(step, stage, c);
    }
}

// The ring's first steps, of the last buffer's only the copies that a step's
// predecessors make (kSoon), and the wait for the first.
template <class P>
__device__ __forceinline__ void fill_ring(const P &p, uint32_t ring, int steps, int whole) {
    constexpr int S = P::kStages;
    if constexpr (P::kRuns) p.first_run();
#pragma unroll
    for (int i = 0; i < S; ++i)
        if (i < steps) copy_step(p, ring + i * P::kStage, i, whole, 0, i == S - 1 ? P::kSoon : P::kPer);
    if (S <= steps)
        wait_copies<(S - 2) * P::kPer + P::kSoon>();
    else
        wait_copies<0>();
}

// What a step copies into the buffer that it reads out: a whole step, one with chunks past the rows' end, nothing more.
enum Copies { kLast, kWhole, kPartial };

// One tile's reduction for a wave: acc[i][j] += the products of the rows'
// side fragment i < ACT and the weights' side fragment j < NT over all steps,
// the first `whole` of which need no check for the end of the rows. A step is
// two halves of 64 bytes per row. While one half's matrix instructions run,
// the next half's fragments are read into registers (and the MXFP4 form's
// scales with them); the workgroup meets once a step, in its middle, when the
// step's buffer has been read out and the next one's must have landed; in the
// second half the copies of the step kStages ahead follow, evenly (all at its
// start they queue: 3315 us against 2998 for both gradients of 32768 rows, 8
// experts of 4096 x 7168). The order of the source is kept (pin): a few matrix
// instructions, then a read or a copy, and so on, so that the matrix unit
// always has work queued. (The last step reads a next one that is none;
// nothing uses it.) 16 x 16 matrix instructions, not 32 x 32: those take 4%
// fewer cycles, but move twice the accumulators per product, and the clock
// under them falls further (3245 us).
template <class P>
__device__ __forceinline__ void reduce(const P &p, uint32_t ring, int steps, int whole, f32x4 (&acc)[P::ACT][P::NT]) {
    constexpr int ACT = P::ACT, NT = P::NT, S = P::kStages;
    fill_ring(p, ring, steps, whole);
    typename P::Frags h0, h1;
#pragma unroll
    for (int f = 0; f < P::kReads; ++f) p.read(h0, p.place(ring, 0, 0), f);
    int slot = 0, step = 0;
    auto body = [&](auto copies) __attribute__((always_inline)) {
        constexpr int COPIES = decltype(copies)::value;
        constexpr int M = ACT * NT, R = P::kReads, C = P::kPer, H = M / (2 * C);
        const uint32_t st = ring + slot * P::kStage;
        slot = slot + 1 == S ? 0 : slot + 1;
        const uint32_t nx = ring + slot * P::kStage;
        const auto half = p.place(st, step, 1), next = p.place(nx, step + 1, 0);
#pragma unroll
        for (int m = 0; m < M; ++m) {
#pragma unroll
            for (int f = m * R / M; f < (m + 1) * R / M; ++f) p.read(h1, half, f);
            p.mfma(h0, m / NT, m % NT, acc[m / NT][m % NT]);
            if (m % 2) pin();
        }
        wait_copies<(COPIES == kLast ? 0 : (S - 2) * P::kPer)>();
#pragma unroll
        for (int m = 0; m < M; ++m) {
#pragma unroll
            for (int f = (m + H) * C / M; f < (m + 1 + H) * C / M && f < C; ++f)  // between the reads
                if (COPIES != kLast) p.template copy<COPIES == kWhole>(step + S, st, f);
#pragma unroll
            for (int f = m * R / M; f < (m + 1) * R / M; ++f) p.read(h0, next, f);
            p.mfma(h1, m / NT, m % NT, acc[m / NT][m % NT]);
            if (m % 2) pin();
        }
        if (P::kAcc && COPIES == kLast) settle();
        ++step;
    };
    while (step + S < whole) body(std::integral_constant<int, kWhole>());
    if (!P::kRuns)
        while (step + S < steps) body(std::integral_constant<int, kPartial>());
    while (step < steps) body(std::integral_constant<int, kLast>());
}

// The FP8 form's reduction: a step is one block of 128 channels, its products
// of a row tile summed by one matrix instruction from zero and added times
// the row's and the weights' scale. A row tile's sums are added while the
// next row tile's matrix instructions run, four additions behind each; the
// next fragments are read meanwhile, at the step's last row tile those of the
// next step. (K is a multiple of 128: all steps are whole.)
template <class P>
__device__ __forceinline__ void reduce_fp8(const P &p, uint32_t ring, int steps, constant_f32 w_scales,
                                           f32x4 (&acc)[P::ACT][P::NT]) {
    constexpr int ACT = P::ACT, NT = P::NT, S = P::kStages;
    static_assert(ACT == 1 || ACT % 2 == 0, "row tiles alternate between two registers");
    fill_ring(p, ring, steps, steps);
    i32x8 w[NT], x[2];
    f32x4 part[2][NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        w[j] = P::w_whole(p.w_base(ring, 0), p.w_base(ring, 1), j);
        part[1][j] = f32x4{0, 0, 0, 0};
    }
    x[0] = P::x_whole(p.x_base(ring, 0), p.x_base(ring, 1), 0);
    float s_next = P::x_scale(p.scale_base(ring, 0), 0), f = 0.0f, f_prev = 0.0f;  // times 0: there is no tile before the first
    float ws = w_scales[0];
    int slot = 0, step = 0;
    auto body = [&](auto copies) __attribute__((always_inline)) {
        constexpr int COPIES = decltype(copies)::value;
        const uint32_t pv = ring + (slot == 0 ? S - 1 : slot - 1) * P::kStage;
        const uint32_t st = ring + slot * P::kStage;
        slot = slot + 1 == S ? 0 : slot + 1;
        const uint32_t nx = ring + slot * P::kStage;
        constexpr int SOON = P::kSoon, LATE = P::kPer - SOON, L = ACT * NT >= 8 ? ACT * NT * 3 / 8 : ACT * NT;
        if (COPIES == kLast && step + S - 1 < steps) copy_step(p, pv, step + S - 1, steps, SOON, P::kPer);
        const float ws_next = w_scales[step + 1 < steps ? step + 1 : step];
        const uint32_t x0 = p.x_base(st, 0), x1 = p.x_base(st, 1), nx0 = p.x_base(nx, 0), nx1 = p.x_base(nx, 1);
        const uint32_t w0 = p.w_base(nx, 0), w1 = p.w_base(nx, 1), xs = p.scale_base(st, step);
#pragma unroll
        for (int i = 0; i < ACT; ++i) {
            const bool last = i == ACT - 1;
            if (last) {  // the step's buffer has been read out, the next one's must have landed
                wait_copies<(COPIES == kLast ? 0 : (S - 2) * P::kPer)>();
            }
            f_prev = f;
            f = s_next * ws;
            if (!last) {
                x[(i + 1) & 1] = P::x_whole(x0, x1, i + 1);
                s_next = P::x_scale(xs, i + 1);
            } else {
                s_next = P::x_scale(p.scale_base(nx, step + 1), 0);
                if (ACT > 1) x[0] = P::x_whole(nx0, nx1, 0);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const f32x4 before = part[(i + 1) & 1][j];
                part[i & 1][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    w[j], x[i & 1], f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
                const int m = i * NT + j;
#pragma unroll
                for (int c = m * LATE / L; c < (m + 1) * LATE / L && c < LATE; ++c)
                    if (COPIES == kWhole) p.template copy<true>(step + S - 1, pv, SOON + c);
                if (last) {
#pragma unroll
                    for (int c = j * SOON / NT; c < (j + 1) * SOON / NT; ++c)
                        if (COPIES == kWhole) p.template copy<true>(step + S, st, c);
                    w[j] = P::w_whole(w0, w1, j);
                }
                const int to = (i + ACT - 1) % ACT;
                if (ACT > 1) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[to][j][q] = fmaf(before[q], f_prev, acc[to][j][q]);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[0][j][q] = fmaf(part[0][j][q], f, acc[0][j][q]);
                }
                pin();
            }
            if (ACT == 1) x[0] = P::x_whole(nx0, nx1, 0);
        }
        ws = ws_next;
        ++step;
    };
    while (step + S < steps) body(std::integral_constant<int, kWhole>());
    while (step < steps) body(std::integral_constant<int, kLast>());
    if (ACT > 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[ACT - 1][j][q] = fmaf(part[1][j][q], f, acc[ACT - 1][j][q]);
    }
}

// One half's fragments: weights' side, rows' side, MXFP4 scales of both.
template <int ACT, int NT, bool SCALES>
struct HalfFrags {
    i32x4 w[NT], x[ACT];
    int ws[SCALES ? NT : 1], xs[SCALES ? ACT : 1];
};

// ---------------------------------------------------------------------------
// product and dgrad
// ---------------------------------------------------------------------------

// A tile: up to MOST = 16 * WM * MT rows of one expert by BN channels, by WM x
// WN waves. Row tiles of 16 are dealt to the WM waves in turn, so that a tile
// with few rows costs each of them as little, in steps of half, a quarter, an
// eighth (ACT row tiles per wave), of rows copied as well as multiplied.
//
// Scales are copied in runs of several steps, 16 bytes per row, where
// their rows allow it (RUNS: K % 512 == 0): a copy instruction takes a cycle
// or more per memory line its lanes touch, and every row of the scales is
// another line. (Step by step they cost 12% of a 256 x 256 tile's time.)
template <int FORM, bool WTR, int BN, int WM, int WN, int MT, bool RUNS>
struct Product {
    static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    static constexpr int MOST = 16 * WM * MT, NTILES = BN / 16 / WN;
    static constexpr bool kAccumulate = MT * NTILES >= 64;  // 256 accumulators a lane: all registers of a SIMD
    static constexpr bool kScaled = FORM != kBf16;
    // steps per run of scales, and the runs' bytes (three in LDS: one read, one or two on their way)
    static constexpr int kRun = FORM == kFp8 ? 4 : 2, kXsRun = RUNS ? MOST * 16 : 0;
    static constexpr int kWsRun = RUNS && FORM == kMx4 ? BN * 16 : 0;
    static constexpr int kRing = (BN >= 256 ? (!RUNS ? 144 : FORM == kMx4 ? 128 : 136) : RUNS ? 64 : 72) * 1024;
    static constexpr int kMaxStages = RUNS ? 3 : 4;
    static_assert(!RUNS || (FORM == kFp8 && MOST == 32 * kWaves) || (FORM == kMx4 && MOST == 64 * kWaves && BN == MOST),
                  "who copies which rows' scales");
    static_assert(!WTR || FORM == kBf16, "only bf16 has a transposing read");

    struct Shared {
        uint8_t ring[kRing];
        uint8_t scales[RUNS ? 3 * (kXsRun + kWsRun) : 16];
        int ends[ep::kGroupsMaxExperts];
        int row[MOST];
        int tiles[3];
    };

    // what a wave needs to copy and read a tile's steps, for ACT row tiles per wave; ONCE: no other tile reads these weights
    template <int ACT_, bool ONCE>
    struct Tile {
        static constexpr int ACT = ACT_, NT = NTILES, ROWS = 16 * WM * ACT;
        static constexpr int kXBytes = ROWS * kStepBytes, kWBytes = BN * kStepBytes;
        // single steps' scales follow the tiles: FP8 one float per row; MX4 eight bytes per row of both sides
        static constexpr bool kRuns = RUNS, kSingle = kScaled && !RUNS;
        static constexpr int kXScale = !kSingle ? 0 : FORM == kFp8 ? (ROWS < 64 ? 64 : ROWS) * 4 : ROWS * 8;
        static constexpr int kWScale = kSingle && FORM == kMx4 ? BN * 8 : 0;
        static constexpr int kStage = kXBytes + kWBytes + kXScale + kWScale;
        static constexpr int kStages = kRing / kStage < kMaxStages ? kRing / kStage : kMaxStages;
        // copies per step; every wave issues as many (some repeat another's), so that one count of copies in flight
        // holds for each
        static constexpr int kXIns = kXBytes / 1024, kWIns = kWBytes / 1024;
        static constexpr int kXPer = (kXIns + kWaves - 1) / kWaves, kWPer = (kWIns + kWaves - 1) / kWaves;
        static constexpr int kXsIns = kXScale / 256, kWsIns = kWScale / 256;
        static constexpr int kXsPer = (kXsIns + kWaves - 1) / kWaves, kWsPer = (kWsIns + kWaves - 1) / kWaves;
        static constexpr int kPer = kXPer + kWPer + (RUNS ? 1 : kXsPer + kWsPer);
        // of these, made right when a buffer is free; the others in the step after
        static constexpr int kSoon = FORM == kFp8 && ACT > 1 ? kPer / 3 : kPer;
        static_assert(kStages >= 2 && kPer * (kStages - 1) < 64, "ring");
        using Frags = HalfFrags<ACT, NT, FORM == kMx4>;
        static constexpr int kReads = (FORM == kMx4 ? 2 : 1) * (ACT + NT);
        static constexpr bool kAcc = kAccumulate;

        // sources: one base per operand, offsets within the tile per lane
        const uint8_t *xb, *wb, *xsb, *wsb;
        uint32_t xo[kXPer], wo[kWPer], xso[RUNS ? 2 : kXsPer > 0 ? kXsPer : 1], wso[kWsPer > 0 ? kWsPer : 1];
        uint32_t scales;  // the runs, in LDS
        int64_t wstep;   // bytes of the weights' base per step
        int row_bytes;   // of a reduction-contiguous row
        int wave, lane, K;
        // LDS offsets of this lane's reads
        uint32_t xr, wr, half[2];

        __device__ __forceinline__ Tile(const ProductArgs &a, const Shared &sh, int wave_, int lane_, int e, int n0)
            : wave(wave_), lane(lane_), K(a.K) {
            scales = lds_address(sh.scales);
            const int64_t row0 = __builtin_amdgcn_readfirstlane(sh.row[0]);
            row_bytes = FORM == kBf16 ? a.K * 2 : FORM == kFp8 ? a.K : a.K / 2;
            xb = uniform(a.x + row0 * row_bytes);
            const uint32_t chunk = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
            for (int i = 0; i < kXPer; ++i)
                xo[i] = (uint32_t)(sh.row[(wave + i * kWaves) % kXIns * 8 + (lane >> 3)] - (int)row0) * row_bytes + chunk;
            if (WTR) {  // W[e] is [K reduction rows][N columns]; columns past the end repeat the last chunk
                wb = uniform(a.w + ((int64_t)e * a.K * a.N + n0) * 2);
                wstep = (int64_t)64 * a.N * 2;
            } else {  // rows past the end repeat the last one
                wb = uniform(a.w + ((int64_t)e * a.N + n0) * row_bytes);
                wstep = kStepBytes;
            }
#pragma unroll
            for (int i = 0; i < kWPer; ++i) {
                const int ins = (wave + i * kWaves) % kWIns;
                if (WTR) {
                    int r, c;
                    tr_place<BN>(ins, lane, r, c);
                    wo[i] = ((uint32_t)r * a.N + min(c, a.N - 8 - n0)) * 2;
                } else {
                    wo[i] = (uint32_t)min(ins * 8 + (lane >> 3), a.N - 1 - n0) * row_bytes + chunk;
                }
            }
            xsb = wsb = nullptr;
            if constexpr (kScaled) {
                const int sb = FORM == kFp8 ? a.K / 128 * 4 : a.K / 32;  // bytes of a row's scales
                xsb = uniform(a.x_scales + row0 * sb);
                if constexpr (FORM == kMx4) wsb = uniform(a.w_scales + ((int64_t)e * a.N + n0) * sb);
                if constexpr (RUNS && FORM == kFp8) {  // 16 rows of 16 bytes a wave, two turns
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        xso[i] = (uint32_t)(sh.row[(i * kWaves + wave) * 16 + (lane >> 2)] - (int)row0) * sb + (lane & 3) * 4;
                } else if constexpr (RUNS) {  // 64 rows of 16 bytes a wave, half the waves each side, two turns
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = (i * (kWaves / 2) + wave % (kWaves / 2)) * 64 + lane;
                        xso[i] = (uint32_t)(wave < kWaves / 2 ? sh.row[r] - (int)row0 : min(r, a.N - 1 - n0)) * sb;
                    }
                    if (wave >= kWaves / 2) xsb = wsb;
                } else {
                    constexpr int kRow = FORM == kFp8 ? 1 : 2;  // words per row and step
#pragma unroll
                    for (int i = 0; i < kXsPer; ++i) {
                        const int at = (wave + i * kWaves) % (kXsIns > 0 ? kXsIns : 1) * 64 + lane;
                        xso[i] = (uint32_t)(sh.row[min(at / kRow, ROWS - 1)] - (int)row0) * sb + at % kRow * 4;
                    }
#pragma unroll
                    for (int i = 0; i < kWsPer; ++i) {
                        const int at = (wave + i * kWaves) % (kWsIns > 0 ? kWsIns : 1) * 64 + lane;
                        wso[i] = (uint32_t)min(at / kRow, a.N - 1 - n0) * sb + at % kRow * 4;
                    }
                }
            }
            const int g = lane >> 4, r = lane & 15, wm = wave / WN, wn = wave % WN;
            xr = wm * 16 * kStepBytes + r * kStepBytes;
            wr = kXBytes + (wn * NT * 16 + r) * kStepBytes;
            // chunks of the two halves: MX4's are neighbours, as are their scales
            half[0] = ((FORM == kMx4 ? 2 * g : g) ^ (r & 7)) * 16;
            half[1] = ((FORM == kMx4 ? 2 * g + 1 : g + 4) ^ (r & 7)) * 16;
        }

        // the wave's c-th copy of a step into the buffer at `stage`; WHOLE: no chunk of the step lies past the end (those
        // come from zeros)
        template <bool WHOLE>
        __device__ __forceinline__ void copy(int step, uint32_t stage, int c) const {
            const int64_t at = (int64_t)step * kStepBytes;
            const uint8_t *zero = (const uint8_t *)&k_zero_chunk;
            const bool in = WHOLE || (int)at + (((lane & 7) ^ (lane >> 3)) * 16) < row_bytes;
            if (c < kXPer) {
                const uint32_t to = stage + (wave + c * kWaves) % kXIns * 1024;
                if (WHOLE)
                    copy16(xb + at, xo[c], to);
                else
                    copy16(in ? xb + at + xo[c] : zero, to);
            } else if (c < kXPer + kWPer) {
                const int i = c - kXPer, ins = (wave + i * kWaves) % kWIns;
                const uint32_t to = stage + kXBytes + ins * 1024;
                if (WHOLE && ONCE) {
                    copy16_once(wb + step * wstep, wo[i], to);
                } else if (WHOLE) {
                    copy16(wb + step * wstep, wo[i], to);
                } else {
                    const bool ok = WTR ? step * 64 + (ins * 64 + lane) / (BN / 8) < K : in;
                    copy16(ok ? wb + step * wstep + wo[i] : zero, to);
                }
            } else if constexpr (RUNS) {  // this step's share of the next run
                copy_run(step / kRun + 1, step & 1);
            } else if (c < kXPer + kWPer + kXsPer) {
                const int i = c - kXPer - kWPer;
                const uint32_t to = stage + kXBytes + kWBytes + (wave + i * kWaves) % (kXsIns > 0 ? kXsIns : 1) * 256;
                if (FORM == kFp8)
                    copy4(xsb + step * 4, xso[i], to);
                else if (WHOLE)
                    copy4(xsb + step * 8, xso[i], to);
                else  // half a step: one word of four scales per row
                    copy4((lane & 1) ? zero : xsb + step * 8 + xso[i], to);
            } else {
                const int i = c - kXPer - kWPer - kXsPer;
                const uint32_t to =
                    stage + kXBytes + kWBytes + kXScale + (wave + i * kWaves) % (kWsIns > 0 ? kWsIns : 1) * 256;
                if (WHOLE)
                    copy4(wsb + step * 8, wso[i], to);
                else
                    copy4((lane & 1) ? zero : wsb + step * 8 + wso[i], to);
            }
        }

        // The wave's copy of turn `turn` of run `run` of scales, beside a step of the run before: there when that run's
        // last step is, and three runs keep clear of the one being read. Past the rows' end the last run again (not read).
        __device__ __forceinline__ void copy_run(int run, int turn) const {
            const uint8_t *base = xsb + min(run, row_bytes / (kRun * kStepBytes) - 1) * 16;
            const uint32_t off = turn ? xso[1] : xso[0], to = scales + run % 3 * (kXsRun + kWsRun);
            if constexpr (FORM == kFp8)
                copy4(base, off, to + (turn * kWaves + wave) * 256);
            else
                copy16(base, off, to + (wave < kWaves / 2 ? 0 : kXsRun) + (turn * (kWaves / 2) + wave % (kWaves / 2)) * 1024);
        }
        __device__ __forceinline__ void first_run() const {
            copy_run(0, 0);
            copy_run(0, 1);
        }

        // where a buffer's fragments of half s begin for this lane: one sum a buffer, the tiles' offsets constants
        __device__ __forceinline__ uint32_t x_base(uint32_t stage, int s) const { return stage + xr + half[s]; }
        __device__ __forceinline__ uint32_t w_base(uint32_t stage, int s) const { return stage + wr + half[s]; }
        static __device__ __forceinline__ i32x8 x_whole(uint32_t a, uint32_t b, int i) {
            const uint32_t at = i * WM * 16 * kStepBytes;
            return join(lds_read<i32x4>(a + at), lds_read<i32x4>(b + at));
        }
        static __device__ __forceinline__ i32x8 w_whole(uint32_t a, uint32_t b, int j) {
            const uint32_t at = j * 16 * kStepBytes;
            return join(lds_read<i32x4>(a + at), lds_read<i32x4>(b + at));
        }
        // the same of the row tiles' FP8 scales
        __device__ __forceinline__ uint32_t scale_base(uint32_t stage, int step) const {
            const uint32_t row = wave / WN * 16 + (lane & 15);
            return RUNS ? scales + step / kRun % 3 * kXsRun + step % kRun * 4 + row * 16 : stage + kXBytes + kWBytes + row * 4;
        }
        static __device__ __forceinline__ float x_scale(uint32_t base, int i) {
            return lds_read<float>(base + i * WM * 16 * (RUNS ? 16 : 4));
        }
        struct Half {
            uint32_t x, w, xs, stage;
            int s;
        };
        __device__ __forceinline__ Half place(uint32_t stage, int step, int s) const {
            Half h = {x_base(stage, s), w_base(stage, s), 0, stage, s};
            if constexpr (FORM == kMx4)
                h.xs = (RUNS ? scales + step / 2 % 3 * (kXsRun + kWsRun) + step % 2 * 8 : stage + kXBytes + kWBytes) +
                       (wave / WN * 16 + (lane & 15)) * (RUNS ? 16 : 8) + (lane >> 4) * 2 + s;
            return h;
        }
        // the f-th read of a half: the weights' fragments (and scales), then the rows'
        __device__ __forceinline__ void read(Frags &h, const Half &at, int f) const {
            const int i = FORM == kMx4 ? f / 2 : f;
            if (FORM == kMx4 && f % 2 == 1) {
                constexpr int kRow = RUNS ? 16 : 8;
                if (i < NT)
                    h.ws[i] = lds_read<uint8_t>(at.xs + (RUNS ? kXsRun : kXScale) + (wave % WN * NT - wave / WN + i) * 16 * kRow);
                else
                    h.xs[i - NT] = lds_read<uint8_t>(at.xs + (i - NT) * WM * 16 * kRow);
            } else if (i < NT) {
                if constexpr (WTR)
                    h.w[i] = read_tr<BN>(at.stage + kXBytes, wave % WN * NT + i, at.s);
                else
                    h.w[i] = lds_read<i32x4>(at.w + i * 16 * kStepBytes);
            } else {
                h.x[i - NT] = lds_read<i32x4>(at.x + (i - NT) * WM * 16 * kStepBytes);
            }
        }
        __device__ __forceinline__ void mfma(const Frags &h, int i, int j, f32x4 &c) const {
            if constexpr (FORM == kMx4)
                mfma_mx4<kAcc>(h.w[j], h.x[i], c, h.ws[j], h.xs[i]);
            else
                mfma_bf16<kAcc>(h.w[j], h.x[i], c);
        }
    };

    template <int ACT, bool ONCE>
    static __device__ __forceinline__ void tile(const ProductArgs &a, const Shared &sh, uint32_t ring, int wave,
                                                int lane, int e, int n0, int rows) {
        const int wm = wave / WN, wn = wave % WN;
        f32x4 acc[ACT][NTILES];
#pragma unroll
        for (int i = 0; i < ACT; ++i)
#pragma unroll
            for (int j = 0; j < NTILES; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
        const Tile<ACT, ONCE> t(a, sh, wave, lane, e, n0);
        if constexpr (FORM == kFp8) {
            static_assert(128 % (NTILES * 16) == 0, "a wave's channels share one weight scale");
            const int nb = min(n0 + wn * NTILES * 16, a.N - 1) / 128;
            reduce_fp8(t, ring, a.steps,
                       (constant_f32)(uintptr_t)a.w_scales + ((int64_t)e * ((a.N + 127) / 128) + nb) * (a.K / 128), acc);
        } else {
            reduce(t, ring, a.steps, t.row_bytes / kStepBytes, acc);
        }
#pragma unroll
        for (int i = 0; i < ACT; ++i) {
            const int m = (wm + i * WM) * 16 + (lane & 15);
            uint16_t *o = a.out + (int64_t)sh.row[m < rows ? m : 0] * a.N;
#pragma unroll
            for (int j = 0; j < NTILES; j += 4) {
                u32x4 v[2];
                to_row(acc[i] + j, v);
                const int n = n0 + (wn * NTILES + j + (lane >> 4)) * 16;
                if (m < rows && n < a.N) *(u32x4 *)(o + n) = v[0];
                if (m < rows && n + 8 < a.N) *(u32x4 *)(o + n + 8) = v[1];
            }
        }
    }

    // Tile height: the counts are known here only. The fewest rounds of the
    // grid, each as long as its tiles are high (and some 96 rows' time more,
    // for what a tile costs whatever its height): a batch whose rows are few,
    // or all on one expert, gets lower tiles on more compute units. Without the
    // 96 rows' time 32768 ragged FP8 rows on 64 experts take 1502 us in place
    // of 1096, 16384 MXFP4 rows on 8 experts 461 in place of 298 (with 300 rows'
    // time as with 96). Always at the full height 128 FP8 rows on each of 8
    // experts take 96 us in place of 81, 256 MXFP4 rows on one 41 in place of
    // 27. (That lower tiles read the weights again is not counted.)
    static __device__ __forceinline__ int choose_height(const ProductArgs &a, Shared &sh, int ntiles) {
        const int tid = threadIdx.x;
        if (tid < 3) sh.tiles[tid] = 0;
        __syncthreads();
        int t[3] = {0, 0, 0};
        for (int e = tid; e < a.g.E; e += kThreads) {
            const int c = ep::group_count(a.g, e);
            sh.ends[e] = c;
#pragma unroll
            for (int i = 0; i < 3; ++i) t[i] = ep::group_add(t[i], (int)(((int64_t)c + (MOST >> i) - 1) / (MOST >> i)));
        }
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (t[i]) atomicAdd(&sh.tiles[i], t[i]);
        __syncthreads();
        int best = MOST;
        int64_t least = INT64_MAX;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int64_t rounds = ((int64_t)sh.tiles[i] * ntiles + gridDim.x - 1) / gridDim.x;
            const int64_t cost = rounds * ((MOST >> i) + 96);
            if (cost < least) least = cost, best = MOST >> i;
        }
        for (int e = tid; e < a.g.E; e += kThreads) sh.ends[e] = (int)(((int64_t)sh.ends[e] + best - 1) / best);
        ep::group_prefix(sh.ends, a.g.E);
        return __builtin_amdgcn_readfirstlane(best);
    }

    static __device__ __forceinline__ void body(const ProductArgs &a, Shared &sh) {
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const uint32_t ring = lds_address(sh.ring);
        const int ntiles = (a.N + BN - 1) / BN;
        const int bm = choose_height(a, sh, ntiles);
        const int64_t tiles = (int64_t)sh.ends[a.g.E - 1] * ntiles;
        // workgroups of one XCD (block index mod 8) take neighbouring tiles: they share rows and weights in its L2
        const int grid = gridDim.x;
        const int first = grid % 8 == 0 ? (blockIdx.x % 8) * (grid / 8) + blockIdx.x / 8 : blockIdx.x;
        for (int64_t t = first; t < tiles; t += grid) {
            // expert, then bands of up to 8 row tiles, within one the row tiles first
            const int e = __builtin_amdgcn_readfirstlane(ep::group_find(sh.ends, a.g.E, (int)(t / ntiles)));
            const int et0 = __builtin_amdgcn_readfirstlane(e ? sh.ends[e - 1] : 0);
            const int em = __builtin_amdgcn_readfirstlane(sh.ends[e]) - et0;
            const int64_t lt = t - (int64_t)et0 * ntiles;
            const int band = (int)(lt / (8 * ntiles));
            const int inb = (int)(lt - (int64_t)band * 8 * ntiles);
            const int high = min(8, em - band * 8);
            const int m0 = (band * 8 + inb % high) * bm, n0 = inb / high * BN;
            const int rows = min(__builtin_amdgcn_readfirstlane(ep::group_count(a.g, e)) - m0, bm);
            if (rows <= 0) continue;  // the counts overflowed the scan
            __syncthreads();          // the last tile's reads of the ring and the row list are done
            for (int i = tid; i < MOST; i += kThreads)
                sh.row[i] = (int)ep::group_row(a.g, e, m0 + (i < rows ? i : rows - 1));
            __syncthreads();
            const int act = (rows + 16 * WM - 1) / (16 * WM);
            // weights that only this tile reads are streamed past the caches (128 tokens' decode on 256 experts, 7.4 GB of
            // weights: 1088 us against 1203); where several row tiles read them that loses (256 rows of one expert: 41
            // against 29)
            const bool once = BN < 256 && em == 1;
            if (MT >= 8 && act <= MT / 8)
                tile<MT / 8 ? MT / 8 : 1, false>(a, sh, ring, wave, lane, e, n0, rows);
            else if (MT >= 4 && act <= MT / 4 && once)
                tile<MT / 4 ? MT / 4 : 1, BN < 256>(a, sh, ring, wave, lane, e, n0, rows);
            else if (MT >= 4 && act <= MT / 4)
                tile<MT / 4 ? MT / 4 : 1, false>(a, sh, ring, wave, lane, e, n0, rows);
            else if (MT >= 2 && act <= MT / 2 && once)
                tile<MT / 2 ? MT / 2 : 1, BN < 256>(a, sh, ring, wave, lane, e, n0, rows);
            else if (MT >= 2 && act <= MT / 2)
                tile<MT / 2 ? MT / 2 : 1, false>(a, sh, ring, wave, lane, e, n0, rows);
            else
                tile<MT, false>(a, sh, ring, wave, lane, e, n0, rows);
        }
    }
};

template <int FORM, bool WTR, int BN, int WM, int WN, int MT, bool RUNS>
__global__ __launch_bounds__(WM *WN * 64, BN >= 256 ? 1 : 2) void k_product(ProductArgs a) {
    using P = Product<FORM, WTR, BN, WM, WN, MT, RUNS>;
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
// unused receive rows hold (NaN included) does not enter a sum. REGIONS: the
// low-latency layout, whose rows are looked up one by one.
template <int BM, int BN, int WM, int WN, bool REGIONS>
struct Wgrad {
    static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
    static constexpr int ACT = BM / 16 / WM, NT = BN / 16 / WN;
    static constexpr int kGBytes = 64 * BM * 2, kXBytes = 64 * BN * 2, kStage = kGBytes + kXBytes, kStages = 2;
    static constexpr int kGPer = kGBytes / 1024 / kWaves, kXPer = kXBytes / 1024 / kWaves, kPer = kGPer + kXPer;
    static constexpr int kSoon = kPer;
    static_assert(kGPer * kWaves * 1024 == kGBytes && kXPer * kWaves * 1024 == kXBytes, "whole copies per wave");
    using Frags = HalfFrags<ACT, NT, false>;
    static constexpr int kReads = ACT + NT;
    static constexpr bool kAcc = ACT * NT >= 64, kRuns = false;

    struct Shared {
        uint8_t ring[kStages * kStage];
    };

    const GroupArgs *g;
    const uint8_t *gb, *xb;  // bases: packed layout, the expert's first row; low-latency, the arrays
    uint32_t go[kGPer], xo[kXPer];
    int e, count, wave, lane, grow, xrow;  // rows' bytes

    __device__ __forceinline__ Wgrad(const WgradArgs &a, int e_, int count_, int n0, int k0, int wave_, int lane_)
        : g(&a.g), e(e_), count(count_), wave(wave_), lane(lane_), grow(a.N * 2), xrow(a.K * 2) {
        const int64_t base = REGIONS || count == 0 ? 0 : ep::group_row(a.g, e, 0);
        gb = uniform(a.grad + base * grow + n0 * 2);
        xb = uniform(a.x + base * xrow + k0 * 2);
        // columns past the end repeat the last chunk
#pragma unroll
        for (int i = 0; i < kGPer; ++i) {
            int r, c;
            tr_place<BM>(wave + i * kWaves, lane, r, c);
            go[i] = (uint32_t)r * grow + min(c, a.N - 8 - n0) * 2;
        }
#pragma unroll
        for (int i = 0; i < kXPer; ++i) {
            int r, c;
            tr_place<BN>(wave + i * kWaves, lane, r, c);
            xo[i] = (uint32_t)r * xrow + min(c, a.K - 8 - k0) * 2;
        }
    }

    template <bool WHOLE>
    __device__ __forceinline__ void copy(int step, uint32_t stage, int c) const {
        const bool of_grad = c < kGPer;
        const int ins = wave + (of_grad ? c : c - kGPer) * kWaves;
        const uint32_t to = stage + (of_grad ? 0 : kGBytes) + ins * 1024;
        const int width = of_grad ? grow : xrow;
        const uint8_t *base = of_grad ? gb : xb;
        const uint32_t off = of_grad ? go[c < kGPer ? c : 0] : xo[c < kGPer ? 0 : c - kGPer];
        if (WHOLE) {  // packed layout, all rows the expert's
            copy16(base + (int64_t)step * 64 * width, off, to);
            return;
        }
        const int r = (ins * 64 + lane) / ((of_grad ? BM : BN) / 8), m = step * 64 + r;
        const uint8_t *p = (const uint8_t *)&k_zero_chunk;
        if (m < count)
            p = REGIONS ? base + ep::group_row(*g, e, m) * width + (off - (uint32_t)r * width)
                        : base + (int64_t)step * 64 * width + off;
        copy16(p, to);
    }
    struct Half {
        uint32_t stage;
        int s;
    };
    __device__ __forceinline__ Half place(uint32_t stage, int, int s) const { return {stage, s}; }
    __device__ __forceinline__ void read(Frags &h, const Half &at, int f) const {
        if (f < NT)
            h.w[f] = read_tr<BN>(at.stage + kGBytes, wave % WN * NT + f, at.s);
        else
            h.x[f - NT] = read_tr<BM>(at.stage, wave / WN + (f - NT) * WM, at.s);
    }
    __device__ __forceinline__ void mfma(const Frags &h, int i, int j, f32x4 &c) const {
        mfma_bf16<kAcc>(h.w[j], h.x[i], c);
    }

    static __device__ __forceinline__ void body(const WgradArgs &a, Shared &sh) {
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WN, wn = wave % WN;
        const int nt = (a.N + BM - 1) / BM, kt = (a.K + BN - 1) / BN;
        const int64_t tiles = (int64_t)a.g.E * nt * kt;
        const int grid = gridDim.x;
        const int first = grid % 8 == 0 ? (blockIdx.x % 8) * (grid / 8) + blockIdx.x / 8 : blockIdx.x;
        for (int64_t t = first; t < tiles; t += grid) {
            const int e = __builtin_amdgcn_readfirstlane((int)(t / (nt * kt)));
            const int lt = __builtin_amdgcn_readfirstlane((int)(t - (int64_t)e * nt * kt));
            const int band = lt / (8 * kt), inb = lt - band * 8 * kt, high = min(8, nt - band * 8);
            const int n0 = (band * 8 + inb % high) * BM, k0 = inb / high * BN;
            const int count = __builtin_amdgcn_readfirstlane(ep::group_count(a.g, e));
            f32x4 acc[ACT][NT];
#pragma unroll
            for (int i = 0; i < ACT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
            if (count > 0) {
                __syncthreads();  // the last tile's reads of the ring are done
                reduce(Wgrad(a, e, count, n0, k0, wave, lane), lds_address(sh.ring), (count + 63) / 64,
                       REGIONS ? 0 : count / 64, acc);
            } else if (a.accumulate) {
                continue;
            }
#pragma unroll
            for (int i = 0; i < ACT; ++i) {
                const int n = n0 + (wm + i * WM) * 16 + (lane & 15);
                const int64_t row = ((int64_t)e * a.N + n) * a.K;
                if (a.out_f32) {
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const int k = k0 + (wn * NT + j) * 16 + (lane >> 4) * 4;
                        if (n >= a.N || k >= a.K) continue;
                        f32x4 *o = (f32x4 *)((float *)a.out + row + k);
                        *o = a.accumulate ? *o + acc[i][j] : acc[i][j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < NT; j += 4) {
                        u32x4 v[2];
                        to_row(acc[i] + j, v);
                        const int k = k0 + (wn * NT + j + (lane >> 4)) * 16;
                        if (n < a.N && k < a.K) *(u32x4 *)((uint16_t *)a.out + row + k) = v[0];
                        if (n < a.N && k + 8 < a.K) *(u32x4 *)((uint16_t *)a.out + row + k + 8) = v[1];
                    }
                }
            }
        }
    }
};

template <int BM, int BN, int WM, int WN, bool REGIONS>
__global__ __launch_bounds__(WM *WN * 64, BN >= 256 ? 1 : 2) void k_wgrad(WgradArgs a) {
    using P = Wgrad<BM, BN, WM, WN, REGIONS>;
    __shared__ typename P::Shared sh;
    P::body(a, sh);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// A launch fills the chip with as many workgroups as it holds at once (they
// loop over the tiles), or fewer where there cannot be that many tiles.
template <int FORM, bool WTR, int BN, int WM, int WN, int MT>
hipError_t launch_product(const ProductArgs &a, int grid, hipStream_t s) {
    // the MXFP4 form's small tiles have too few rows for its waves to share a run out
    constexpr bool kRuns = FORM == kFp8 || (FORM == kMx4 && BN >= 256);
    if (kRuns && a.K % 512 == 0)
        k_product<FORM, WTR, BN, WM, WN, MT, kRuns><<<grid, WM * WN * 64, 0, s>>>(a);
    else
        k_product<FORM, WTR, BN, WM, WN, MT, false><<<grid, WM * WN * 64, 0, s>>>(a);
    return hipGetLastError();
}

// 256-channel tiles of up to 256 rows where the experts have rows for them and
// there are enough for the chip, else 128-channel tiles of up to 128 rows, two
// workgroups to a CU: where the weights' bytes are the time, one streams while
// the other starts or ends its tile.
template <int FORM, bool WTR>
hipError_t launch_product_form(const ProductArgs &a, int64_t rows, int cus, hipStream_t s) {
    const int64_t experts = rows < a.g.E ? rows : a.g.E;
    const int64_t big = (rows / 256 > experts ? rows / 256 : experts) * ((a.N + 255) / 256);
    if (rows > 64 * (int64_t)a.g.E && big >= cus)
        return launch_product<FORM, WTR, 256, 2, FORM == kFp8 ? 4 : 2, 8>(a, cus, s);
    const int64_t most = (rows / 32 + experts) * ((a.N + 127) / 128);
    return launch_product<FORM, WTR, 128, 2, 2, 4>(a, (int)(most < 2 * cus ? most : 2 * cus), s);
}

template <int BM, int BN, int WM, int WN, bool REGIONS>
hipError_t launch_wgrad(const WgradArgs &a, int cus, hipStream_t s) {
    const int64_t tiles = (int64_t)a.g.E * ((a.N + BM - 1) / BM) * ((a.K + BN - 1) / BN);
    const int64_t most = (int64_t)cus * (BN >= 256 ? 1 : 2);
    const int grid = (int)(tiles < most ? tiles : most);
    k_wgrad<BM, BN, WM, WN, REGIONS><<<grid, WM * WN * 64, 0, s>>>(a);
    return hipGetLastError();
}

bool misaligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// a tile's rows lie within 4 GiB of its first: 32-bit offsets (packed rows are neighbours, an expert's regions are not)
bool far_regions(const GroupArgs &g, int row_bytes) { return (int64_t)g.R * g.region_rows * row_bytes >= (int64_t)1 << 32; }

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
    const size_t scale_align = form == EP_FORM_MXFP4 ? 16 : 4;
    if (misaligned(rows, 16) || misaligned(weights, 16) || misaligned(out, 16) || misaligned(row_scales, scale_align) ||
        misaligned(weight_scales, scale_align))
        return EP_ERR_ALIGN;
    const int64_t all = ep::group_rows(groups), E = a.g.E;
    const int64_t width = form == EP_FORM_BF16 ? K * 2 : form == EP_FORM_FP8 ? K : K / 2;
    if (far_regions(a.g, (int)width)) return EP_ERR_ARG;
    const int64_t per_row = form == EP_FORM_FP8 ? K / 128 * 4 : K / 32, out_bytes = all * N * 2;  // a row's scales
    if (ep::overlap(out, out_bytes, rows, all * width) || ep::overlap(out, out_bytes, weights, E * N * width) ||
        ep::overlap(out, out_bytes, row_scales, all * per_row) ||
        ep::overlap(out, out_bytes, weight_scales, E * (form == EP_FORM_FP8 ? (N + 127) / 128 : N) * per_row))
        return EP_ERR_ARG;
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
    if (far_regions(a.g, N * 2)) return EP_ERR_ARG;
    const int64_t all = ep::group_rows(groups);
    if (ep::overlap(grad_rows, all * K * 2, grad_out, all * N * 2) ||
        ep::overlap(grad_rows, all * K * 2, weights, (int64_t)a.g.E * N * K * 2))
        return EP_ERR_ARG;
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
    const int64_t all = ep::group_rows(groups), out_bytes = (int64_t)a.g.E * N * K * (out_f32 ? 4 : 2);
    if (ep::overlap(grad_weights, out_bytes, grad_out, all * N * 2) ||
        ep::overlap(grad_weights, out_bytes, rows, all * K * 2))
        return EP_ERR_ARG;
    int cus;
    if (int r = ep::device_cus(&cus)) return r;
    a.x = (const uint8_t *)rows;
    a.grad = (const uint8_t *)grad_out;
    a.out = grad_weights;
    a.K = K;
    a.N = N;
    a.out_f32 = out_f32 != 0;
    a.accumulate = accumulate != 0;
    // 256 x 256 tiles where there are enough for the chip and rows enough to sum, else 128 x 128 (48 experts of 7 rows,
    // 126 MB of fp32 results: 27.5 us against 58; 8 experts of 4096 rows, 4096 x 7168: 1.5 ms against 2.4). The low-latency
    // layout takes the small tile: its rows are looked up for each copy, which keeps the loop from being unrolled and puts
    // the accumulators into scratch memory (2048 rows on 64 experts of 4096 x 2048: 3.1 ms against 0.6 for packed rows)
    const int64_t big = (int64_t)a.g.E * ((N + 255) / 256) * ((K + 255) / 256);
    const bool wide = big >= cus && ep::group_rows_expected(groups) >= 128 * (int64_t)a.g.E;
    const hipStream_t s = (hipStream_t)stream;
    const hipError_t e = a.g.region_rows > 0 ? launch_wgrad<128, 128, 2, 2, true>(a, cus, s)
                         : wide              ? launch_wgrad<256, 256, 2, 2, false>(a, cus, s)
                                             : launch_wgrad<128, 128, 2, 2, false>(a, cus, s);
    return ep::hip_status(e, "ep_expert_gemm_wgrad");
}

}  // extern "C"
