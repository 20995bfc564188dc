// What the tiled products share: the epilogue, the operands' tiles in LDS and
// the loops over their summed index.  Device code, included by the kernels'
// files; not part of the public ABI.
#pragma once

#include "learn_internal.h"

namespace fa {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int STEP_BYTES = 128; // k per step, as bytes of one row
constexpr int WAVE = 64;

// Elements of an operand in 16 bytes, and the vector of sums of a fragment.
template <typename T> struct traits;
template <> struct traits<__bf16> {
    static constexpr int EPC = 8;
    typedef f32x4 sums;
};
template <> struct traits<_Float16> {
    static constexpr int EPC = 8;
    typedef f32x4 sums;
};
template <> struct traits<float> {
    static constexpr int EPC = 4;
    typedef f32x4 sums;
};
template <> struct traits<int8_t> {
    static constexpr int EPC = 16;
    typedef i32x4 sums;
};

// ------------------------------------------------------------ activations
// GELU is the exact one, z Phi(z).  With x = |z| / sqrt(2),
//     Phi(-|z|) = exp(-x^2) P(t) / 2,  t = 1 / (1 + 0.33 x),
// P a polynomial without constant term fitted to exp(x^2) erfc(x) on
// [0, 10] for the least relative error (9.4e-8 there, 5e-7 as evaluated in
// fp32).  It costs a third of the library's erff, and the slope's
// exp(-z^2 / 2) comes with it.  The sigmoid likewise uses the hardware's exp2
// and reciprocal (one unit in the last place each, results below 2^-126
// flushed).  An exponent y is rounded when it is formed, which is a relative
// error of up to 2^-24 |y| of its exp2: 8e-6 of GELU's tail at z = -13, 4e-6 of
// the sigmoid's at z = -87.  For fp32 (EXACT) what that left off is multiplied
// in; for bf16, whose results are rounded to 2^-9, it is not worth the
// instructions.

// exp(y c) for the two parts c = hi + lo of a constant and y^n = p + rest
// (rest: what p lost, 0 for y itself)
template <bool EXACT> __device__ __forceinline__ float exp_of(float p, float rest, float hi, float lo)
{
    const float y = p * hi;
    float e = __builtin_amdgcn_exp2f(y);
    if (EXACT) {
        const float off = __builtin_fmaf(p, lo, __builtin_fmaf(rest, hi, __builtin_fmaf(p, hi, -y)));
        // beyond, e is 0 or infinite and `off` may be NaN
        e *= fabsf(y) < 256.f ? __builtin_fmaf(off, 0.69314718055994531f, 1.f) : 1.f;
    }
    return e;
}

constexpr double LOG2E = 1.44269504088896340736;
constexpr float LOG2E_HI = (float)LOG2E, LOG2E_LO = (float)(LOG2E - (double)LOG2E_HI);

template <bool EXACT> __device__ __forceinline__ float phi_below(float z, float &e) // Phi(-|z|); e = exp(-z^2 / 2)
{
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(z), 0.33f * 0.70710678118654752f, 1.f));
    const float h = z * z;
    e = exp_of<EXACT>(h, EXACT ? __builtin_fmaf(z, z, -h) : 0.f, -0.5f * LOG2E_HI, -0.5f * LOG2E_LO);
    float q = -0.1353444159f;
    q = __builtin_fmaf(q, t, 0.4602320194f);
    q = __builtin_fmaf(q, t, -0.3511412442f);
    q = __builtin_fmaf(q, t, 0.4084925056f);
    q = __builtin_fmaf(q, t, 0.04722447693f);
    q = __builtin_fmaf(q, t, 0.2012227625f);
    q = __builtin_fmaf(q, t, 0.1829561144f);
    q = __builtin_fmaf(q, t, 0.1863577962f);
    return 0.5f * (q * t) * e;
}

template <bool EXACT> __device__ __forceinline__ float sigmoid(float z)
{
    return __builtin_amdgcn_rcpf(1.f + exp_of<EXACT>(z, 0.f, -LOG2E_HI, -LOG2E_LO));
}

// z[i] = act(z[i]); NaN stays NaN
template <bool EXACT, int W> __device__ __forceinline__ void apply_act(float *z, int act)
{
    if (act == FA_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < W; i++)
            z[i] = z[i] < 0.f ? 0.f : z[i];
    } else if (act == FA_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < W; i++) {
            float e;
            const float q = phi_below<EXACT>(z[i], e);
            z[i] *= z[i] > 0.f ? 1.f - q : q;
        }
    } else if (act == FA_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < W; i++)
            z[i] *= sigmoid<EXACT>(z[i]);
    }
}

// d[i] *= act'(z[i])
template <bool EXACT, int W> __device__ __forceinline__ void apply_slope(float *d, const float *z, int act)
{
    if (act == FA_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < W; i++)
            d[i] *= z[i] > 0.f ? 1.f : z[i] == z[i] ? 0.f : z[i];
    } else if (act == FA_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < W; i++) {
            float e;
            const float q = phi_below<EXACT>(z[i], e);
            d[i] *= __builtin_fmaf(z[i] * e, 0.39894228040143268f, z[i] > 0.f ? 1.f - q : q);
        }
    } else if (act == FA_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < W; i++) {
            const float s = sigmoid<EXACT>(z[i]);
            d[i] *= s * __builtin_fmaf(z[i], 1.f - s, 1.f);
        }
    }
}

// 16 bytes of T from an address that is only element-aligned, of which the
// first `valid` elements may be read; the rest are zero.
template <typename T> __device__ __forceinline__ u32x4 load_chunk(const T *p, int valid)
{
    constexpr int EPC = traits<T>::EPC;
    u32x4 r = {0, 0, 0, 0};
    if (valid >= EPC) {
        __builtin_memcpy(&r, p, 16);
    } else if (valid > 0) {
        T e[EPC];
#pragma unroll
        for (int i = 0; i < EPC; i++)
            e[i] = i < valid ? p[i] : (T)0;
        __builtin_memcpy(&r, e, 16);
    }
    return r;
}

// W consecutive values of a row, of which `valid` may be touched.  Rows are
// only element-aligned; the hardware takes such vector accesses.
template <typename T, int W> __device__ __forceinline__ void load_n(const T *p, int valid, float *v)
{
    if (valid >= W) {
        T e[W];
        __builtin_memcpy(e, p, sizeof e);
#pragma unroll
        for (int i = 0; i < W; i++)
            v[i] = (float)e[i];
    } else {
#pragma unroll
        for (int i = 0; i < W; i++)
            v[i] = i < valid ? (float)p[i] : 0.f;
    }
}

template <typename T, int W, typename V> __device__ __forceinline__ void store_n(T *p, int valid, const V *v)
{
    if (valid >= W) {
        T e[W];
#pragma unroll
        for (int i = 0; i < W; i++)
            e[i] = (T)v[i]; // round to nearest even
        __builtin_memcpy(p, e, sizeof e);
    } else {
#pragma unroll
        for (int i = 0; i < W; i++)
            if (i < valid)
                p[i] = (T)v[i];
    }
}

// W values of a row as they are stored, so that they can be fetched ahead;
// zeros where there is nothing to fetch.
template <typename T, int W> struct Raw {
    T e[W];
    __device__ __forceinline__ void fetch(const T *p, int valid)
    {
        if (valid >= W) {
            __builtin_memcpy(e, p, sizeof e);
        } else if (valid > 0) {
            // no load is under a condition of its own, so none waits for another
#pragma unroll
            for (int i = 0; i < W; i++)
                e[i] = p[i < valid ? i : valid - 1];
#pragma unroll
            for (int i = 0; i < W; i++)
                e[i] = i < valid ? e[i] : (T)0;
        } else {
#pragma unroll
            for (int i = 0; i < W; i++)
                e[i] = (T)0;
        }
    }
};

template <typename T, int W> __device__ __forceinline__ void fetch_bias(const GemmArgs &p, int n, Raw<T, W> &b)
{
    b.fetch(p.bias ? static_cast<const T *>(p.bias) + n : nullptr, p.bias ? p.N - n : 0);
}

template <typename T, int W>
__device__ __forceinline__ void fetch_residual(const GemmArgs &p, int64_t m, int n, Raw<T, W> &r)
{
    const bool any = p.res && m < p.M;
    r.fetch(any ? static_cast<const T *>(p.res) + m * p.ldr + n : nullptr, any ? p.N - n : 0);
}

// Sums of 8-bit products as the values they stand for: times the row's scale,
// then the column's, in fp32.
template <int W>
__device__ __forceinline__ void scaled_sums(const int32_t *s, float row, const float *col, float *v)
{
#pragma unroll
    for (int i = 0; i < W; i++)
        v[i] = (float)s[i] * row * col[i];
}

// out(m, n..n+W-1) from the finished sums: z = alpha s + bias, then the
// activation, then the residual, all in fp32, each result rounded once.
template <typename T, int W>
__device__ __forceinline__ void epilogue(const GemmArgs &p, int64_t m, int n, const float *s, const Raw<T, W> &bias,
                                         const Raw<T, W> &res)
{
    const int valid = p.N - n;
    float z[W];
#pragma unroll
    for (int i = 0; i < W; i++)
        z[i] = __builtin_fmaf(p.alpha, s[i], (float)bias.e[i]);
    if (p.pre)
        store_n<T, W>(static_cast<T *>(p.pre) + m * p.ldp + n, valid, z);
    apply_act<sizeof(T) == 4, W>(z, p.act);
    if (p.res) {
#pragma unroll
        for (int i = 0; i < W; i++)
            z[i] += (float)res.e[i];
    }
    store_n<T, W>(static_cast<T *>(p.out) + m * p.ldo + n, valid, z);
}

// ------------------------------------------------------------ LDS tiles
// An inner operand's tile holds `rows` rows of STEP bytes; its 16-byte chunk c
// of row r lies at chunk c ^ inner_swizzle(r), so the 16 rows that a fragment
// read touches spread over all banks.  An outer operand's tile holds one row of
// `cols` elements per k; there the chunks of row k are exchanged by
// outer_swizzle, so the rows that one transposing read touches do.
template <typename T, int COLS> __device__ __forceinline__ int outer_swizzle(int k)
{
    constexpr int CPR = COLS * (int)sizeof(T) / 16;
    if constexpr (sizeof(T) == 2)
        return (((k & 3) | ((k >> 1) & 4)) << 1) & (CPR - 1);
    else
        return (((k >> 2) & 3) << 2) & (CPR - 1);
}

template <int STEP> __device__ __forceinline__ int inner_swizzle(int r)
{
    return STEP == 128 ? r & 7 : (r >> 1) & 3;
}

struct Frag {
    u32x4 v; // 16-bit types: 8 values of k;  fp32: 4;  8-bit integers: 16
};

// Fragment of 16 rows (or columns) starting at r0, the 64 bytes kk of the
// step's k: lane l holds row l % 16 and the 16 bytes of group l / 16.
template <typename T, bool OUTER, int ROWS, int STEP>
__device__ __forceinline__ Frag read_frag(const char *tile, int r0, int kk, int lane)
{
    const int i = lane & 15, g = lane >> 4;
    Frag f;
    if constexpr (!OUTER) {
        const int r = r0 + i, c = g + 4 * kk;
        f.v = *reinterpret_cast<const u32x4 *>(tile + (r * STEP + ((c ^ inner_swizzle<STEP>(r)) << 4)));
    } else if constexpr (sizeof(T) == 2) {
        // Two transposing reads, k = 8g .. 8g+3 and 8g+4 .. 8g+7.  Within 16
        // lanes, lane i supplies the address of row i/4, columns 4(i%4) and
        // up, and receives column i of the four rows.
        s16x4 h[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int k = kk * 32 + 8 * g + 4 * j + (i >> 2);
            const int col = r0 + (i & 3) * 4;
            const int c = (col >> 3) ^ outer_swizzle<T, ROWS>(k);
            const char *at = tile + (k * (ROWS * 2) + (c << 4) + ((col & 4) << 1));
            h[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4 *)const_cast<char *>(at));
        }
        const u32x2 a = __builtin_bit_cast(u32x2, h[0]), b = __builtin_bit_cast(u32x2, h[1]);
        f.v = u32x4{a.x, a.y, b.x, b.y};
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int k = kk * 16 + 4 * g + j, col = r0 + i;
            const int c = (col >> 2) ^ outer_swizzle<T, ROWS>(k);
            f.v[j] = *reinterpret_cast<const uint32_t *>(tile + (k * (ROWS * 4) + (c << 4) + ((col & 3) << 2)));
        }
    }
    return f;
}

// acc += the 16x16 product of the two fragments.  The rows of the result are
// B's (n), the columns A's (m): lane l then holds m = l % 16 and the four
// consecutive n = 4 (l / 16) + i, which the epilogue writes as one vector.
// For fp32, element j of a fragment is the summed index 4 (l / 16) + j of
// both operands, so the four products of 4 cover the 16.
template <typename T>
__device__ __forceinline__ typename traits<T>::sums mma(const Frag &b, const Frag &a, typename traits<T>::sums acc)
{
    if constexpr (__is_same(T, __bf16)) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b.v),
                                                       __builtin_bit_cast(bf16x8, a.v), acc, 0, 0, 0);
    } else if constexpr (__is_same(T, _Float16)) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b.v),
                                                      __builtin_bit_cast(f16x8, a.v), acc, 0, 0, 0);
    } else if constexpr (__is_same(T, int8_t)) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b.v), __builtin_bit_cast(i32x4, a.v),
                                                     acc, 0, 0, 0);
    } else {
        const f32x4 bv = __builtin_bit_cast(f32x4, b.v), av = __builtin_bit_cast(f32x4, a.v);
#pragma unroll
        for (int j = 0; j < 4; j++)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(bv[j], av[j], acc, 0, 0, 0);
        return acc;
    }
}

// One operand's share of a step, staged through registers: each thread moves
// CH chunks of 16 bytes from any element-aligned address.
template <typename T, bool OUTER, int ROWS, int THREADS> struct Stage {
    static constexpr int EPC = traits<T>::EPC;
    static constexpr int BK = STEP_BYTES / (int)sizeof(T);
    static constexpr int CHUNKS = ROWS * STEP_BYTES / 16;
    static constexpr int CH = (CHUNKS + THREADS - 1) / THREADS;
    u32x4 v[CH];

    // k0: first k of the step; kend: end of this workgroup's k range
    __device__ __forceinline__ void load(const T *base, int64_t ld, int r0, int rows, int k0, int kend)
    {
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int q = threadIdx.x + c * THREADS;
            if (CHUNKS % THREADS != 0 && q >= CHUNKS)
                break;
            int64_t at;
            int valid;
            if constexpr (!OUTER) {
                const int r = r0 + q / 8, k = k0 + (q % 8) * EPC;
                at = (int64_t)r * ld + k;
                valid = r < rows ? kend - k : 0;
            } else {
                constexpr int CPR = ROWS / EPC;
                const int k = k0 + q / CPR, r = r0 + (q % CPR) * EPC;
                at = (int64_t)k * ld + r;
                valid = k < kend ? rows - r : 0;
            }
            v[c] = load_chunk(base + at, valid);
        }
    }

    __device__ __forceinline__ void store(char *tile) const
    {
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int q = threadIdx.x + c * THREADS;
            if (CHUNKS % THREADS != 0 && q >= CHUNKS)
                break;
            int at;
            if constexpr (!OUTER) {
                const int r = q / 8;
                at = r * STEP_BYTES + (((q % 8) ^ (r & 7)) << 4);
            } else {
                constexpr int CPR = ROWS / EPC;
                const int k = q / CPR;
                at = k * (ROWS * (int)sizeof(T)) + (((q % CPR) ^ outer_swizzle<T, ROWS>(k)) << 4);
            }
            *reinterpret_cast<u32x4 *>(tile + at) = v[c];
        }
    }
};

// The same moved straight from memory into LDS (16 bytes a lane, no
// registers), for operands whose rows start on 16 bytes and end on a whole
// chunk.  The hardware places a wavefront's 64 chunks one after another, so
// the exchange of chunks within a row is made on the addresses read.  A chunk
// outside the operand gets an offset past the buffer's range, which reads 0.
constexpr uint32_t OUT_OF_RANGE = 0x80000000u;

template <typename T, bool OUTER, int ROWS, int THREADS, int STEP> struct Direct {
    static constexpr int EPC = traits<T>::EPC;
    static constexpr int BK = STEP / (int)sizeof(T);
    static constexpr int CHUNKS = ROWS * STEP / 16;
    static constexpr int CH = (CHUNKS + THREADS - 1) / THREADS;
    static constexpr int CPR = OUTER ? ROWS / EPC : STEP / 16;
    uint32_t off[CH]; // byte offset of each chunk from the tile's base
    const char *base;
    int64_t advance; // bytes from one step to the next

    __device__ __forceinline__ void init(const T *p, int64_t ld, int r0, int rows, int k0)
    {
        base = reinterpret_cast<const char *>(OUTER ? p + (int64_t)k0 * ld + r0 : p + (int64_t)r0 * ld + k0);
        advance = OUTER ? BK * ld * (int64_t)sizeof(T) : STEP;
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int q = threadIdx.x + c * THREADS;
            if constexpr (!OUTER) {
                const int r = q / CPR, ch = (q % CPR) ^ inner_swizzle<STEP>(r);
                off[c] = r0 + r < rows ? (uint32_t)(r * ld * (int64_t)sizeof(T)) + ch * 16 : OUT_OF_RANGE;
            } else {
                const int k = q / CPR, ch = (q % CPR) ^ outer_swizzle<T, ROWS>(k);
                off[c] = r0 + ch * EPC < rows ? (uint32_t)(k * ld * (int64_t)sizeof(T)) + ch * 16 : OUT_OF_RANGE;
            }
        }
    }

    // For an outer operand whose rows hold two matrices' columns in turns of `turn`:
    // the tile's rows get the first matrix's, then the second's.  r0: the first column.
    __device__ __forceinline__ void halves(int64_t ld, int r0, int turn)
    {
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int q = threadIdx.x + c * THREADS, k = q / CPR;
            const int at = ((q % CPR) ^ outer_swizzle<T, ROWS>(k)) * EPC, col = at % (ROWS / 2);
            off[c] = 2 * (r0 + col) < ld ? (uint32_t)((k * ld + col + col / turn * turn + at / (ROWS / 2) * turn) * (int64_t)sizeof(T))
                                         : OUT_OF_RANGE;
        }
    }

    // Starts the copies of one step; `left`: values of k from its first on.
    __device__ __forceinline__ void start(char *tile, int left)
    {
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base), 0, (int)OUT_OF_RANGE, 0x00020000);
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int first = (threadIdx.x / WAVE) * WAVE + c * THREADS;
            if (CHUNKS % THREADS != 0 && first >= CHUNKS)
                break;
            uint32_t o = off[c];
            if (left < BK) {
                const int q = threadIdx.x + c * THREADS;
                const int k = OUTER ? q / CPR : ((q % CPR) ^ inner_swizzle<STEP>(q / CPR)) * EPC;
                o = k < left ? o : OUT_OF_RANGE;
            }
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void *)(tile + first * 16), 16, o, 0, 0, 0);
        }
        base += advance;
    }

    // The same `shift` bytes from the base, which stays.
    __device__ __forceinline__ void start_at(char *tile, int64_t shift, int left) const
    {
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base + shift), 0, (int)OUT_OF_RANGE, 0x00020000);
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int first = (threadIdx.x / WAVE) * WAVE + c * THREADS;
            if (CHUNKS % THREADS != 0 && first >= CHUNKS)
                break;
            uint32_t o = off[c];
            if (left < BK) {
                const int q = threadIdx.x + c * THREADS;
                const int k = OUTER ? q / CPR : ((q % CPR) ^ inner_swizzle<STEP>(q / CPR)) * EPC;
                o = k < left ? o : OUT_OF_RANGE;
            }
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void *)(tile + first * 16), 16, o, 0, 0, 0);
        }
    }

    // The same of a step that is all there, where chunks c and c + 2 of a thread lie
    // `apart` bytes from each other; two offsets stay in registers.
    __device__ __forceinline__ void start_apart(char *tile, uint32_t apart) const
    {
        static_assert(CHUNKS % THREADS == 0, "every thread copies as much");
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base), 0, (int)OUT_OF_RANGE, 0x00020000);
#pragma unroll
        for (int c = 0; c < CH; c++)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void *)(tile + ((threadIdx.x / WAVE) * WAVE + c * THREADS) * 16), 16,
                off[c & 1] + (c >> 1) * apart, 0, 0, 0);
    }
};

// s_waitcnt with at most n copies outstanding, and the LDS accesses done or as
// they are.
constexpr int wait_copies(int n, bool lds) { return 0x0070 | (n & 15) | (n >> 4) << 14 | (lds ? 0 : 0x0f00); }

// Waits for all but the last COPIES of this wavefront's copies into LDS, with
// LDS also for its reads, then for the other wavefronts; no access to memory
// moves across.
template <int COPIES, bool LDS> __device__ __forceinline__ void copies_done()
{
    static_assert(COPIES < 64, "the counter's bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_copies(COPIES, LDS));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <typename T, int BM, int BN, int WM, int WN, bool AO, bool BO> struct Tile {
    static constexpr int THREADS = WM * WN * WAVE;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    typedef typename traits<T>::sums Sums;
    Sums acc[FM][FN];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < FN; j++)
                acc[i][j] = Sums{0, 0, 0, 0};
    }

    // acc += the products of one step's tiles
    __device__ __forceinline__ void step(const char *ta, const char *tb, int wm, int wn, int lane)
    {
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
            Frag fa[FM], fb[FN];
#pragma unroll
            for (int i = 0; i < FM; i++)
                fa[i] = read_frag<T, AO, BM, STEP_BYTES>(ta, wm + i * 16, kk, lane);
#pragma unroll
            for (int j = 0; j < FN; j++)
                fb[j] = read_frag<T, BO, BN, STEP_BYTES>(tb, wn + j * 16, kk, lane);
#pragma unroll
            for (int i = 0; i < FM; i++)
#pragma unroll
                for (int j = 0; j < FN; j++)
                    acc[i][j] = mma<T>(fb[j], fa[i], acc[i][j]);
        }
    }

    // Steps of 128 bytes of k through two buffers.  copy(l, s) starts the copies
    // of step s into l: A's tile, then B's.
    template <typename COPY>
    __device__ __forceinline__ void run(char *l0, char *l1, int steps, int wm, int wn, int lane, COPY copy)
    {
        constexpr int AB = BM * STEP_BYTES;
        if (steps > 0)
            copy(l0, 0);
        int s = 0;
        for (; s + 1 < steps; s += 2) {
            copies_done<0, true>();
            copy(l1, s + 1);
            step(l0, l0 + AB, wm, wn, lane);
            copies_done<0, true>();
            if (s + 2 < steps)
                copy(l0, s + 2);
            step(l1, l1 + AB, wm, wn, lane);
        }
        copies_done<0, true>();
        if (s < steps)
            step(l0, l0 + AB, wm, wn, lane);
        __syncthreads();
    }

    // The same through four buffers, three steps on their way.  COPIES: the least
    // that a wavefront copies in a step.
    template <int COPIES, typename COPY>
    __device__ __forceinline__ void run(char *l0, char *l1, char *l2, char *l3, int steps, int wm, int wn, int lane, COPY copy)
    {
        constexpr int AB = BM * STEP_BYTES;
        // step t from `cur`; `free` held step t - 1 and takes step t + 3
        const auto turn = [&](const char *cur, char *free, int t) {
            if (t + 2 < steps)
                copies_done<2 * COPIES, true>();
            else if (t + 1 < steps)
                copies_done<COPIES, true>();
            else
                copies_done<0, true>();
            if (t + 3 < steps)
                copy(free, t + 3);
            step(cur, cur + AB, wm, wn, lane);
        };
        if (steps > 0)
            copy(l0, 0);
        if (steps > 1)
            copy(l1, 1);
        if (steps > 2)
            copy(l2, 2);
        for (int t = 0; t < steps; t += 4) {
            turn(l0, l3, t);
            if (t + 1 < steps)
                turn(l1, l0, t + 1);
            if (t + 2 < steps)
                turn(l2, l1, t + 2);
            if (t + 3 < steps)
                turn(l3, l2, t + 3);
        }
        __syncthreads();
    }
};

// Steps of 64 bytes of k through four buffers: while the matrix cores work on
// step t from registers, the fragments of step t + 1 are read from LDS (A's
// replace theirs row by row, B's have a second set), and the copies of steps
// t + 2 and t + 3 are on their way.  One barrier a step.  (Five buffers, one
// more step ahead, were no faster: 8192x14336x4096 827 us against 813; nor four
// wavefronts of 128x128 each: 1333.)
constexpr int PIPE_STEP = 64;

// LDS reads that read_frag makes.
template <typename T, bool OUTER> constexpr int reads_per_frag() { return !OUTER ? 1 : sizeof(T) == 2 ? 2 : 4; }

template <typename T, int BM, int BN, int WM, int WN, bool AO, bool BO> struct Pipe {
    static constexpr int THREADS = WM * WN * WAVE;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    static constexpr int AB = BM * PIPE_STEP, BB = BN * PIPE_STEP;
    static constexpr int COPIES = (AB + BB) / 16 / THREADS; // per thread and step
    static_assert(AB % (16 * THREADS) == 0 && BB % (16 * THREADS) == 0, "every thread copies the same number of chunks");
    static_assert(FN <= FM, "B's fragments are read along A's");
    typedef typename traits<T>::sums Sums;
    Sums acc[FM][FN];

    // copy(l) starts the copies of the next step into l: A's tile, then B's.
    // It is called for up to three steps past the end.
    template <typename COPY>
    __device__ __forceinline__ void run(char *l0, char *l1, char *l2, char *l3, int steps, COPY copy)
    {
        const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
        const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < FN; j++)
                acc[i][j] = Sums{0, 0, 0, 0};
        Frag fa[FM], fb[2][FN];
        constexpr int RA = reads_per_frag<T, AO>(), RB = reads_per_frag<T, BO>();
        // step t: `next` holds step t + 1, `free` step t - 1.  A's fragments are
        // replaced as soon as their row of products is issued, so only B's take
        // two sets of registers.
        const auto step = [&](char *next, char *free, int s) {
            // step t + 1 is here, t + 2 may be under way.  The reads of `free` were
            // used up by the last step's products, which no scheduling moves here.
            copies_done<COPIES, false>();
            __builtin_amdgcn_sched_barrier(0);
            copy(free);
#pragma unroll
            for (int i = 0; i < FM; i++) {
#pragma unroll
                for (int j = 0; j < FN; j++)
                    acc[i][j] = mma<T>(fb[s][j], fa[i], acc[i][j]);
                fa[i] = read_frag<T, AO, BM, PIPE_STEP>(next, wm + i * 16, 0, lane);
                if (i < FN)
                    fb[s ^ 1][i] = read_frag<T, BO, BN, PIPE_STEP>(next + AB, wn + i * 16, 0, lane);
            }
            constexpr int ROW = FN * (sizeof(T) == 4 ? 4 : 1);
#pragma unroll
            for (int i = 0; i < FN; i++) {
                __builtin_amdgcn_sched_group_barrier(0x008, ROW, 0);     // matrix instructions
                __builtin_amdgcn_sched_group_barrier(0x100, RA + RB, 0); // reads of LDS
                __builtin_amdgcn_sched_group_barrier(0x020, (COPIES + FN - 1) / FN, 0); // copies
            }
#pragma unroll
            for (int i = FN; i < FM; i++) {
                __builtin_amdgcn_sched_group_barrier(0x008, ROW, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, RA, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        copy(l0);
        copy(l1);
        copy(l2);
        copies_done<2 * COPIES, false>();
#pragma unroll
        for (int i = 0; i < FM; i++)
            fa[i] = read_frag<T, AO, BM, PIPE_STEP>(l0, wm + i * 16, 0, lane);
#pragma unroll
        for (int j = 0; j < FN; j++)
            fb[0][j] = read_frag<T, BO, BN, PIPE_STEP>(l0 + AB, wn + j * 16, 0, lane);
        int t = 0;
        for (; t + 4 <= steps; t += 4) {
            step(l1, l3, 0);
            step(l2, l0, 1);
            step(l3, l1, 0);
            step(l0, l2, 1);
        }
        if (t < steps)
            step(l1, l3, 0);
        if (t + 1 < steps)
            step(l2, l0, 1);
        if (t + 2 < steps)
            step(l3, l1, 0);
        copies_done<0, true>(); // also those past the end
    }
};

// Which tile a workgroup takes.  Consecutive workgroups go to the 8 XCDs in
// turn; each XCD gets a contiguous run of tiles, walked in bands of GROUP tile
// rows, so the operand rows that it reads again stay in its own L2.
constexpr int XCDS = 8, GROUP = 8;

__device__ __forceinline__ void tile_of(unsigned id, unsigned tiles_m, unsigned tiles_n, unsigned &tm, unsigned &tn)
{
    const unsigned total = tiles_m * tiles_n, per = total / XCDS, rest = total % XCDS;
    const unsigned x = id % XCDS, at = id / XCDS;
    id = x * per + (x < rest ? x : rest) + at;
    const unsigned band = GROUP * tiles_n, first = id / band * GROUP;
    const unsigned high = tiles_m - first < GROUP ? tiles_m - first : GROUP;
    tm = first + id % band % high;
    tn = id % band / high;
}

// The finished tile goes through LDS, 16 rows of each row of wavefronts at a
// time, so that whole rows are read and written from consecutive lanes.  Two
// buffers of BYTES take turns; where one does not hold that many rows, the
// columns go in parts.
constexpr int EPI_W = 8;

// Where four columns from n of row r lie in such a buffer: the rows that one
// fragment holds are spread over the banks.
template <int COLS> __device__ __forceinline__ int write_tile_at(int r, int n)
{
    return r * COLS + (((n >> 2) ^ (r & 15 & (COLS / 4 - 1))) << 2);
}

template <typename T, int BM, int BN, int WM, int WN, int BYTES, typename Sums>
__device__ __forceinline__ void write_tile(const GemmArgs &p, int m0, int n0, const Sums (&acc)[BM / WM / 16][BN / WN / 16],
                                           char *b0, char *b1, float *part)
{
    constexpr bool INT = __is_same(Sums, i32x4);
    constexpr int THREADS = WM * WN * WAVE, FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr int W = EPI_W, ROWS = WM * 16, PARTS = (ROWS * BN * 4 + BYTES - 1) / BYTES, COLS = BN / PARTS;
    constexpr int PER = (ROWS * COLS / W + THREADS - 1) / THREADS; // chunks a thread writes in a pass
    static_assert(WN % PARTS == 0, "a part is whole wavefronts");
    static_assert(THREADS % (COLS / W) == 0, "a thread keeps its columns");
    const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE, wn = (wave % WN) * (BN / WN);
    const int c = threadIdx.x % (COLS / W) * W, r0 = threadIdx.x / (COLS / W);
    const auto row = [&](int q, int e) { // of the thread's e-th chunk in pass q
        const int r = r0 + e * (THREADS / (COLS / W));
        return r < ROWS ? m0 + r / 16 * (BM / WM) + q / PARTS * 16 + r % 16 : p.M;
    };
    Raw<T, W> bias[PARTS], res[2][PER];
    Raw<float, W> cs[INT ? PARTS : 1];
    if (!part) {
#pragma unroll
        for (int h = 0; h < PARTS; h++) {
            fetch_bias(p, n0 + h * COLS + c, bias[h]);
            if constexpr (INT)
                cs[h].fetch(p.col_scale + n0 + h * COLS + c, p.N - (n0 + h * COLS + c));
        }
#pragma unroll
        for (int e = 0; e < PER; e++)
            fetch_residual(p, row(0, e), n0 + c, res[0][e]);
    }
#pragma unroll
    for (int q = 0; q < FM * PARTS; q++) {
        const int i = q / PARTS, h = q % PARTS, c0 = h * COLS;
        float *o = reinterpret_cast<float *>(q & 1 ? b1 : b0);
        if (PARTS == 1 || (wn >= c0 && wn < c0 + COLS)) {
#pragma unroll
            for (int j = 0; j < FN; j++)
                *reinterpret_cast<Sums *>(
                    o + write_tile_at<COLS>((wave / WN) * 16 + (lane & 15), wn - c0 + j * 16 + (lane >> 4) * 4)) = acc[i][j];
        }
        // the next pass's residual is on its way while this pass is written
        if (!part && q + 1 < FM * PARTS) {
#pragma unroll
            for (int e = 0; e < PER; e++)
                fetch_residual(p, row(q + 1, e), n0 + (q + 1) % PARTS * COLS + c, res[(q + 1) & 1][e]);
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < PER; e++) {
            const int n = n0 + c0 + c, m = row(q, e);
            if (m < p.M && n < p.N) {
                float v[W];
                int32_t w[W];
                void *raw = INT ? (void *)w : (void *)v;
#pragma unroll
                for (int g = 0; g < W; g += 4)
                    __builtin_memcpy((char *)raw + 4 * g, o + write_tile_at<COLS>(r0 + e * (THREADS / (COLS / W)), c + g), 16);
                if (part) {
                    const int64_t at = ((int64_t)blockIdx.y * p.M + m) * p.N + n;
                    if constexpr (INT)
                        store_n<int32_t, W>(reinterpret_cast<int32_t *>(part) + at, p.N - n, w);
                    else
                        store_n<float, W>(part + at, p.N - n, v);
                } else {
                    if constexpr (INT)
                        scaled_sums<W>(w, p.row_scale[m], cs[h].e, v);
                    epilogue<T, W>(p, m, n, v, bias[h], res[q & 1][e]);
                }
            }
        }
    }
}

} // namespace
} // namespace fa
