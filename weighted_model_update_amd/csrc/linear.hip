// The linear layer of an adapter or a head: products with a fused epilogue
// (bias, activation, residual) and the two products of its gradient.
//
// All three are C(m,n) = sum_k A(m,k) B(n,k) with operands stored with the
// summed index fastest ("inner") or slowest ("outer"):
//     y  = x w^T     A = x  inner, B = w inner
//     dx = dz w      A = dz inner, B = w outer
//     dw = dz^T x    A = dz outer, B = x outer
// Two tiled kernels serve them: pipe_kernel for large products, gemm_kernel for
// small and thin ones.  A workgroup owns a BM x BN tile of C and walks over k.
// Products run on the matrix cores with fp32 sums: bf16 as 16x16x32, fp32 as
// 16x16x4.
#include "learn_internal.h"

#include <algorithm>

namespace fa {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int STEP_BYTES = 128; // k per step, as bytes of one row
constexpr int WAVE = 64;

template <typename T> struct traits;
template <> struct traits<__bf16> { static constexpr int EPC = 8; };
template <> struct traits<float> { static constexpr int EPC = 4; };

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
            e[i] = i < valid ? p[i] : (T)0.f;
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

template <typename T, int W> __device__ __forceinline__ void store_n(T *p, int valid, const float *v)
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
        } else {
#pragma unroll
            for (int i = 0; i < W; i++)
                e[i] = i < valid ? p[i] : (T)0.f;
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
    u32x4 v; // bf16: 8 values of k;  fp32: 4 values of k
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
template <typename T> __device__ __forceinline__ f32x4 mma(const Frag &b, const Frag &a, f32x4 acc)
{
    if constexpr (sizeof(T) == 2) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b.v),
                                                       __builtin_bit_cast(bf16x8, a.v), acc, 0, 0, 0);
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
};

template <typename T, int BM, int BN, int WM, int WN, bool AO, bool BO> struct Tile {
    static constexpr int THREADS = WM * WN * WAVE;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    f32x4 acc[FM][FN];

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
};

// s_waitcnt with at most n copies outstanding, and the LDS accesses done or as
// they are.
constexpr int wait_copies(int n, bool lds) { return 0x0070 | n | (lds ? 0 : 0x0f00); }

// Waits for all but the last COPIES of this wavefront's copies into LDS, with
// LDS also for its reads, then for the other wavefronts; no access to memory
// moves across.
template <int COPIES, bool LDS> __device__ __forceinline__ void copies_done()
{
    static_assert(COPIES < 16, "the counter's low bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_copies(COPIES, LDS));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

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

template <typename T, int BM, int BN, int WM, int WN, int BYTES>
__device__ __forceinline__ void write_tile(const GemmArgs &p, int m0, int n0, const f32x4 (&acc)[BM / WM / 16][BN / WN / 16],
                                           char *b0, char *b1, float *part)
{
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
    if (!part) {
#pragma unroll
        for (int h = 0; h < PARTS; h++)
            fetch_bias(p, n0 + h * COLS + c, bias[h]);
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
                *reinterpret_cast<f32x4 *>(
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
#pragma unroll
                for (int g = 0; g < W; g += 4)
                    __builtin_memcpy(v + g, o + write_tile_at<COLS>(r0 + e * (THREADS / (COLS / W)), c + g), 16);
                if (part)
                    store_n<float, W>(part + ((int64_t)blockIdx.y * p.M + m) * p.N + n, p.N - n, v);
                else
                    epilogue<T, W>(p, m, n, v, bias[h], res[q & 1][e]);
            }
        }
    }
}

// Workgroup (tile, split): the sums over k in [split * kper, + kper).  With
// more than one split they go to `part` [split][M][N], else to the epilogue.
// Two buffers of 128 bytes of k.  Thin products are bound by memory, and the
// splits are what fills the card: one row through 14336 x 4096 bf16 weights in
// 18 us and the join's 4 (117 MB, 4.7 TB/s over the whole call), 8192 x 4096 to
// 16 columns in 13 and 4; as 128 x 128 tiles, unsplit, they took 72 and 54.  fp32
// is bound by its matrix rate: 777 x 2048 x 2048 with GELU, residual and saved
// pre-activation in 78 us (84 TFLOP/s).
template <typename T, int BM, int BN, int WM, int WN, bool AO, bool BO, bool DIRECT>
__global__ __launch_bounds__(WM *WN *WAVE) void gemm_kernel(GemmArgs p, int tiles_m, int tiles_n, int kper, float *part)
{
    constexpr int THREADS = WM * WN * WAVE;
    constexpr int BK = STEP_BYTES / (int)sizeof(T);
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr int AB = BM * STEP_BYTES, BB = BN * STEP_BYTES;
    // two buffers as objects of their own: the compiler then knows that the
    // copies into one do not touch what is read from the other
    __shared__ __attribute__((aligned(1024))) char l0[AB + BB];
    __shared__ __attribute__((aligned(1024))) char l1[AB + BB];

    unsigned tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int m0 = (int)tm * BM, n0 = (int)tn * BN;
    const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
    const T *a = static_cast<const T *>(p.a), *b = static_cast<const T *>(p.b);
    const int k0 = blockIdx.y * kper, kend = p.K - k0 < kper ? p.K : k0 + kper;
    const int steps = (kend - k0 + BK - 1) / BK;
    Tile<T, BM, BN, WM, WN, AO, BO> t;
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++)
            t.acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if constexpr (DIRECT) {
        Direct<T, AO, BM, THREADS, STEP_BYTES> da;
        Direct<T, BO, BN, THREADS, STEP_BYTES> db;
        da.init(a, p.lda, m0, p.M, k0);
        db.init(b, p.ldb, n0, p.N, k0);
        if (steps > 0) {
            da.start(l0, kend - k0);
            db.start(l0 + AB, kend - k0);
        }
        int s = 0;
        for (; s + 1 < steps; s += 2) {
            copies_done<0, true>();
            da.start(l1, kend - k0 - (s + 1) * BK);
            db.start(l1 + AB, kend - k0 - (s + 1) * BK);
            t.step(l0, l0 + AB, wm, wn, lane);
            copies_done<0, true>();
            if (s + 2 < steps) {
                da.start(l0, kend - k0 - (s + 2) * BK);
                db.start(l0 + AB, kend - k0 - (s + 2) * BK);
            }
            t.step(l1, l1 + AB, wm, wn, lane);
        }
        copies_done<0, true>();
        if (s < steps)
            t.step(l0, l0 + AB, wm, wn, lane);
        __syncthreads();
    } else {
        Stage<T, AO, BM, THREADS> sa;
        Stage<T, BO, BN, THREADS> sb;
        if (steps > 0) {
            sa.load(a, p.lda, m0, p.M, k0, kend);
            sb.load(b, p.ldb, n0, p.N, k0, kend);
            sa.store(l0);
            sb.store(l0 + AB);
        }
        __syncthreads();
        for (int s = 0; s < steps; s++) {
            char *cur = s & 1 ? l1 : l0, *next = s & 1 ? l0 : l1;
            if (s + 1 < steps) {
                sa.load(a, p.lda, m0, p.M, k0 + (s + 1) * BK, kend);
                sb.load(b, p.ldb, n0, p.N, k0 + (s + 1) * BK, kend);
            }
            t.step(cur, cur + AB, wm, wn, lane);
            if (s + 1 < steps) {
                sa.store(next);
                sb.store(next + AB);
            }
            __syncthreads();
        }
    }
    write_tile<T, BM, BN, WM, WN, AB + BB>(p, m0, n0, t.acc, l0, l1, part);
}

// The kernel of large products, bound by the matrix cores (1183 TFLOP/s at
// 8192x14336x4096 bf16, 1290 at 8192^3; the cores are busy 53% of the cycles at
// the 1.66 GHz that the card holds under this load).  Steps of 64 bytes of k,
// four buffers: while the matrix cores work on step t from registers, the
// fragments of step t + 1 are read from LDS (A's replace theirs row by row, B's
// have a second set), and the copies of steps t + 2 and t + 3 are on their way.
// One barrier a step.  (Five buffers, one more step ahead,
// were no faster: 8192x14336x4096 827 us against 813; nor four wavefronts of
// 128x128 each: 1333.)
constexpr int PIPE_STEP = 64;

// LDS reads that read_frag makes.
template <typename T, bool OUTER> constexpr int reads_per_frag() { return !OUTER ? 1 : sizeof(T) == 2 ? 2 : 4; }

template <typename T, int BM, int BN, int WM, int WN, bool AO, bool BO>
__global__ __launch_bounds__(WM *WN *WAVE) void pipe_kernel(GemmArgs p, int tiles_m, int tiles_n)
{
    constexpr int THREADS = WM * WN * WAVE;
    constexpr int BK = PIPE_STEP / (int)sizeof(T);
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr int AB = BM * PIPE_STEP, BB = BN * PIPE_STEP;
    constexpr int COPIES = (AB + BB) / 16 / THREADS; // per thread and step
    __shared__ __attribute__((aligned(1024))) char l0[AB + BB];
    __shared__ __attribute__((aligned(1024))) char l1[AB + BB];
    __shared__ __attribute__((aligned(1024))) char l2[AB + BB];
    __shared__ __attribute__((aligned(1024))) char l3[AB + BB];
    static_assert(AB % (16 * THREADS) == 0 && BB % (16 * THREADS) == 0, "every thread copies the same number of chunks");

    unsigned tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int m0 = (int)tm * BM, n0 = (int)tn * BN;
    const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
    const int steps = (p.K + BK - 1) / BK;
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    Direct<T, AO, BM, THREADS, PIPE_STEP> da;
    Direct<T, BO, BN, THREADS, PIPE_STEP> db;
    da.init(static_cast<const T *>(p.a), p.lda, m0, p.M, 0);
    db.init(static_cast<const T *>(p.b), p.ldb, n0, p.N, 0);
    int left = p.K; // of the next step to copy; steps past the end copy zeros
    const auto copy = [&](char *l) {
        da.start(l, left);
        db.start(l + AB, left);
        left -= BK;
    };
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
        constexpr int ROW = FN * (sizeof(T) == 2 ? 1 : 4);
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
    static_assert(FN <= FM, "B's fragments are read along A's");
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
    write_tile<T, BM, BN, WM, WN, AB + BB>(p, m0, n0, acc, l0, l1, nullptr);
}

constexpr int FINISH_THREADS = 256, JOIN_W = 4;

// Joins four neighbouring sums of a product's splits in split order, the same
// bits on every call, and finishes them.
template <typename T> __device__ __forceinline__ void join_splits(const GemmArgs &p, const float *part, int splits, int64_t at)
{
    const int64_t groups = (p.N + JOIN_W - 1) / JOIN_W;
    if (at >= p.M * groups)
        return;
    const int64_t m = at / groups;
    const int n = (int)(at % groups) * JOIN_W;
    float s[JOIN_W] = {};
#pragma unroll 4
    for (int z = 0; z < splits; z++) {
        float v[JOIN_W];
        load_n<float, JOIN_W>(part + ((int64_t)z * p.M + m) * p.N + n, p.N - n, v);
#pragma unroll
        for (int i = 0; i < JOIN_W; i++)
            s[i] += v[i];
    }
    Raw<T, JOIN_W> bias, res;
    fetch_bias(p, n, bias);
    fetch_residual(p, m, n, res);
    epilogue<T, JOIN_W>(p, m, n, s, bias, res);
}

// CJ_COLS columns of db a workgroup: each of the CJ_GROUPS groups of threads
// adds every CJ_GROUPS-th partial, and the groups' sums are added in order.
constexpr int CJ_COLS = 32, CJ_GROUPS = FINISH_THREADS / CJ_COLS;

template <typename T> __device__ __forceinline__ void join_columns(const ActGradArgs &p, int64_t parts, int64_t block)
{
    __shared__ float sums[CJ_GROUPS][CJ_COLS];
    const int col = threadIdx.x % CJ_COLS, group = threadIdx.x / CJ_COLS;
    const int64_t n = block * CJ_COLS + col;
    float s = 0.f;
    if (n < p.N) {
#pragma unroll 8
        for (int64_t q = group; q < parts; q += CJ_GROUPS)
            s += p.part[q * p.N + n];
    }
    sums[group][col] = s;
    __syncthreads();
    if (group == 0 && n < p.N) {
#pragma unroll
        for (int w = 1; w < CJ_GROUPS; w++)
            s += sums[w][col];
        static_cast<T *>(p.db)[n] = (T)s;
    }
}

// What a call's kernels leave to be joined, in one launch: bound by the launch
// itself, 4.0 us for 6 splits of 8192 x 16, 4.9 for 256 partials of 8192
// columns.
template <typename T> __global__ __launch_bounds__(FINISH_THREADS) void finish_kernel(Finish f)
{
    const int64_t block = blockIdx.x;
    if (block < f.blocks[0])
        join_splits<T>(f.p[0], f.part[0], f.splits[0], block * FINISH_THREADS + threadIdx.x);
    else if (block < f.blocks[0] + f.blocks[1])
        join_splits<T>(f.p[1], f.part[1], f.splits[1], (block - f.blocks[0]) * FINISH_THREADS + threadIdx.x);
    else
        join_columns<T>(f.g, f.parts, block - f.blocks[0] - f.blocks[1]);
}

// Steps of `bytes` of k a split, and how many splits that makes.
struct Split {
    int kper, splits;
};

template <typename T> Split split_of(int K, int splits, int bytes)
{
    const int bk = bytes / (int)sizeof(T), steps = std::max(1, (K + bk - 1) / bk), per = (steps + splits - 1) / splits;
    return {per * bk, (steps + per - 1) / per};
}

// An operand copied with its rows on 16 bytes and zeros up to whole chunks;
// bound by memory, one read and one write of the operand.
constexpr int PACK_THREADS = 256;

template <typename T>
__global__ __launch_bounds__(PACK_THREADS) void pack_kernel(const T *src, int64_t ld, int64_t rows, int64_t cols, T *dst)
{
    constexpr int EPC = traits<T>::EPC;
    const int64_t per = (cols + EPC - 1) / EPC, step = (int64_t)gridDim.x * PACK_THREADS;
    for (int64_t at = (int64_t)blockIdx.x * PACK_THREADS + threadIdx.x; at < rows * per; at += step) {
        const int64_t r = at / per, c = at % per * EPC;
        const u32x4 v = load_chunk(src + r * ld + c, (int)(cols - c < EPC ? cols - c : EPC));
        *reinterpret_cast<u32x4 *>(dst + at * EPC) = v;
    }
}

template <typename T, int BM, int BN, int WM, int WN, bool DIRECT>
hipError_t run_tile(const GemmArgs &a, int layout, int splits, float *ws, Finish &f, hipStream_t s)
{
    const int64_t tm = ((int64_t)a.M + BM - 1) / BM, tn = ((int64_t)a.N + BN - 1) / BN;
    const Split k = split_of<T>(a.K, splits, STEP_BYTES);
    float *part = k.splits > 1 ? ws : nullptr;
    const dim3 grid((unsigned)(tm * tn), (unsigned)k.splits), block(WM * WN * WAVE);
    if (layout == 0)
        gemm_kernel<T, BM, BN, WM, WN, false, false, DIRECT><<<grid, block, 0, s>>>(a, (int)tm, (int)tn, k.kper, part);
    else if (layout == GEMM_B_OUTER)
        gemm_kernel<T, BM, BN, WM, WN, false, true, DIRECT><<<grid, block, 0, s>>>(a, (int)tm, (int)tn, k.kper, part);
    else
        gemm_kernel<T, BM, BN, WM, WN, true, true, DIRECT><<<grid, block, 0, s>>>(a, (int)tm, (int)tn, k.kper, part);
    if (k.splits > 1) {
        const int j = f.blocks[0] > 0;
        f.p[j] = a;
        f.part[j] = part;
        f.splits[j] = k.splits;
        f.blocks[j] = ((int64_t)a.M * ((a.N + JOIN_W - 1) / JOIN_W) + FINISH_THREADS - 1) / FINISH_THREADS;
    }
    return hipGetLastError();
}

template <typename T, int BM, int BN, int WM, int WN> hipError_t run_pipe(const GemmArgs &a, int layout, hipStream_t s)
{
    const int64_t tm = ((int64_t)a.M + BM - 1) / BM, tn = ((int64_t)a.N + BN - 1) / BN;
    const dim3 grid((unsigned)(tm * tn)), block(WM * WN * WAVE);
    if (layout == 0)
        pipe_kernel<T, BM, BN, WM, WN, false, false><<<grid, block, 0, s>>>(a, (int)tm, (int)tn);
    else if (layout == GEMM_B_OUTER)
        pipe_kernel<T, BM, BN, WM, WN, false, true><<<grid, block, 0, s>>>(a, (int)tm, (int)tn);
    else
        pipe_kernel<T, BM, BN, WM, WN, true, true><<<grid, block, 0, s>>>(a, (int)tm, (int)tn);
    return hipGetLastError();
}

// ------------------------------------------------------------ dz and db
// Eight columns a thread; the threads of a workgroup stand `across` side by side
// in a row, a power of two up to a wavefront, and in AG_THREADS / across groups
// below one another, which take the rows in turn, AG_U on their way at a time.
// A column's partial sum is added in fp32 over a group's rows in order, then
// over the groups, and the partials in a fixed order, so db is the same bits on
// every call.  Bound by memory: 4096 x
// 8192 bf16 with GELU (dy and the pre-activation read, dz written: 201 MB) in
// 44 us, 4.5 TB/s; small ones by the latency of a thread's own elements, so
// rows are spread over idle threads: GELU of 1126 x 112 16.2 -> 5.4 us, of
// 1594 x 2440 21.9 -> 12.2 (against 16 rows a thread, 2048 columns a workgroup).
constexpr int AG_THREADS = 256, AG_W = 8, AG_U = 4;

template <typename T> __global__ __launch_bounds__(AG_THREADS) void act_grad_kernel(ActGradArgs p, int64_t rows_per, int across)
{
    __shared__ float sums[AG_THREADS][AG_W + 1];
    const int col = threadIdx.x & (across - 1), group = threadIdx.x / across, groups = AG_THREADS / across;
    const int64_t n = ((int64_t)blockIdx.x * across + col) * AG_W;
    const int valid = (int)(p.N - n < AG_W ? p.N - n : AG_W);
    const int64_t r0 = (int64_t)blockIdx.y * rows_per, r1 = r0 + rows_per < p.M ? r0 + rows_per : p.M;
    float sum[AG_W] = {};
    for (int64_t m0 = r0 + group; m0 < r1 && n < p.N; m0 += groups * AG_U) {
        float d[AG_U][AG_W], z[AG_U][AG_W];
#pragma unroll
        for (int u = 0; u < AG_U; u++) { // rows past the end read nothing
            const int64_t m = m0 + u * groups;
            const int v = m < r1 ? valid : 0;
            load_n<T, AG_W>(static_cast<const T *>(p.dy) + m * p.lddy + n, v, d[u]);
            if (p.act != FA_ACT_NONE)
                load_n<T, AG_W>(static_cast<const T *>(p.pre) + m * p.ldp + n, v, z[u]);
        }
#pragma unroll
        for (int u = 0; u < AG_U; u++) {
            const int64_t m = m0 + u * groups;
            if (m >= r1)
                break;
            apply_slope<sizeof(T) == 4, AG_W>(d[u], z[u], p.act);
            if (p.dz)
                store_n<T, AG_W>(static_cast<T *>(p.dz) + m * p.lddz + n, AG_W, d[u]);
#pragma unroll
            for (int i = 0; i < AG_W; i++)
                sum[i] += d[u][i];
        }
    }
    if (!p.db)
        return;
#pragma unroll
    for (int i = 0; i < AG_W; i++)
        sums[threadIdx.x][i] = sum[i];
    __syncthreads();
    for (int g = 1; g < groups && group == 0; g++)
#pragma unroll
        for (int i = 0; i < AG_W; i++)
            sum[i] += sums[g * across + col][i];
    if (group == 0 && n < p.N)
        store_n<float, AG_W>(p.part + (int64_t)blockIdx.y * p.N + n, valid, sum);
}

} // namespace

namespace {

// Whether a tile of an operand with this row pitch stays within the 31 bits of
// a buffer offset.
bool pitch_ok(int64_t bytes) { return bytes * 257 < (int64_t)OUT_OF_RANGE; }

// Whether an operand's rows start on 16 bytes and end on a whole chunk (or in
// zeros up to one), and its pitch suits the direct loads.
bool direct_ok(const void *p, int64_t ld, int64_t row, bool padded, size_t es)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld * (int64_t)es % 16 == 0 &&
           (padded || row * (int64_t)es % 16 == 0) && pitch_ok(ld * (int64_t)es);
}

// Tiles: PIPE_* by the pipelined kernel, the others by the two-buffer one.
enum { PIPE_256_256, PIPE_256_128, PIPE_128_256, PIPE_128_128, TILE_64, TILE_THIN_N, TILE_THIN_M };

struct Plan {
    int tile, splits;
    bool large; // enough products to repay aligned copies of odd operands
};

int64_t tiles(int64_t M, int64_t N, int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

// The time of a pipelined tile per k is steady, so tiles are compared by the
// rounds that they need on all CUs: one 256x256, 256x128 or 128x256 tile fits a
// CU at a time, two of 128x128.  Measured on 256 CUs, us of a round for bf16
// and K = 8192, by which operands are outer (none, B, both); the last column is
// a round of 128x128 with one tile a CU.  For example 8192x5000x4000: 256x256
// 331 us, 256x128 366, 128x256 351, 128x128 412; 4096x2048x8192: 173, 135, 144,
// 161; 2048x2048x4096: 87, 63, 57, 45.  fp32 is bound by the matrix cores at
// any tile (128x128 140 TFLOP/s, 256x128 142, 64x64 133).
int pipe_for(int64_t M, int64_t N, int layout, int cus)
{
    static const int us[3][5] = {{222, 140, 138, 155, 90}, {215, 130, 121, 140, 86}, {215, 123, 125, 130, 86}};
    const int *c = us[layout == 0 ? 0 : layout == GEMM_B_OUTER ? 1 : 2];
    const auto rounds = [&](int64_t t) { return (t + cus - 1) / cus; };
    const int64_t t128 = tiles(M, N, 128, 128), whole = t128 / (2 * cus), rest = t128 % (2 * cus);
    const int64_t costs[4] = {c[0] * rounds(tiles(M, N, 256, 256)), c[1] * rounds(tiles(M, N, 256, 128)),
                              c[2] * rounds(tiles(M, N, 128, 256)),
                              c[3] * whole + (rest > cus ? c[3] : rest > 0 ? c[4] : 0)};
    return (int)(std::min_element(costs, costs + 4) - costs);
}

// Small products: 64x64 tiles with k split.  The number of splits is the one of
// least estimated time: a step of 128 bytes of k takes a workgroup 0.5 us (bf16)
// while there are two a CU or fewer; in fp32, bound by the matrix cores, 0.75 us
// while there is one a CU, else 0.55 us a round; joining takes 3.5 us and the sums' way to memory and back at 3 TB/s.
// Measured, us for bf16 with K = 4096: 512x1024 unsplit 34, in 2 23, in 4 17, in
// 8 19; 256x1024 22, 16, 13, 15; 32x4096 34, 22, 14, 12; 1024x2048 with K = 512
// unsplit 7.5, in 2 20.  fp32: 512x1024x4096 in 1, 2, 3, 5 99, 57, 59, 53;
// 777x2048x2048 84, 82, 81, 84; 1500x1500x600 39, 44, 44, 47.  Against the pipelined kernel: 2048x2048x4096 64x64 49,
// 128x128 45.
int small_splits(int64_t M, int64_t N, int64_t steps, int64_t count, size_t es, int cus)
{
    int best = 1;
    double least = 0;
    for (int s = 1; s <= 64 && (s == 1 || (steps >= 2 * s && count * s <= 5 * cus)); s++) {
        const double wgs = (double)count * s;
        const int64_t rounds = (count * s + cus - 1) / cus;
        const double step = es == 2 ? 0.5 * std::max(1.0, wgs / (2 * cus)) : rounds == 1 ? 0.75 : 0.55 * (double)rounds;
        const double join = s == 1 ? 0 : 3.5 + s * (double)M * (double)N * 8 / 3e6;
        const double t = (double)((steps + s - 1) / s) * step + join;
        if (s == 1 || t < least) {
            best = s;
            least = t;
        }
    }
    return best;
}

// Thin ones stream one operand: about three workgroups to two CUs keep the
// memory busy and more only add sums to join: 8192x16x4096 in 4, 6, 8, 16
// splits of 64 tiles 16.0, 15.8, 16.0, 17.6 us; 1x14336x4096 of 112 tiles in 2,
// 4, 8 22.7, 20.7, 21.5; 16x4096x4096 of 32 tiles in 4, 8, 16 13.4, 10.8, 12.2.
constexpr int THIN_MIN_STEPS = 4, THIN_MAX_SPLITS = 16;

// M N K from which a product of 64x64 tiles repays the copies of odd operands.
// Staged and copied, us for y, dx, dw in bf16: 1001x1001x1001 14, 19, 25 and
// 20, 21, 22; 1125x4239x775 37, 57, 44 and 37, 41, 37; 4716x2938x341 38, 64,
// 126 and 38, 47, 61; 2047x4095x1023 dx 102 and 54.
constexpr double PACK_LEAST = 2e9;

Plan plan_of(int64_t M, int64_t N, int64_t K, size_t es, int layout, int cus)
{
    const int64_t steps = K * (int64_t)es / STEP_BYTES;
    const auto thin = [&](int64_t count) {
        const int64_t want = (3 * cus / 2 + count - 1) / count;
        return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(want, steps / THIN_MIN_STEPS), THIN_MAX_SPLITS));
    };
    if (N <= 16)
        return {TILE_THIN_N, thin(std::max<int64_t>(1, tiles(M, N, 128, 16))), false};
    if (M <= 16)
        return {TILE_THIN_M, thin(std::max<int64_t>(1, tiles(M, N, 16, 128))), false};
    if (es == 2 && tiles(M, N, 128, 128) >= cus)
        return {pipe_for(M, N, layout, cus), 1, true};
    if (es == 4 && tiles(M, N, 128, 128) >= 2 * cus)
        return {PIPE_128_128, 1, true};
    return {TILE_64, small_splits(M, N, steps, std::max<int64_t>(1, tiles(M, N, 64, 64)), es, cus),
            (double)M * (double)N * (double)K >= PACK_LEAST};
}

// Bytes of the copy of an operand of `rows` rows of `row` elements, 0 where
// the rows are whole chunks or the copy's would be too long for direct loads.
size_t pack_bytes(int64_t rows, int64_t row, size_t es)
{
    const int64_t bytes = (row * (int64_t)es + 15) / 16 * 16;
    return bytes == row * (int64_t)es || !pitch_ok(bytes) ? 0 : ((size_t)(rows * bytes) + 255) / 256 * 256;
}

template <typename T> hipError_t pack(const void *&p, int64_t &ld, int64_t rows, int64_t row, void *to, hipStream_t s)
{
    constexpr int EPC = traits<T>::EPC;
    const int64_t per = (row + EPC - 1) / EPC, chunks = rows * per;
    const unsigned grid = (unsigned)std::min<int64_t>((chunks + PACK_THREADS - 1) / PACK_THREADS, 1 << 22);
    pack_kernel<T><<<grid, PACK_THREADS, 0, s>>>(
        static_cast<const T *>(p), ld, rows, row, static_cast<T *>(to));
    p = to;
    ld = per * EPC;
    return hipGetLastError();
}

// Bytes of the partial sums, at the front of the workspace.
size_t part_bytes(const Plan &p, int64_t M, int64_t N)
{
    return p.splits > 1 ? ((size_t)p.splits * M * N * sizeof(float) + 255) / 256 * 256 : 0;
}

template <typename T> hipError_t gemm_of(GemmArgs a, int layout, float *ws, int cus, Finish &f, hipStream_t s)
{
    const Plan p = plan_of(a.M, a.N, a.K, sizeof(T), layout, cus);
    const int64_t row_a = layout & GEMM_A_OUTER ? a.M : a.K, row_b = layout & GEMM_B_OUTER ? a.N : a.K;
    const int64_t rows_a = layout & GEMM_A_OUTER ? a.K : a.M, rows_b = layout & GEMM_B_OUTER ? a.K : a.N;
    bool ok_a = direct_ok(a.a, a.lda, row_a, a.a_padded, sizeof(T)), ok_b = direct_ok(a.b, a.ldb, row_b, false, sizeof(T));
    if (p.large && !(ok_a && ok_b)) {
        // A large product repays the copies that the direct loads need:
        // 8192x5001x4001 bf16 552 us staged through registers, 461 copied
        // (dx 581 and 336, dw 907 and 420).  Operands whose rows are whole
        // chunks but start off 16 bytes have no room in the workspace, whose
        // size goes by M, N and K alone; they are staged (8192x5000x4000 one
        // element off: y, dx, dw 628, 480, 530 us, against 300, 270, 335).
        const size_t need_a = pack_bytes(rows_a, row_a, sizeof(T)), need_b = pack_bytes(rows_b, row_b, sizeof(T));
        if ((ok_a || need_a) && (ok_b || need_b)) {
            char *to = reinterpret_cast<char *>(ws) + part_bytes(p, a.M, a.N);
            hipError_t e = ok_a ? hipSuccess : pack<T>(a.a, a.lda, rows_a, row_a, to, s);
            if (e == hipSuccess && !ok_b)
                e = pack<T>(a.b, a.ldb, rows_b, row_b, to + need_a, s);
            if (e != hipSuccess)
                return e;
            ok_a = ok_b = true;
        }
    }
    const bool direct = ok_a && ok_b;
    if (p.tile <= PIPE_128_128) {
        if (!direct)
            return run_tile<T, 128, 128, 2, 2, false>(a, layout, 1, ws, f, s);
        if constexpr (sizeof(T) == 2) {
            if (p.tile == PIPE_256_256)
                return run_pipe<T, 256, 256, 2, 4>(a, layout, s);
            if (p.tile == PIPE_256_128)
                return run_pipe<T, 256, 128, 4, 2>(a, layout, s);
            if (p.tile == PIPE_128_256)
                return run_pipe<T, 128, 256, 2, 4>(a, layout, s);
        }
        return run_pipe<T, 128, 128, 2, 4>(a, layout, s);
    }
    if (p.tile == TILE_64)
        return direct ? run_tile<T, 64, 64, 2, 2, true>(a, layout, p.splits, ws, f, s)
                      : run_tile<T, 64, 64, 2, 2, false>(a, layout, p.splits, ws, f, s);
    if (p.tile == TILE_THIN_N)
        return direct ? run_tile<T, 128, 16, 4, 1, true>(a, layout, p.splits, ws, f, s)
                      : run_tile<T, 128, 16, 4, 1, false>(a, layout, p.splits, ws, f, s);
    return direct ? run_tile<T, 16, 128, 1, 4, true>(a, layout, p.splits, ws, f, s)
                  : run_tile<T, 16, 128, 1, 4, false>(a, layout, p.splits, ws, f, s);
}

} // namespace

size_t gemm_workspace_bytes(int dt, int64_t M, int64_t N, int64_t K, int layout, int cus)
{
    const size_t es = dt == FA_BF16 ? 2 : 4;
    const Plan p = plan_of(M, N, K, es, layout, cus);
    size_t bytes = part_bytes(p, M, N);
    if (p.large)
        bytes += (layout & GEMM_A_OUTER ? pack_bytes(K, M, es) : pack_bytes(M, K, es)) +
                 (layout & GEMM_B_OUTER ? pack_bytes(K, N, es) : pack_bytes(N, K, es));
    return bytes;
}

hipError_t launch_gemm(const GemmArgs &a, int dt, int layout, void *ws, int cus, Finish &f, hipStream_t s)
{
    if (a.M == 0 || a.N == 0)
        return hipSuccess;
    float *part = static_cast<float *>(ws);
    return dt == FA_BF16 ? gemm_of<__bf16>(a, layout, part, cus, f, s) : gemm_of<float>(a, layout, part, cus, f, s);
}

namespace {

// Threads side by side for N columns.
int act_grad_across(int64_t N)
{
    int c = 1;
    while (c < WAVE && (int64_t)c * AG_W < N)
        c *= 2;
    return c;
}

} // namespace

// Enough workgroups for the chip.  Up to 256 partials a group's rows may be as
// few as one; beyond, where the partials cost more to join, at least 16.
int64_t act_grad_partials(int64_t M, int64_t N, int cus)
{
    const int across = act_grad_across(N), groups = AG_THREADS / across;
    const int64_t wide = std::max<int64_t>(1, (N + (int64_t)across * AG_W - 1) / ((int64_t)across * AG_W));
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(4 * (int64_t)cus / wide, 1024));
    const auto of = [&](int64_t rows) { return (M + rows * groups - 1) / (rows * groups); };
    return std::max<int64_t>(1, std::min(want, std::max(std::min<int64_t>(of(1), 256), of(16))));
}

hipError_t launch_act_grad(const ActGradArgs &a, int dt, int cus, Finish &f, hipStream_t s)
{
    if (a.N == 0)
        return hipSuccess;
    const int across = act_grad_across(a.N);
    const int64_t want = act_grad_partials(a.M, a.N, cus);
    const int64_t rows_per = std::max<int64_t>(1, (a.M + want - 1) / want);
    const int64_t parts = std::max<int64_t>(1, (a.M + rows_per - 1) / rows_per);
    const int64_t columns = (int64_t)across * AG_W;
    const dim3 grid((unsigned)((a.N + columns - 1) / columns), (unsigned)parts);
    if (dt == FA_BF16)
        act_grad_kernel<__bf16><<<grid, AG_THREADS, 0, s>>>(a, rows_per, across);
    else
        act_grad_kernel<float><<<grid, AG_THREADS, 0, s>>>(a, rows_per, across);
    if (a.db) {
        f.g = a;
        f.parts = parts;
        f.columns = (a.N + CJ_COLS - 1) / CJ_COLS;
    }
    return hipGetLastError();
}

hipError_t launch_finish(const Finish &f, int dt, hipStream_t s)
{
    const int64_t blocks = f.blocks[0] + f.blocks[1] + f.columns;
    if (blocks == 0)
        return hipSuccess;
    if (dt == FA_BF16)
        finish_kernel<__bf16><<<(unsigned)blocks, FINISH_THREADS, 0, s>>>(f);
    else
        finish_kernel<float><<<(unsigned)blocks, FINISH_THREADS, 0, s>>>(f);
    return hipGetLastError();
}

} // namespace fa
