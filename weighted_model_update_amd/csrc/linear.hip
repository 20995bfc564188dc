// The linear layer of an adapter or a head: products with a fused epilogue
// (bias, activation, residual) and the two products of its gradient.
//
// All three are C(m,n) = sum_k A(m,k) B(n,k) with operands stored with the
// summed index fastest ("inner") or slowest ("outer"):
//     y  = x w^T     A = x  inner, B = w inner
//     dx = dz w      A = dz inner, B = w outer
//     dw = dz^T x    A = dz outer, B = x outer
// One tiled kernel serves them.  A workgroup owns a BM x BN tile of C and
// walks over k in steps of 128 bytes (64 bf16 or 32 fp32).  Products run on
// the matrix cores with fp32 sums: bf16 as 16x16x32, fp32 as 16x16x4.
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
// In IEEE arithmetic as written; GELU is the exact one, z Phi(z).
__device__ __forceinline__ float act_of(float z, int act)
{
    if (act == FA_ACT_RELU)
        return z > 0.f ? z : (z == z ? 0.f : z);
    if (act == FA_ACT_GELU)
        return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    if (act == FA_ACT_SILU)
        return z / (1.f + expf(-z));
    return z;
}

__device__ __forceinline__ float act_slope(float z, int act)
{
    if (act == FA_ACT_RELU)
        return z > 0.f ? 1.f : (z == z ? 0.f : z);
    if (act == FA_ACT_GELU)
        return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
    if (act == FA_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-z));
        return s * (1.f + z * (1.f - s));
    }
    return 1.f;
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

// Four consecutive values of a row, of which `valid` may be touched.  Rows
// are only element-aligned; the hardware takes such vector accesses.
template <typename T> __device__ __forceinline__ void load4(const T *p, int valid, float *v)
{
    if (valid >= 4) {
        T e[4];
        __builtin_memcpy(e, p, sizeof e);
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = (float)e[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = i < valid ? (float)p[i] : 0.f;
    }
}

template <typename T> __device__ __forceinline__ void store4(T *p, int valid, const float *v)
{
    if (valid >= 4) {
        T e[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            e[i] = (T)v[i]; // round to nearest even
        __builtin_memcpy(p, e, sizeof e);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (i < valid)
                p[i] = (T)v[i];
    }
}

// out(m, n..n+3) from the finished sums: z = alpha s + bias, then the
// activation, then the residual, all in fp32, each result rounded once.
template <typename T>
__device__ __forceinline__ void epilogue4(const GemmArgs &p, int64_t m, int n, const float *s)
{
    const int valid = p.N - n;
    float z[4], b[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.bias)
        load4(static_cast<const T *>(p.bias) + n, valid, b);
#pragma unroll
    for (int i = 0; i < 4; i++)
        z[i] = __builtin_fmaf(p.alpha, s[i], b[i]);
    if (p.pre)
        store4(static_cast<T *>(p.pre) + m * p.ldp + n, valid, z);
    if (p.act != FA_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            z[i] = act_of(z[i], p.act);
    }
    if (p.res) {
        load4(static_cast<const T *>(p.res) + m * p.ldr + n, valid, b);
#pragma unroll
        for (int i = 0; i < 4; i++)
            z[i] += b[i];
    }
    store4(static_cast<T *>(p.out) + m * p.ldo + n, valid, z);
}

// ------------------------------------------------------------ LDS tiles
// An inner operand's tile holds `rows` rows of 128 bytes; its 16-byte chunk c
// of row r lies at chunk c ^ (r & 7), so the 16 rows that a fragment read
// touches spread over all banks.  An outer operand's tile holds one row of
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

struct Frag {
    u32x4 v; // bf16: 8 values of k;  fp32: 4 values of k
};

// Fragment of 16 rows (or columns) starting at r0, k half kk (0, 1) of the
// step: lane l holds row l % 16 and the 16 bytes of k of group l / 16.
template <typename T, bool OUTER, int ROWS>
__device__ __forceinline__ Frag read_frag(const char *tile, int r0, int kk, int lane)
{
    const int i = lane & 15, g = lane >> 4;
    Frag f;
    if constexpr (!OUTER) {
        const int r = r0 + i, c = g + 4 * kk;
        f.v = *reinterpret_cast<const u32x4 *>(tile + r * STEP_BYTES + ((c ^ (r & 7)) << 4));
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
            const char *at = tile + k * (ROWS * 2) + (c << 4) + ((col & 4) << 1);
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
            f.v[j] = *reinterpret_cast<const uint32_t *>(tile + k * (ROWS * 4) + (c << 4) + ((col & 3) << 2));
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

template <typename T, int BM, int BN, int WM, int WN, bool AO, bool BO>
__global__ __launch_bounds__(WM *WN *WAVE) void gemm_kernel(GemmArgs p, int tiles_n)
{
    constexpr int THREADS = WM * WN * WAVE;
    constexpr int BK = STEP_BYTES / (int)sizeof(T);
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    __shared__ __attribute__((aligned(16))) char lds[2][(BM + BN) * STEP_BYTES];

    const int m0 = (int)(blockIdx.x / tiles_n) * BM, n0 = (int)(blockIdx.x % tiles_n) * BN;
    const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
    const T *a = static_cast<const T *>(p.a), *b = static_cast<const T *>(p.b);

    f32x4 acc[FM][FN] = {};
    Stage<T, AO, BM, THREADS> sa;
    Stage<T, BO, BN, THREADS> sb;
    const int steps = (p.K + BK - 1) / BK;
    if (steps > 0) {
        sa.load(a, p.lda, m0, p.M, 0, p.K);
        sb.load(b, p.ldb, n0, p.N, 0, p.K);
        sa.store(lds[0]);
        sb.store(lds[0] + BM * STEP_BYTES);
    }
    __syncthreads();
    for (int t = 0; t < steps; t++) {
        const char *ta = lds[t & 1], *tb = ta + BM * STEP_BYTES;
        const bool more = t + 1 < steps;
        if (more) {
            sa.load(a, p.lda, m0, p.M, (t + 1) * BK, p.K);
            sb.load(b, p.ldb, n0, p.N, (t + 1) * BK, p.K);
        }
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
            Frag fa[FM], fb[FN];
#pragma unroll
            for (int i = 0; i < FM; i++)
                fa[i] = read_frag<T, AO, BM>(ta, wm + i * 16, kk, lane);
#pragma unroll
            for (int j = 0; j < FN; j++)
                fb[j] = read_frag<T, BO, BN>(tb, wn + j * 16, kk, lane);
#pragma unroll
            for (int i = 0; i < FM; i++)
#pragma unroll
                for (int j = 0; j < FN; j++)
                    acc[i][j] = mma<T>(fb[j], fa[i], acc[i][j]);
        }
        if (more) {
            sa.store(lds[(t + 1) & 1]);
            sb.store(lds[(t + 1) & 1] + BM * STEP_BYTES);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < FM; i++) {
        const int m = m0 + wm + i * 16 + (lane & 15);
        if (m >= p.M)
            continue;
#pragma unroll
        for (int j = 0; j < FN; j++) {
            const int n = n0 + wn + j * 16 + (lane >> 4) * 4;
            if (n < p.N) {
                const float s[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                epilogue4<T>(p, m, n, s);
            }
        }
    }
}

template <typename T, int BM, int BN, int WM, int WN>
hipError_t run_tile(const GemmArgs &a, int layout, hipStream_t s)
{
    const int64_t tm = ((int64_t)a.M + BM - 1) / BM, tn = ((int64_t)a.N + BN - 1) / BN;
    const dim3 grid((unsigned)(tm * tn)), block(WM * WN * WAVE);
    if (layout == 0)
        gemm_kernel<T, BM, BN, WM, WN, false, false><<<grid, block, 0, s>>>(a, (int)tn);
    else if (layout == GEMM_B_OUTER)
        gemm_kernel<T, BM, BN, WM, WN, false, true><<<grid, block, 0, s>>>(a, (int)tn);
    else
        gemm_kernel<T, BM, BN, WM, WN, true, true><<<grid, block, 0, s>>>(a, (int)tn);
    return hipGetLastError();
}

// ------------------------------------------------------------ dz and db
// Four columns a thread, a workgroup's rows in order: a column's partial sum
// is added in fp32 in row order, and the partials in workgroup order, so db
// is the same bits on every call.
constexpr int AG_THREADS = 256;
constexpr int AG_COLS = AG_THREADS * 4;
constexpr int AG_MIN_ROWS = 16;

template <typename T> __global__ __launch_bounds__(AG_THREADS) void act_grad_kernel(ActGradArgs p, int64_t rows_per)
{
    const int64_t n = ((int64_t)blockIdx.x * AG_THREADS + threadIdx.x) * 4;
    if (n >= p.N)
        return;
    const int valid = (int)(p.N - n < 4 ? p.N - n : 4);
    const int64_t r0 = (int64_t)blockIdx.y * rows_per, r1 = r0 + rows_per < p.M ? r0 + rows_per : p.M;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t m = r0; m < r1; m++) {
        float d[4], z[4];
        load4(static_cast<const T *>(p.dy) + m * p.lddy + n, valid, d);
        if (p.act != FA_ACT_NONE) {
            load4(static_cast<const T *>(p.pre) + m * p.ldp + n, valid, z);
#pragma unroll
            for (int i = 0; i < 4; i++)
                d[i] *= act_slope(z[i], p.act);
        }
        if (p.dz)
            store4(static_cast<T *>(p.dz) + m * p.N + n, valid, d);
#pragma unroll
        for (int i = 0; i < 4; i++)
            sum[i] += d[i];
    }
    if (p.db)
        store4(p.part + (int64_t)blockIdx.y * p.N + n, valid, sum);
}

template <typename T> __global__ __launch_bounds__(AG_THREADS) void column_join_kernel(ActGradArgs p, int64_t parts)
{
    const int64_t n = (int64_t)blockIdx.x * AG_THREADS + threadIdx.x;
    if (n >= p.N)
        return;
    float s = 0.f;
    for (int64_t q = 0; q < parts; q++)
        s += p.part[q * p.N + n];
    static_cast<T *>(p.db)[n] = (T)s;
}

} // namespace

size_t gemm_workspace_bytes(int, int64_t, int64_t, int64_t, int, int) { return 0; }

hipError_t launch_gemm(const GemmArgs &a, int dt, int layout, void *, int, hipStream_t s)
{
    if (a.M == 0 || a.N == 0)
        return hipSuccess;
    if (dt == FA_BF16)
        return run_tile<__bf16, 128, 128, 2, 2>(a, layout, s);
    return run_tile<float, 128, 128, 2, 2>(a, layout, s);
}

int64_t act_grad_partials(int64_t M, int64_t N, int cus)
{
    // enough workgroups for the chip, at least AG_MIN_ROWS rows each
    const int64_t across = (N + AG_COLS - 1) / AG_COLS;
    const int64_t want = std::max<int64_t>(1, 8 * (int64_t)cus / std::max<int64_t>(across, 1));
    return std::max<int64_t>(1, std::min(std::min<int64_t>(want, 1024), (M + AG_MIN_ROWS - 1) / AG_MIN_ROWS));
}

hipError_t launch_act_grad(const ActGradArgs &a, int dt, int cus, hipStream_t s)
{
    if (a.N == 0)
        return hipSuccess;
    const int64_t want = act_grad_partials(a.M, a.N, cus);
    const int64_t rows_per = std::max<int64_t>(1, (a.M + want - 1) / want);
    const int64_t parts = std::max<int64_t>(1, (a.M + rows_per - 1) / rows_per);
    const dim3 grid((unsigned)((a.N + AG_COLS - 1) / AG_COLS), (unsigned)parts);
    if (dt == FA_BF16)
        act_grad_kernel<__bf16><<<grid, AG_THREADS, 0, s>>>(a, rows_per);
    else
        act_grad_kernel<float><<<grid, AG_THREADS, 0, s>>>(a, rows_per);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.db)
        return e;
    const unsigned g = (unsigned)((a.N + AG_THREADS - 1) / AG_THREADS);
    if (dt == FA_BF16)
        column_join_kernel<__bf16><<<g, AG_THREADS, 0, s>>>(a, parts);
    else
        column_join_kernel<float><<<g, AG_THREADS, 0, s>>>(a, parts);
    return hipGetLastError();
}

} // namespace fa
