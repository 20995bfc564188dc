// Layers on 8-bit weights: rows of a matrix as 8-bit integers with a scale each,
// the products of such rows, and the weights as values for the input gradient.
//
// A row r is held as q(r,c) = rint(x(r,c) / s(r)), s(r) = max |x(r,.)| / 127, so
//     x w^T (m,n)  ~  sx(m) sw(n) sum_k xq(m,k) wq(n,k),
// a sum of whole numbers that the matrix cores form exactly (16x16x64); the
// scales come once per result, in the epilogue.
#include "tiles.h"

#include <algorithm>

namespace fa {
namespace {

// ------------------------------------------------------------ rows to 8 bits
// A group of threads holds its row in registers between the maximum and the
// quotients, QR_W values a thread at a time; what does not fit is read again.
// Bound by memory once the quotients are products: 14336 x 4096 bf16 (176 MB) in
// 38 us, 4.6 TB/s, where a copy of x (235 MB) takes 56, 4.2 TB/s; with a division for
// each value 48.  A row of 4096 on 256 threads takes 54 us, on a wavefront with one
// piece held and the others read twice, in fewer registers, 49.
constexpr int QR_THREADS = 256, QR_W = 16, QR_HELD = 4;

// Largest magnitude among W values, as the bits of an fp32 (NaN and infinities
// are the largest).
template <int W> __device__ __forceinline__ uint32_t top_bits(const Raw<float, W> &v, uint32_t top)
{
#pragma unroll
    for (int i = 0; i < W; i++) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v.e[i]) & 0x7fffffffu;
        top = b > top ? b : top;
    }
    return top;
}

template <int W> __device__ __forceinline__ uint32_t top_bits(const Raw<__bf16, W> &v, uint32_t top)
{
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 most = {(uint16_t)(top >> 16), 0};
#pragma unroll
    for (int i = 0; i < W; i += 2) {
        u16x2 b;
        __builtin_memcpy(&b, v.e + i, 4);
        most = __builtin_elementwise_max(most, b & (uint16_t)0x7fff);
    }
    return (uint32_t)(most.x > most.y ? most.x : most.y) << 16;
}

__device__ __forceinline__ int quotient(float x, float scale)
{
    const float q = __builtin_rintf(x / scale); // to even, as the division is IEEE's
    return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// q = the whole number nearest to fp32(x / scale).  t = fma(x, 1 / scale, 3 2^22)
// has it in its low bits; x times the rounded inverse is off by at most 127 2^-24
// and so is the rounded quotient, so only within 2.3e-5 of a tie can the two
// differ, and values that near are divided.  Scales below 2^-100, whose inverse
// leaves fp32 or loses bits, divide throughout.
constexpr float QR_MAGIC = 12582912.f, QR_TIE = 0.4999f, QR_LEAST = 0x1p-100f;

template <typename T> __device__ __forceinline__ u32x4 quotients(const Raw<T, QR_W> &v, float scale, float inverse)
{
    u32x4 out;
    float far = 0.f;
#pragma unroll
    for (int w = 0; w < 4; w++) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float x = (float)v.e[w * 4 + i], t = __builtin_fmaf(x, inverse, QR_MAGIC);
            far = fmaxf(far, fabsf(__builtin_fmaf(x, inverse, QR_MAGIC - t)));
            b[i] = __builtin_bit_cast(uint32_t, t);
        }
        // the low bytes of four words
        out[w] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400), __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400),
                                       0x05040100);
    }
    if (!(far < QR_TIE) || scale < QR_LEAST) {
#pragma unroll
        for (int w = 0; w < 4; w++) {
            uint32_t word = 0;
#pragma unroll
            for (int i = 0; i < 4; i++)
                word |= (uint32_t)(quotient((float)v.e[w * 4 + i], scale) & 255) << (8 * i);
            out[w] = word;
        }
    }
    return out;
}

// ACROSS threads take a row.  `fill`: columns up to which zeros follow the row.
template <typename T, int ACROSS>
__global__ __launch_bounds__(QR_THREADS) void quantize_kernel(const T *x, int64_t ldx, int64_t R, int64_t C, int8_t *q,
                                                              int64_t ldq, int64_t fill, float *scale)
{
    constexpr int ROWS = QR_THREADS / ACROSS;
    __shared__ uint32_t tops[2][QR_THREADS / WAVE];
    const int t = threadIdx.x % ACROSS;
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < R; r0 += (int64_t)gridDim.x * ROWS, turn ^= 1) {
        const int64_t r = r0 + threadIdx.x / ACROSS;
        const int64_t cols = r < R ? C : 0;
        const T *row = x + (r < R ? r : 0) * ldx;
        Raw<T, QR_W> held[QR_HELD];
        uint32_t top = 0;
#pragma unroll
        for (int h = 0; h < QR_HELD; h++) {
            const int64_t c = ((int64_t)h * ACROSS + t) * QR_W, left = cols - c;
            held[h].fetch(row + c, (int)(left < 0 ? 0 : left < QR_W ? left : QR_W));
        }
#pragma unroll
        for (int h = 0; h < QR_HELD; h++)
            top = top_bits(held[h], top);
        for (int64_t c = ((int64_t)QR_HELD * ACROSS + t) * QR_W; c < cols; c += ACROSS * QR_W) {
            Raw<T, QR_W> v;
            v.fetch(row + c, (int)(cols - c < QR_W ? cols - c : QR_W));
            top = top_bits(v, top);
        }
#pragma unroll
        for (int d = 1; d < (ACROSS < WAVE ? ACROSS : WAVE); d *= 2) {
            const uint32_t other = __shfl_xor(top, d);
            top = other > top ? other : top;
        }
        if constexpr (ACROSS > WAVE) {
            if (threadIdx.x % WAVE == 0)
                tops[turn][threadIdx.x / WAVE] = top;
            __syncthreads();
            top = tops[turn][0];
#pragma unroll
            for (int w = 1; w < ACROSS / WAVE; w++)
                top = tops[turn][w] > top ? tops[turn][w] : top;
        }
        const float s = top >= 0x7f800000u ? __builtin_nanf("") : __builtin_bit_cast(float, top) / 127.f;
        if (t == 0 && r < R)
            scale[r] = s;
        const bool live = s > 0.f;
        const float inverse = 1.f / s;
        const auto put = [&](int64_t c, const Raw<T, QR_W> &v) {
            const int64_t end = r < R ? fill : 0;
            if (c >= end)
                return;
            const u32x4 b = live ? quotients(v, s, inverse) : u32x4{0, 0, 0, 0};
            int8_t *to = q + r * ldq + c;
            if (end - c >= QR_W && (reinterpret_cast<uintptr_t>(to) & 15) == 0) {
                __builtin_nontemporal_store(b, reinterpret_cast<u32x4 *>(to)); // 40.7 us against 43.1 through the caches
            } else if (end - c >= QR_W) {
                __builtin_memcpy(to, &b, QR_W);
            } else {
#pragma unroll
                for (int i = 0; i < QR_W; i++)
                    if (i < end - c)
                        to[i] = (int8_t)(b[i / 4] >> (i % 4 * 8));
            }
        };
#pragma unroll
        for (int h = 0; h < QR_HELD; h++)
            put(((int64_t)h * ACROSS + t) * QR_W, held[h]);
        for (int64_t c = ((int64_t)QR_HELD * ACROSS + t) * QR_W; c < fill; c += ACROSS * QR_W) {
            Raw<T, QR_W> v;
            const int64_t left = cols - c;
            v.fetch(row + c, (int)(left < 0 ? 0 : left < QR_W ? left : QR_W));
            put(c, v);
        }
    }
}

// ------------------------------------------------------------ products
// Workgroup (tile, split), as for the other products; partial sums are whole
// numbers too, so a split changes no result.  Steps are short, so aligned operands
// go through four buffers: 777 x 2048 x 8192 in 64 x 64 tiles 33 us, with two 37.
// Fragments and bytes are those of the 16-bit products, at twice the operations:
// 8192 x 14336 x 4096 in 525 us (1.83 POP/s; the vendor library's product alone 505).
template <typename O, int BM, int BN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(WM *WN *WAVE) void gemm8_kernel(GemmArgs p, int tiles_m, int tiles_n, int kper, float *part)
{
    typedef int8_t T;
    constexpr int THREADS = WM * WN * WAVE, BK = STEP_BYTES;
    constexpr int AB = BM * STEP_BYTES, BB = BN * STEP_BYTES;
    __shared__ __attribute__((aligned(1024))) char l0[AB + BB];
    __shared__ __attribute__((aligned(1024))) char l1[AB + BB];
    __shared__ __attribute__((aligned(1024))) char l2[DIRECT ? AB + BB : 16];
    __shared__ __attribute__((aligned(1024))) char l3[DIRECT ? AB + BB : 16];

    unsigned tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int m0 = (int)tm * BM, n0 = (int)tn * BN;
    const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
    const T *a = static_cast<const T *>(p.a), *b = static_cast<const T *>(p.b);
    const int k0 = blockIdx.y * kper, kend = p.K - k0 < kper ? p.K : k0 + kper;
    const int steps = (kend - k0 + BK - 1) / BK;
    Tile<T, BM, BN, WM, WN, false, false> t;
    t.clear();
    if constexpr (DIRECT) {
        Direct<T, false, BM, THREADS, STEP_BYTES> da;
        Direct<T, false, BN, THREADS, STEP_BYTES> db;
        da.init(a, p.lda, m0, p.M, k0);
        db.init(b, p.ldb, n0, p.N, k0);
        t.template run<AB / 16 / THREADS + BB / 16 / THREADS>(l0, l1, l2, l3, steps, wm, wn, lane, [&](char *l, int s) {
            da.start(l, kend - k0 - s * BK);
            db.start(l + AB, kend - k0 - s * BK);
        });
    } else {
        Stage<T, false, BM, THREADS> sa;
        Stage<T, false, BN, THREADS> sb;
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
    write_tile<O, BM, BN, WM, WN, AB + BB>(p, m0, n0, t.acc, l0, l1, part);
}

template <typename O, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM *WN *WAVE) void pipe8_kernel(GemmArgs p, int tiles_m, int tiles_n)
{
    typedef int8_t T;
    constexpr int THREADS = WM * WN * WAVE, BK = PIPE_STEP;
    constexpr int AB = BM * PIPE_STEP, BB = BN * PIPE_STEP;
    __shared__ __attribute__((aligned(1024))) char l0[AB + BB];
    __shared__ __attribute__((aligned(1024))) char l1[AB + BB];
    __shared__ __attribute__((aligned(1024))) char l2[AB + BB];
    __shared__ __attribute__((aligned(1024))) char l3[AB + BB];

    unsigned tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int m0 = (int)tm * BM, n0 = (int)tn * BN;
    Pipe<T, BM, BN, WM, WN, false, false> t;
    Direct<T, false, BM, THREADS, PIPE_STEP> da;
    Direct<T, false, BN, THREADS, PIPE_STEP> db;
    da.init(static_cast<const T *>(p.a), p.lda, m0, p.M, 0);
    db.init(static_cast<const T *>(p.b), p.ldb, n0, p.N, 0);
    int left = p.K; // of the next step to copy; steps past the end copy zeros
    t.run(l0, l1, l2, l3, (p.K + BK - 1) / BK, [&](char *l) {
        da.start(l, left);
        db.start(l + AB, left);
        left -= BK;
    });
    write_tile<O, BM, BN, WM, WN, AB + BB>(p, m0, n0, t.acc, l0, l1, nullptr);
}

// Joins the splits' sums, four neighbours a thread, and finishes them.
constexpr int J8_THREADS = 256, J8_W = 4;

template <typename O> __global__ __launch_bounds__(J8_THREADS) void join8_kernel(GemmArgs p, const int32_t *part, int splits)
{
    const int64_t groups = (p.N + J8_W - 1) / J8_W;
    const int64_t at = (int64_t)blockIdx.x * J8_THREADS + threadIdx.x;
    if (at >= p.M * groups)
        return;
    const int64_t m = at / groups;
    const int n = (int)(at % groups) * J8_W, valid = p.N - n;
    int32_t sum[J8_W] = {};
#pragma unroll 4
    for (int z = 0; z < splits; z++) {
        Raw<int32_t, J8_W> v;
        v.fetch(part + ((int64_t)z * p.M + m) * p.N + n, valid);
#pragma unroll
        for (int i = 0; i < J8_W; i++)
            sum[i] += v.e[i];
    }
    Raw<float, J8_W> cs;
    cs.fetch(p.col_scale + n, valid);
    Raw<O, J8_W> bias, res;
    fetch_bias(p, n, bias);
    fetch_residual(p, m, n, res);
    float v[J8_W];
    scaled_sums<J8_W>(sum, p.row_scale[m], cs.e, v);
    epilogue<O, J8_W>(p, m, n, v, bias, res);
}

// ------------------------------------------------------------ few tokens
// Up to FEW_M rows of x against all weights, in one launch: bound by the weights'
// bytes and by latency.  A workgroup has 16 columns and each of its wavefronts a
// range of k (the next 16 after them, where there are more than FEW_PER_CU
// workgroups a CU); the first 2 FEW_AHEAD fragments of the weights are on their way
// before the workgroup looks at x, which it brings to 8 bits itself (X: its type;
// int8_t: as it is), FEW_PIECES pieces of 4096 in all.  One token of bf16 through
// 14336 x 4096 weights (59 MB): 12.7 to 13.7 us.  Other forms were timed beside an
// earlier one of 15.4: as 16 x 128 tiles after a launch for x, with the join of two
// splits, 18.6; with 8 fragments on their way, or loads past the caches, 18.4.
constexpr int FEW_M = 4, FEW_WAVES = 4, FEW_THREADS = FEW_WAVES * WAVE, FEW_AHEAD = 4, FEW_PER_CU = 4, FEW_PIECES = 4;

__device__ __forceinline__ int64_t few_pitch(int64_t K) { return (K + WAVE - 1) / WAVE * WAVE; }

template <typename O, typename X>
__global__ __launch_bounds__(FEW_THREADS) void few_kernel(GemmArgs p, int range)
{
    extern __shared__ __attribute__((aligned(16))) int8_t xq[]; // [M][pitch], zeros behind the rows
    __shared__ int32_t sums[FEW_WAVES][FEW_M][16];
    __shared__ uint32_t tops[FEW_PIECES][FEW_WAVES];
    __shared__ float scales[FEW_M];
    const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE, i = lane & 15, g = lane >> 4;
    const int pitch = (int)few_pitch(p.K);
    const int k0 = wave * range, k1 = p.K - k0 < range ? p.K : k0 + range; // may be empty
    const int steps = k1 > k0 ? (k1 - k0 + WAVE - 1) / WAVE : 0;
    // fragments of row n0 + i, 16 bytes each; past the row's end or the last row zeros
    Frag fw[2][FEW_AHEAD];
    const auto fetch = [&](Frag (&f)[FEW_AHEAD], int64_t n0, int first) {
        const int8_t *w = static_cast<const int8_t *>(p.b) + (n0 + i) * p.ldb + k0 + g * 16;
        const int left = n0 + i < p.N ? k1 - k0 - g * 16 : 0;
#pragma unroll
        for (int e = 0; e < FEW_AHEAD; e++) {
            const int k = (first + e) * WAVE;
            f[e].v = u32x4{0, 0, 0, 0};
            if (k < left)
                f[e].v = *reinterpret_cast<const u32x4 *>(w + k);
        }
    };

    // x in pieces of a row, one a thread, FEW_PIECES in all: they are on their way
    // before the weights, which they would have to wait for otherwise
    constexpr bool WHOLE = __is_same(X, int8_t);
    const int per_row = (pitch + FEW_THREADS * 16 - 1) / (FEW_THREADS * 16);
    const auto piece = [&](int e, int &m, int &c) {
        m = e / per_row;
        c = (e % per_row * FEW_THREADS + threadIdx.x) * 16;
    };
    Raw<X, 16> x[FEW_PIECES];
#pragma unroll
    for (int e = 0; e < FEW_PIECES; e++) {
        int m, c;
        piece(e, m, c);
        const int n = m < p.M ? p.K - c : 0;
        x[e].fetch(static_cast<const X *>(p.a) + m * p.lda + c, n < 0 ? 0 : n < 16 ? n : 16);
    }
    int64_t n0 = (int64_t)blockIdx.x * 16;
    fetch(fw[0], n0, 0);
    fetch(fw[1], n0, FEW_AHEAD);
    uint32_t top[FEW_PIECES] = {};
    if constexpr (!WHOLE) {
#pragma unroll
        for (int e = 0; e < FEW_PIECES; e++) {
            top[e] = top_bits(x[e], 0);
#pragma unroll
            for (int d = 1; d < WAVE; d *= 2) {
                const uint32_t other = __shfl_xor(top[e], d);
                top[e] = other > top[e] ? other : top[e];
            }
            if (lane == 0)
                tops[e][wave] = top[e];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < FEW_PIECES; e++)
#pragma unroll
            for (int f = 0; f < FEW_PIECES; f++)
                if (e / per_row == f / per_row)
#pragma unroll
                    for (int v = 0; v < FEW_WAVES; v++)
                        top[e] = tops[f][v] > top[e] ? tops[f][v] : top[e];
    }
#pragma unroll
    for (int e = 0; e < FEW_PIECES; e++) {
        int m, c;
        piece(e, m, c);
        u32x4 q;
        if constexpr (WHOLE) {
            __builtin_memcpy(&q, x[e].e, 16);
        } else {
            const float s = top[e] >= 0x7f800000u ? __builtin_nanf("") : __builtin_bit_cast(float, top[e]) / 127.f;
            q = s > 0.f ? quotients(x[e], s, 1.f / s) : u32x4{0, 0, 0, 0};
            if (threadIdx.x == 0 && m < p.M)
                scales[m] = s;
        }
        if (m < p.M && c < pitch)
            *reinterpret_cast<u32x4 *>(xq + m * pitch + c) = q;
    }
    __syncthreads();

    // rows of x past M repeat the last: their results are not looked at
    const int8_t *xr = xq + (i < p.M ? i : p.M - 1) * pitch + k0 + g * 16;
    for (;;) {
        i32x4 acc = {0, 0, 0, 0};
        const auto use = [&](const Frag (&f)[FEW_AHEAD], int first) {
#pragma unroll
            for (int e = 0; e < FEW_AHEAD; e++)
                if (first + e < steps) {
                    Frag fx;
                    fx.v = *reinterpret_cast<const u32x4 *>(xr + (first + e) * WAVE);
                    acc = mma<int8_t>(f[e], fx, acc);
                }
        };
        const int64_t next = n0 + (int64_t)gridDim.x * 16;
        for (int s = 0; s < steps; s += 2 * FEW_AHEAD) {
            // behind the last steps the next columns' first fragments
            const bool more = s + 2 * FEW_AHEAD < steps;
            use(fw[0], s);
            fetch(fw[0], more ? n0 : next, more ? s + 2 * FEW_AHEAD : 0);
            use(fw[1], s + FEW_AHEAD);
            fetch(fw[1], more ? n0 : next, more ? s + 3 * FEW_AHEAD : FEW_AHEAD);
        }
        // lane l holds row l % 16, columns 4 (l / 16) ..
        if (i < p.M)
            *reinterpret_cast<i32x4 *>(&sums[wave][i][g * 4]) = acc;
        __syncthreads();
        const int m = threadIdx.x / 16;
        const int64_t n = n0 + threadIdx.x % 16;
        if (m < p.M && n < p.N) {
            int32_t sum[1] = {0};
#pragma unroll
            for (int e = 0; e < FEW_WAVES; e++)
                sum[0] += sums[e][m][threadIdx.x % 16];
            const float row = WHOLE ? p.row_scale[m] : scales[m];
            const float col[1] = {p.col_scale[n]};
            float v[1];
            Raw<O, 1> bias, res;
            fetch_bias(p, (int)n, bias);
            fetch_residual(p, m, (int)n, res);
            scaled_sums<1>(sum, row, col, v);
            epilogue<O, 1>(p, m, (int)n, v, bias, res);
        }
        n0 = next;
        if (n0 >= p.N)
            break;
        __syncthreads();
    }
}

// ------------------------------------------------------------ the input gradient
// dx(m,k) = sum_n u(m,n) w(n,k) with u = dz sw in PLANES of bf16: one for bf16
// results, three for fp32 (u = a + 2^-8 b + 2^-16 c, 8 bits each, exactly).  The
// 8-bit weights are exact in bf16 as well, so three products on the 16-bit matrix
// cores, whose sums are joined at the end, give fp32's precision at five times its
// rate.  w stays in 8 bits up to the
// registers: a transposing read gives a lane its column's eight bytes.
// 4096 x 8192 x 2048 fp32 in 451 us with the pass over dz (0.91 PFLOP/s of
// 16-bit products), as products in fp32 1035; 64 x 14336 x 4096 bf16 in 29, with the
// weights written out as values first 82.  Small tiles take four buffers where
// they are short (bf16), two and a second workgroup on the CU where not: 512 x 8192
// x 2048 fp32 82 us, with four 102.
constexpr int GRAD_STEP = 64; // n a step

// Rows of 8-bit weights, GRAD_STEP of them by COLS; the 16-byte chunks of row k
// are exchanged so that the rows that a read touches spread over the banks.
template <int COLS, int THREADS> struct ByteRows {
    static constexpr int CPR = COLS / 16, CHUNKS = GRAD_STEP * CPR, CH = CHUNKS / THREADS;
    static_assert(CHUNKS % THREADS == 0, "every thread copies as much");
    uint32_t off[CH];
    const char *base;
    int64_t advance;

    static __device__ __forceinline__ int swizzle(int k) { return COLS == 64 ? (k >> 2) & 3 : (k >> 1) & 7; }

    __device__ __forceinline__ void init(const int8_t *w, int64_t ld, int c0, int cols, int k0)
    {
        base = reinterpret_cast<const char *>(w + (int64_t)k0 * ld + c0);
        advance = GRAD_STEP * ld;
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int q = threadIdx.x + c * THREADS, k = q / CPR, ch = (q % CPR) ^ swizzle(k);
            off[c] = c0 + ch * 16 < cols ? (uint32_t)(k * ld) + ch * 16 : OUT_OF_RANGE;
        }
    }

    __device__ __forceinline__ void start(char *tile, int64_t shift, int left) const
    {
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base + shift), 0, (int)OUT_OF_RANGE, 0x00020000);
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int first = (threadIdx.x / WAVE) * WAVE + c * THREADS;
            uint32_t o = off[c];
            if (left < GRAD_STEP)
                o = (threadIdx.x + c * THREADS) / CPR < left ? o : OUT_OF_RANGE;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void *)(tile + first * 16), 16, o, 0, 0, 0);
        }
    }

    // Columns c0 .. c0 + 15 at the rows 32 kk .. 32 kk + 31 as a fragment in bf16.
    static __device__ __forceinline__ Frag read(const char *tile, int c0, int kk, int lane)
    {
        typedef int v2i __attribute__((ext_vector_type(2)));
        const int i = lane & 15, g = lane >> 4, k = kk * 32 + 8 * g + (i >> 1);
        const char *at = tile + (k * COLS + (((c0 >> 4) ^ swizzle(k)) << 4) + 8 * (i & 1));
        const v2i b = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) v2i *)const_cast<char *>(at));
        Frag f;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; e++)
                v[e] = __builtin_bit_cast(uint32_t, (float)(int8_t)(b[h] >> (8 * e)));
            f.v[2 * h] = __builtin_amdgcn_perm(v[1], v[0], 0x07060302); // the upper halves: exact
            f.v[2 * h + 1] = __builtin_amdgcn_perm(v[3], v[2], 0x07060302);
        }
        return f;
    }
};

template <typename O, int PLANES, int BM, int BN, int WM, int WN, int BUFS>
__global__ __launch_bounds__(WM *WN *WAVE) void grad8_kernel(GemmArgs p, int64_t plane, int tiles_m, int tiles_n, int kper, float *part)
{
    typedef __bf16 T;
    constexpr int THREADS = WM * WN * WAVE, FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr int AB = BM * STEP_BYTES, BYTES = PLANES * AB + GRAD_STEP * BN; // of a buffer
    constexpr int COPIES = BYTES / 16 / THREADS;
    static_assert(AB % (16 * THREADS) == 0 && (BUFS == 2 || BUFS == 4), "every thread copies as much");
    __shared__ __attribute__((aligned(1024))) char l0[BYTES];
    __shared__ __attribute__((aligned(1024))) char l1[BYTES];
    __shared__ __attribute__((aligned(1024))) char l2[BUFS == 4 ? BYTES : 16];
    __shared__ __attribute__((aligned(1024))) char l3[BUFS == 4 ? BYTES : 16];

    unsigned tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int m0 = (int)tm * BM, n0 = (int)tn * BN;
    const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
    const int k0 = blockIdx.y * kper, kend = p.K - k0 < kper ? p.K : k0 + kper;
    const int steps = (kend - k0 + GRAD_STEP - 1) / GRAD_STEP;
    Direct<T, false, BM, THREADS, STEP_BYTES> a;
    ByteRows<BN, THREADS> b;
    a.init(static_cast<const T *>(p.a), p.lda, m0, p.M, k0);
    b.init(static_cast<const int8_t *>(p.b), p.ldb, n0, p.N, k0);
    f32x4 acc[PLANES][FM][FN];
#pragma unroll
    for (int q = 0; q < PLANES; q++)
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < FN; j++)
                acc[q][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const auto copy = [&](char *l, int s) {
        const int left = kend - k0 - s * GRAD_STEP;
#pragma unroll
        for (int q = 0; q < PLANES; q++)
            a.start_at(l + q * AB, s * a.advance + q * plane * 2, left);
        b.start(l + PLANES * AB, s * b.advance, left);
    };
    const auto step = [&](const char *l) {
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
            Frag fa[PLANES][FM], fb[FN];
#pragma unroll
            for (int j = 0; j < FN; j++)
                fb[j] = ByteRows<BN, THREADS>::read(l + PLANES * AB, wn + j * 16, kk, lane);
#pragma unroll
            for (int q = 0; q < PLANES; q++)
#pragma unroll
                for (int i = 0; i < FM; i++)
                    fa[q][i] = read_frag<T, false, BM, STEP_BYTES>(l + q * AB, wm + i * 16, kk, lane);
#pragma unroll
            for (int q = 0; q < PLANES; q++)
#pragma unroll
                for (int i = 0; i < FM; i++)
#pragma unroll
                    for (int j = 0; j < FN; j++)
                        acc[q][i][j] = mma<T>(fb[j], fa[q][i], acc[q][i][j]);
        }
    };
    if constexpr (BUFS == 4) {
        const auto turn = [&](const char *cur, char *free, int t) {
            if (t + 2 < steps)
                copies_done<2 * COPIES, true>();
            else if (t + 1 < steps)
                copies_done<COPIES, true>();
            else
                copies_done<0, true>();
            if (t + 3 < steps)
                copy(free, t + 3);
            step(cur);
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
    } else {
        if (steps > 0)
            copy(l0, 0);
        for (int s = 0; s < steps; s += 2) {
            copies_done<0, true>();
            if (s + 1 < steps)
                copy(l1, s + 1);
            step(l0);
            if (s + 1 < steps) {
                copies_done<0, true>();
                if (s + 2 < steps)
                    copy(l0, s + 2);
                step(l1);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = PLANES - 1; q > 0; q--)
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < FN; j++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    acc[q - 1][i][j][e] = __builtin_fmaf(0x1p-8f, acc[q][i][j][e], acc[q - 1][i][j][e]);
    write_tile<O, BM, BN, WM, WN, BYTES>(p, m0, n0, acc[0], l0, l1, part);
}

// ------------------------------------------------------------ weights as values
// The whole numbers of wq in T (exact), rows of `ldo` elements with zeros behind
// the row; with T = int8_t a copy whose rows are whole chunks.  Bound by memory.
constexpr int WV_THREADS = 256, WV_W = 16;

template <typename T>
__global__ __launch_bounds__(WV_THREADS) void widen_kernel(const int8_t *w, int64_t ldw, int64_t rows, int64_t cols, T *out,
                                                           int64_t ldo)
{
    const int64_t per = (ldo + WV_W - 1) / WV_W, step = (int64_t)gridDim.x * WV_THREADS;
    for (int64_t at = (int64_t)blockIdx.x * WV_THREADS + threadIdx.x; at < rows * per; at += step) {
        const int64_t r = at / per, c = at % per * WV_W, left = cols - c;
        Raw<int8_t, WV_W> v;
        v.fetch(w + r * ldw + c, (int)(left < 0 ? 0 : left < WV_W ? left : WV_W));
        int32_t e[WV_W];
#pragma unroll
        for (int i = 0; i < WV_W; i++)
            e[i] = v.e[i];
        store_n<T, WV_W>(out + r * ldo + c, (int)(ldo - c < WV_W ? ldo - c : WV_W), e);
    }
}

// ------------------------------------------------------------ launches

int64_t tiles8(int64_t M, int64_t N, int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

bool pitch_ok(int64_t bytes) { return bytes * 257 < (int64_t)OUT_OF_RANGE; }

// Whether rows start on 16 bytes and end on a whole chunk, or in zeros up to one.
bool direct_ok(const void *p, int64_t ld, int64_t row, bool padded)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 16 == 0 && (padded || row % 16 == 0) && pitch_ok(ld);
}

enum { P8_256_256, P8_256_128, P8_128_256, P8_128_128, T8_64, T8_THIN_N, T8_THIN_M };

struct Plan8 {
    int tile, splits;
};

// Larger tiles are compared by the rounds that they need on all CUs, as for bf16: one
// of 256x256, 256x128 or 128x256 fits a CU at a time, two of 128x128.  Measured on
// 256 CUs, us of a round for K = 16384; the last is a round of 128x128 with one tile
// a CU.  For example, in that order: 8192x14336x4096 436, 545, 543, 589;
// 4096x2048x16384 172, 132, 133, 161; 2048x2048x16384 158, 103, 97, 77;
// 6144x4096x16384, two rounds of 256x256 of which the second is half, 370, 387, 386,
// 461.
int pipe8_for(int64_t M, int64_t N, int cus)
{
    static const int us[5] = {215, 131, 132, 161, 77};
    const auto rounds = [&](int64_t t) { return (t + cus - 1) / cus; };
    const int64_t t128 = tiles8(M, N, 128, 128), whole = t128 / (2 * cus), rest = t128 % (2 * cus);
    const int64_t costs[4] = {us[0] * rounds(tiles8(M, N, 256, 256)), us[1] * rounds(tiles8(M, N, 256, 128)),
                              us[2] * rounds(tiles8(M, N, 128, 256)),
                              us[3] * whole + (rest > cus ? us[3] : rest > 0 ? us[4] : 0)};
    return (int)(std::min_element(costs, costs + 4) - costs);
}

// Products that 64x64 tiles would cover with more than two a CU take larger ones: us of
// 128x128 and 64x64, operands in turn: 1024x2048x4096 (512 tiles) 32, 21; 1152x2048
// 31.6, 33.7; 1920x2048 33, 38; 777x2048x8192 54, 36; 300x8192x4096 32, 37.  Staged
// through registers, larger tiles pay later: 300x8192x1001 20, 14; 400x8192 21, 17;
// 500x12288 27, 31; 400x14336x2047 35, 42.  Fewer 64x64 tiles than CUs are split
// along k up to the CUs, in four steps or more: 256x1024x4096 in 1, 2, 4, 8 15, 12.5,
// 11.2, 13.5; 100x128x4096 in 4, 8, 16 8.6, 7.7, 8.0; 64x4096x14336 in 2, 4, 8 33, 22,
// 21; 333x555x2048 in 1, 4 9.5, 10.3.  Thin tiles, which stream one operand, up to
// three workgroups for two CUs: 16x4096x4096 (32 tiles) in 4, 8, 12, 16 9.6, 9.9, 11.4,
// 11.8; 16x8192x8192 in 2, 4, 6 21, 17, 19; 8x14336x4096 in 1, 2, 4 17.1, 15.2, 16.4;
// staged 16x8192x4095 in 4, 6, 8 20, 16, 17.
Plan8 plan8(int64_t M, int64_t N, int64_t K, int cus)
{
    const int64_t steps = K / STEP_BYTES;
    const auto split = [&](int64_t count, int64_t want) {
        return (int)std::max<int64_t>(1, std::min<int64_t>(std::min((want + count - 1) / count, steps / 4), 16));
    };
    if (N <= 16)
        return {T8_THIN_N, split(std::max<int64_t>(1, tiles8(M, N, 128, 16)), 3 * cus / 2)};
    if (M <= 16)
        return {T8_THIN_M, split(std::max<int64_t>(1, tiles8(M, N, 16, 128)), 3 * cus / 2)};
    if (tiles8(M, N, 64, 64) > 2 * cus)
        return {pipe8_for(M, N, cus), 1};
    return {T8_64, split(std::max<int64_t>(1, tiles8(M, N, 64, 64)), cus)};
}

template <typename O, int BM, int BN, int WM, int WN>
hipError_t run_tile8(const GemmArgs &a, bool direct, int splits, void *ws, hipStream_t s)
{
    const int64_t tm = ((int64_t)a.M + BM - 1) / BM, tn = ((int64_t)a.N + BN - 1) / BN;
    const int steps = std::max(1, (a.K + STEP_BYTES - 1) / STEP_BYTES), per = (steps + splits - 1) / splits;
    const int used = (steps + per - 1) / per;
    float *part = used > 1 ? static_cast<float *>(ws) : nullptr;
    const dim3 grid((unsigned)(tm * tn), (unsigned)used), block(WM * WN * WAVE);
    constexpr bool SMALL = BM * BN < 128 * 128; // larger tiles of aligned operands are pipe8_kernel's
    const auto kernel = SMALL && direct ? gemm8_kernel<O, BM, BN, WM, WN, SMALL> : gemm8_kernel<O, BM, BN, WM, WN, false>;
    kernel<<<grid, block, 0, s>>>(a, (int)tm, (int)tn, per * STEP_BYTES, part);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && used > 1) {
        const int64_t threads = (int64_t)a.M * ((a.N + J8_W - 1) / J8_W);
        join8_kernel<O><<<(unsigned)((threads + J8_THREADS - 1) / J8_THREADS), J8_THREADS, 0, s>>>(
            a, reinterpret_cast<const int32_t *>(part), used);
        e = hipGetLastError();
    }
    return e;
}

template <typename O, int BM, int BN, int WM, int WN> hipError_t run_pipe8(const GemmArgs &a, hipStream_t s)
{
    const int64_t tm = ((int64_t)a.M + BM - 1) / BM, tn = ((int64_t)a.N + BN - 1) / BN;
    pipe8_kernel<O, BM, BN, WM, WN><<<(unsigned)(tm * tn), WM * WN * WAVE, 0, s>>>(a, (int)tm, (int)tn);
    return hipGetLastError();
}

// Tiles of the input gradient and how often n is split.
struct GradPlan {
    int tile, splits, kper;
};

GradPlan grad_plan(int64_t M, int64_t N, int64_t K, int planes, int cus)
{
    // Small tiles fill a CU three times over (bf16) or twice (fp32): with one, two,
    // three a CU 512 x 8192 x 2048 bf16 72, 51, 46 us, fp32 98, 82, 105.
    const bool large = tiles8(M, N, 128, 128) >= cus;
    const int64_t count = large ? tiles8(M, N, 128, 128) : std::max<int64_t>(1, tiles8(M, N, 64, 64));
    const int64_t steps = std::max<int64_t>(1, (K + GRAD_STEP - 1) / GRAD_STEP);
    const int64_t want = large ? 1 : std::max<int64_t>(1, std::min<int64_t>({(planes == 1 ? 3 : 2) * cus / count, steps / 4, 16}));
    const int64_t per = (steps + want - 1) / want;
    return {large ? 128 : 64, (int)((steps + per - 1) / per), (int)(per * GRAD_STEP)};
}

template <typename O, int PLANES> hipError_t run_grad(const GemmArgs &a, int64_t plane, float *ws, int cus, Finish &f, hipStream_t s)
{
    const GradPlan p = grad_plan(a.M, a.N, a.K, PLANES, cus);
    const int tm = (a.M + p.tile - 1) / p.tile, tn = (a.N + p.tile - 1) / p.tile;
    float *part = p.splits > 1 ? ws : nullptr;
    const dim3 grid((unsigned)((int64_t)tm * tn), (unsigned)p.splits);
    if (p.tile == 128)
        grad8_kernel<O, PLANES, 128, 128, 2, 4, 2><<<grid, 512, 0, s>>>(a, plane, tm, tn, p.kper, part);
    else
        grad8_kernel<O, PLANES, 64, 64, 2, 2, PLANES == 1 ? 4 : 2><<<grid, 256, 0, s>>>(a, plane, tm, tn, p.kper, part);
    if (p.splits > 1) {
        const int j = f.blocks[0] > 0;
        f.p[j] = a;
        f.part[j] = part;
        f.splits[j] = p.splits;
        f.blocks[j] = finish_blocks(a.M, a.N);
    }
    return hipGetLastError();
}

template <typename O, typename X> hipError_t run_few(const GemmArgs &a, int cus, hipStream_t s)
{
    const int per = (a.K + FEW_WAVES - 1) / FEW_WAVES, range = (per + WAVE - 1) / WAVE * WAVE;
    const size_t lds = (size_t)a.M * ((a.K + WAVE - 1) / WAVE * WAVE);
    const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)a.N + 15) / 16, (int64_t)FEW_PER_CU * cus);
    few_kernel<O, X><<<grid, FEW_THREADS, lds, s>>>(a, range);
    return hipGetLastError();
}

template <typename T> hipError_t widen(const int8_t *w, int64_t ldw, int64_t rows, int64_t cols, T *out, int64_t ldo, hipStream_t s)
{
    const int64_t chunks = rows * ((ldo + WV_W - 1) / WV_W);
    const unsigned grid = (unsigned)std::min<int64_t>((chunks + WV_THREADS - 1) / WV_THREADS, 1 << 20);
    widen_kernel<T><<<grid, WV_THREADS, 0, s>>>(w, ldw, rows, cols, out, ldo);
    return hipGetLastError();
}

int64_t row16(int64_t K) { return (K + 15) / 16 * 16; }

// Large products repay copies of odd rows with whole ones, us staged through
// registers and copied: 8191 x 4096 x 4095 269, 189; 4096 x 8191 x 100 60, 50;
// 2047 x 2047 x 513 26, 22; 300 x 4096 x 1001 20, 23; 8 x 14336 x 4097 23, 45.
constexpr double PACK8_LEAST = 2e9;
constexpr int64_t PACK8_ROWS = 512;

bool pack8_wanted(int64_t M, int64_t N, int64_t K)
{
    return K % 16 != 0 && M >= PACK8_ROWS && (double)M * (double)N * (double)K >= PACK8_LEAST && pitch_ok(row16(K));
}

size_t part8_bytes(int64_t M, int64_t N, int64_t K, int cus)
{
    const Plan8 p = plan8(M, N, K, cus);
    return p.splits > 1 ? ((size_t)p.splits * M * N * sizeof(int32_t) + 255) / 256 * 256 : 0;
}

template <typename O> hipError_t gemm8_of(GemmArgs a, void *ws, int cus, hipStream_t s)
{
    const Plan8 p = plan8(a.M, a.N, a.K, cus);
    bool ok_a = direct_ok(a.a, a.lda, a.K, a.a_padded), ok_b = direct_ok(a.b, a.ldb, a.K, false);
    if (!(ok_a && ok_b) && pack8_wanted(a.M, a.N, a.K)) {
        int8_t *to = static_cast<int8_t *>(ws) + part8_bytes(a.M, a.N, a.K, cus);
        const int64_t row = row16(a.K);
        hipError_t e = ok_b ? hipSuccess : widen<int8_t>(static_cast<const int8_t *>(a.b), a.ldb, a.N, a.K, to, row, s);
        if (!ok_b) {
            a.b = to;
            a.ldb = row;
            to += a.N * row;
        }
        if (e == hipSuccess && !ok_a) {
            e = widen<int8_t>(static_cast<const int8_t *>(a.a), a.lda, a.M, a.K, to, row, s);
            a.a = to;
            a.lda = row;
        }
        if (e != hipSuccess)
            return e;
        ok_a = ok_b = true;
    }
    const bool direct = ok_a && ok_b;
    if (few8_ok(a.M, a.K, a.b, a.ldb))
        return run_few<O, int8_t>(a, cus, s);
    if (p.tile <= P8_128_128) {
        if (!direct && tiles8(a.M, a.N, 128, 128) > cus)
            return run_tile8<O, 128, 128, 2, 2>(a, false, 1, ws, s);
        if (!direct)
            return run_tile8<O, 64, 64, 2, 2>(a, false, 1, ws, s);
        if (p.tile == P8_256_256)
            return run_pipe8<O, 256, 256, 2, 4>(a, s);
        if (p.tile == P8_256_128)
            return run_pipe8<O, 256, 128, 4, 2>(a, s);
        if (p.tile == P8_128_256)
            return run_pipe8<O, 128, 256, 2, 4>(a, s);
        return run_pipe8<O, 128, 128, 2, 4>(a, s);
    }
    if (p.tile == T8_64)
        return run_tile8<O, 64, 64, 2, 2>(a, direct, p.splits, ws, s);
    if (p.tile == T8_THIN_N)
        return run_tile8<O, 128, 16, 4, 1>(a, direct, p.splits, ws, s);
    return run_tile8<O, 16, 128, 1, 4>(a, direct, p.splits, ws, s);
}

template <typename T> hipError_t quantize(const QuantizeArgs &a, hipStream_t s)
{
    const T *x = static_cast<const T *>(a.x);
    const auto grid = [&](int64_t rows) { return (unsigned)std::min<int64_t>((a.R + rows - 1) / rows, 1 << 20); };
    if (a.C <= 16 * QR_W * QR_HELD)
        quantize_kernel<T, 16><<<grid(QR_THREADS / 16), QR_THREADS, 0, s>>>(x, a.ldx, a.R, a.C, a.q, a.ldq, a.fill, a.scale);
    else if (a.C <= WAVE * QR_W * QR_HELD)
        quantize_kernel<T, WAVE><<<grid(QR_THREADS / WAVE), QR_THREADS, 0, s>>>(x, a.ldx, a.R, a.C, a.q, a.ldq, a.fill, a.scale);
    else
        quantize_kernel<T, QR_THREADS><<<grid(1), QR_THREADS, 0, s>>>(x, a.ldx, a.R, a.C, a.q, a.ldq, a.fill, a.scale);
    return hipGetLastError();
}

} // namespace

hipError_t launch_quantize(const QuantizeArgs &a, int dt, hipStream_t s)
{
    if (a.R == 0)
        return hipSuccess;
    return dt == FA_BF16 ? quantize<__bf16>(a, s) : quantize<float>(a, s);
}

size_t gemm8_workspace_bytes(int64_t M, int64_t N, int64_t K, int cus)
{
    return part8_bytes(M, N, K, cus) + (pack8_wanted(M, N, K) ? ((size_t)((M + N) * row16(K)) + 255) / 256 * 256 : 0);
}

bool few8_ok(int64_t M, int64_t K, const void *w, int64_t ldw)
{
    return M >= 1 && K >= 1 && M * ((K + FEW_THREADS * 16 - 1) / (FEW_THREADS * 16)) <= FEW_PIECES &&
           (reinterpret_cast<uintptr_t>(w) & 15) == 0 && ldw % 16 == 0 && K % 16 == 0;
}

hipError_t launch_few8(const GemmArgs &a, int dt, int cus, hipStream_t s)
{
    return dt == FA_BF16 ? run_few<__bf16, __bf16>(a, cus, s) : run_few<float, float>(a, cus, s);
}

hipError_t launch_gemm8(const GemmArgs &a, int dt, void *ws, int cus, hipStream_t s)
{
    if (a.M == 0 || a.N == 0)
        return hipSuccess;
    return dt == FA_BF16 ? gemm8_of<__bf16>(a, ws, cus, s) : gemm8_of<float>(a, ws, cus, s);
}

bool grad8_ok(int64_t N, int64_t K, const void *w, int64_t ldw)
{
    // as direct_ok, for the rows of w along K
    return N >= 1 && direct_ok(w, ldw, K, false);
}

size_t grad8_workspace_bytes(int dt, int64_t M, int64_t N, int64_t K, int cus)
{
    const GradPlan p = grad_plan(M, K, N, dt == FA_BF16 ? 1 : 3, cus);
    return p.splits > 1 ? ((size_t)p.splits * M * K * sizeof(float) + 255) / 256 * 256 : 0;
}

hipError_t launch_grad8(const GemmArgs &a, int dt, int64_t plane, void *ws, int cus, Finish &f, hipStream_t s)
{
    if (a.M == 0 || a.N == 0)
        return hipSuccess;
    float *part = static_cast<float *>(ws);
    return dt == FA_BF16 ? run_grad<__bf16, 1>(a, plane, part, cus, f, s) : run_grad<float, 3>(a, plane, part, cus, f, s);
}

hipError_t launch_widen(const int8_t *w, int64_t ldw, int64_t rows, int64_t cols, void *out, int64_t ldo, hipStream_t s)
{
    return rows == 0 || cols == 0 ? hipSuccess : widen<__bf16>(w, ldw, rows, cols, static_cast<__bf16 *>(out), ldo, s);
}

hipError_t launch_copy8(const int8_t *w, int64_t ldw, int64_t rows, int64_t cols, int8_t *out, int64_t ldo, hipStream_t s)
{
    return rows == 0 || cols == 0 ? hipSuccess : widen<int8_t>(w, ldw, rows, cols, out, ldo, s);
}

} // namespace fa
