// The orthogonalised update: X = t / |t| (Frobenius), then for each step
//     G = X X^T,   H = b G + c G^2,   X <- a X + H X
// over the shorter side s of the matrix (a tall one has G = X^T X and X <- a X +
// X H).  The singular values of X go through the odd polynomials a v + b v^3 +
// c v^5 in turn while its singular vectors stay; with suitable coefficients
// all of them end near one.
//
// Two forms.  For s <= 64 the whole sequence is one polynomial P of the first
// Gram matrix, times X: the Gram matrix and P are formed in fp64 (the powers
// of G square its condition), and X is read twice.  More steps than a Gram matrix
// carries in fp64 go in groups, with X in fp64 between them.  Longer sides take matrix
// products of 16-bit floats: a value is held as hi + lo, two fp16 scaled by a
// power of two (22 bits or more), and a product is hi hi + hi lo + lo hi with fp32
// sums, as exact as one in fp32 at a third of the 16-bit rate (835 against 157
// TFLOP/s at the peak).  a X is added to the finished sum: taken into H's
// diagonal it would pass through every rounding of the sum, for three times the
// error.  After 5 steps of a 512 x 512 matrix of rank 64 and noise the relative error is
// 1.0e-6, where fp32 products give 2.1e-6; of 2048 x 2048 1.7e-6 and 2.8e-6.
//
// Steps may run on the Gram matrix alone, as for short sides: with Q = a + H
//     G <- Q G Q,   P <- Q P,   and X <- P X at the end of the group,
// all symmetric, so half the products.  Five steps of 14336 x 4096 take 17 products of
// s x s and two with X instead of 5 and 10: 2.1 times fewer operations.
// Errors of G grow by up to a^2 a step instead of being left behind with the old
// G: over five steps to 6e-6 of the result (noise) .. 7e-4 (2048 x 8192 of rank 1),
// against 1e-6 .. 1e-4 with a new Gram matrix each step.  So results in bf16, whose
// rounding is 1.7e-3 of the norm, take groups (until the growth passes GROWTH_MAX)
// where the matrix is long enough to gain; fp32 results take a Gram matrix each step.
#include "tiles.h"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace fa {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------ the argument t
// v = beta v + u; t = u + beta v (nesterov) or v; without a momentum t = u.
template <typename T, int W>
__device__ __forceinline__ void argument(const OrthoArgs &p, const T *u, float *v, bool update, int valid, float *t)
{
    load_n<T, W>(u, valid, t);
    if (!p.momentum)
        return;
    float m[W];
    load_n<float, W>(v, valid, m);
    if (update) {
#pragma unroll
        for (int i = 0; i < W; i++)
            m[i] = __builtin_fmaf(p.beta, m[i], t[i]);
        store_n<float, W>(v, valid, m);
    }
#pragma unroll
    for (int i = 0; i < W; i++)
        t[i] = p.nesterov ? __builtin_fmaf(p.beta, m[i], t[i]) : m[i];
}

template <typename T> __device__ __forceinline__ const T *update_at(const OrthoArgs &p, int64_t b, int64_t r, int64_t c)
{
    return static_cast<const T *>(p.x) + b * p.stride_x + r * p.ldx + c;
}

__device__ __forceinline__ float *momentum_at(const OrthoArgs &p, int64_t b, int64_t r, int64_t c)
{
    return p.momentum ? p.momentum + b * p.stride_m + r * p.ldm + c : nullptr;
}

// The result: o = rate v, or keep o + rate v where the call steps weights.
template <typename O, int W>
__device__ __forceinline__ void put_result(const OrthoArgs &p, int64_t b, int64_t r, int64_t c, int valid, const float *v)
{
    O *o = static_cast<O *>(p.out) + b * p.stride_o + r * p.ldo + c;
    float old[W], z[W];
    load_n<O, W>(o, p.add ? valid : 0, old);
#pragma unroll
    for (int i = 0; i < W; i++)
        z[i] = p.add ? __builtin_fmaf(p.rate, v[i], p.keep * old[i]) : p.rate * v[i];
    store_n<O, W>(o, valid, z);
}

// What short sides compute on: fp32 values, or the X of fp64 between two groups of
// steps, which is neither scaled nor added to anything.
template <typename T> struct value {
    typedef float type;
};
template <> struct value<double> {
    typedef double type;
};

template <typename T, int W>
__device__ __forceinline__ void values_at(const OrthoArgs &p, int64_t b, int64_t r, int64_t c, bool update, int valid,
                                          typename value<T>::type *t)
{
    if constexpr (__is_same(T, double)) {
        const double *x = update_at<double>(p, b, r, c);
        if (valid >= W) {
            __builtin_memcpy(t, x, W * sizeof(double));
        } else {
#pragma unroll
            for (int i = 0; i < W; i++)
                t[i] = i < valid ? x[i] : 0.0;
        }
    } else {
        argument<T, W>(p, update_at<T>(p, b, r, c), momentum_at(p, b, r, c), update, valid, t);
    }
}

template <typename O, int W>
__device__ __forceinline__ void put_values(const OrthoArgs &p, int64_t b, int64_t r, int64_t c, int valid,
                                           const typename value<O>::type *v)
{
    if constexpr (__is_same(O, double)) {
        double *o = static_cast<double *>(p.out) + b * p.stride_o + r * p.ldo + c;
#pragma unroll
        for (int i = 0; i < W; i++)
            if (i < valid)
                o[i] = v[i];
    } else {
        put_result<O, W>(p, b, r, c, valid, v);
    }
}

// Matrix and part of a workgroup.
__device__ __forceinline__ void matrix_of(int64_t id, int parts, int64_t &b, int &part)
{
    b = id / parts;
    part = (int)(id % parts);
}

// ------------------------------------------------------------ long sides: norm and first X
// Bound by memory.  A part is some rows of a matrix; `across` (a power of two)
// threads stand side by side on NORM_W columns each, and every thread has NORM_U
// such pieces on their way at a time.  14336 x 4096 bf16: the squares' sum in
// 45 us, the split into halves in 80 (352 MB moved).
constexpr int NORM_THREADS = 256, NORM_W = 8, NORM_U = 4, NORM_MAX_PARTS = 1024;

// Walks the pieces of rows [r0, r1), columns [0, cols): take(r, c, t) gets the
// argument's values at c .. c + NORM_W - 1, 0 where t has none.
template <typename T, typename F>
__device__ __forceinline__ void walk(const OrthoArgs &p, int64_t b, int64_t r0, int64_t r1, int64_t cols, int across, bool update,
                                     F take)
{
    const unsigned groups = NORM_THREADS / across, wide = (unsigned)((cols + across * NORM_W - 1) / (across * NORM_W));
    const unsigned all = (unsigned)(r1 - r0) * wide; // a part has at most 2^23 pieces
    const int64_t c0 = (int64_t)(threadIdx.x % across) * NORM_W;
    for (unsigned q0 = threadIdx.x / across; q0 < all; q0 += groups * NORM_U) {
        Raw<T, NORM_W> u[NORM_U];
        Raw<float, NORM_W> m[NORM_U];
        int64_t r[NORM_U], c[NORM_U];
        int valid[NORM_U];
#pragma unroll
        for (int e = 0; e < NORM_U; e++) {
            const unsigned q = q0 + e * groups;
            r[e] = q < all ? r0 + q / wide : r1;
            c[e] = (int64_t)(q % wide) * (across * NORM_W) + c0;
            valid[e] = (int)(r[e] >= r1 || r[e] >= p.m || c[e] >= p.n ? 0 : p.n - c[e] < NORM_W ? p.n - c[e] : NORM_W);
            u[e].fetch(update_at<T>(p, b, r[e], c[e]), valid[e]);
            if (p.momentum)
                m[e].fetch(momentum_at(p, b, r[e], c[e]), valid[e]);
        }
#pragma unroll
        for (int e = 0; e < NORM_U; e++) {
            if (r[e] >= r1)
                break;
            float t[NORM_W];
#pragma unroll
            for (int i = 0; i < NORM_W; i++) {
                t[i] = (float)u[e].e[i];
                if (p.momentum) {
                    if (update)
                        m[e].e[i] = __builtin_fmaf(p.beta, m[e].e[i], t[i]);
                    t[i] = p.nesterov ? __builtin_fmaf(p.beta, m[e].e[i], t[i]) : m[e].e[i];
                }
                t[i] = i < valid[e] ? t[i] : 0.f;
            }
            if (update && p.momentum)
                store_n<float, NORM_W>(momentum_at(p, b, r[e], c[e]), valid[e], m[e].e);
            take(r[e], c[e], t);
        }
    }
}

// The squares are summed in fp64, in an order fixed by the sizes.
template <typename T>
__global__ __launch_bounds__(NORM_THREADS) void norm_kernel(OrthoArgs p, int parts, int64_t rows_per, int across, double *sums)
{
    __shared__ double waves[NORM_THREADS / WAVE];
    int64_t b;
    int part;
    matrix_of(blockIdx.x, parts, b, part);
    const int64_t r0 = part * rows_per, r1 = r0 + rows_per < p.m ? r0 + rows_per : p.m;
    double sum = 0;
    walk<T>(p, b, r0, r1, p.n, across, true, [&](int64_t, int64_t, const float *t) {
#pragma unroll
        for (int i = 0; i < NORM_W; i++)
            sum += (double)t[i] * t[i];
    });
#pragma unroll
    for (int d = 1; d < WAVE; d *= 2)
        sum += __shfl_xor(sum, d);
    if (threadIdx.x % WAVE == 0)
        waves[threadIdx.x / WAVE] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        sums[b * parts + part] = waves[0] + waves[1] + waves[2] + waves[3];
}

// 1 / |t|; 0 for a matrix of zeros, NaN where the sum is NaN or infinite.
__device__ __forceinline__ double inverse_norm(double square)
{
    return square == 0 ? 0.0 : square < INFINITY ? 1.0 / sqrt(square) : __builtin_nan("");
}

__device__ __forceinline__ void split_value(float v, _Float16 &hi, _Float16 &lo)
{
    hi = (_Float16)v;
    lo = (_Float16)(v - (float)hi);
}

// A matrix of a batch as pairs: 32 columns' hi values are followed by their lo
// values, so that a step of one row is a whole cache line: the square of
// 4096 x 4096 in 176 us, 14336 x 4096 by 4096 x 4096 in 1.06 ms; as two matrices
// apart, whose steps are half lines, 213 us and 1.16 ms.
// `ld` columns a row, `stride` elements from one matrix to the next.  Rows and
// columns are followed by zeros up to a multiple of PAD, the longest step of k.
constexpr int PAD = STEP_BYTES / 2, PAIR = 32;

struct Planes {
    _Float16 *p;
    int64_t ld, stride;

    // hi of row r, column c and up, of 8; lo lies PAIR behind
    __device__ __forceinline__ _Float16 *at(int64_t b, int64_t r, int64_t c) const
    {
        return p + b * stride + r * 2 * ld + c + c / PAIR * PAIR;
    }
};

// X = t / |t| times `scale` as planes, with their zeros; also the zeros behind the
// rows of the second X, whose own rows each step writes whole.
template <typename T>
__global__ __launch_bounds__(NORM_THREADS) void split_kernel(OrthoArgs p, int parts, int64_t rows_per, int across,
                                                             const double *sums, float scale, Planes x, Planes y, int64_t rows)
{
    __shared__ double factor;
    int64_t b;
    int part;
    matrix_of(blockIdx.x, parts, b, part);
    if (threadIdx.x < WAVE) {
        double sum = 0;
#pragma unroll 4
        for (int i = threadIdx.x; i < parts; i += WAVE)
            sum += sums[b * parts + i];
#pragma unroll
        for (int d = 1; d < WAVE; d *= 2)
            sum += __shfl_xor(sum, d);
        if (threadIdx.x == 0)
            factor = inverse_norm(sum) * scale;
    }
    __syncthreads();
    const double f = factor;
    const int64_t r0 = part * rows_per, r1 = r0 + rows_per < p.m ? r0 + rows_per : p.m;
    walk<T>(p, b, r0, r1, x.ld, across, false, [&](int64_t r, int64_t c, const float *t) {
        if (c >= x.ld)
            return;
        f16x8 h, l;
#pragma unroll
        for (int i = 0; i < NORM_W; i++) {
            _Float16 hi, lw;
            split_value((float)(t[i] * f), hi, lw);
            // zeros stay zeros behind a row of a matrix whose norm is NaN
            h[i] = c + i < p.n ? hi : (_Float16)0;
            l[i] = c + i < p.n ? lw : (_Float16)0;
        }
        _Float16 *to = x.at(b, r, c);
        *reinterpret_cast<f16x8 *>(to) = h;
        *reinterpret_cast<f16x8 *>(to + PAIR) = l;
    });
    // the rows behind the matrix, of both X
    for (int64_t r = p.m + part; r < rows; r += parts)
        for (int64_t c = threadIdx.x * NORM_W; c < x.ld; c += NORM_THREADS * NORM_W)
            for (_Float16 *to : {x.at(b, r, c), x.at(b, r, c) + PAIR, y.at(b, r, c), y.at(b, r, c) + PAIR})
                *reinterpret_cast<f16x8 *>(to) = f16x8{};
}

// ------------------------------------------------------------ long sides: products
struct PairArgs {
    Planes a, b;
    int M, N, K;
    int tiles_m, tiles_n, tiles; // tiles of one matrix; symmetric: of the lower triangle
    // The first `whole` tiles of the batch are a workgroup's each, the `rest` are
    // split along k into `splits` of `per` steps, whose sums go to `part`.
    unsigned whole, rest, splits;
    int per;
    float *part;
    // v = q (sum) + p T + r U; T nullable, U too, and null without T
    float p, q, r;
    Planes t, u;
    Planes out; // out.p null: the result goes to o.out
    bool even;  // of a symmetric product: the diagonal's tiles are symmetric too
    OrthoArgs o;
};

// Consecutive workgroups go to the 8 XCDs in turn: each gets a contiguous run of
// the tiles, so that the rows which neighbours share stay in its own L2.
__device__ __forceinline__ unsigned xcd_order(unsigned id, unsigned total)
{
    const unsigned per = total / XCDS, rest = total % XCDS, x = id % XCDS;
    return x * per + (x < rest ? x : rest) + id / XCDS;
}

// Tile `id` of a matrix: bands of GROUP tile rows, or, of a symmetric product,
// the lower triangle row by row.
template <bool SYM>
__device__ __forceinline__ void pair_tile(unsigned id, unsigned tiles_m, unsigned tiles_n, unsigned &tm, unsigned &tn)
{
    if constexpr (SYM) {
        tm = (unsigned)((sqrtf(8.f * (float)id + 1.f) - 1.f) * 0.5f);
        while (tm * (tm + 1) / 2 > id)
            tm--;
        while ((tm + 1) * (tm + 2) / 2 <= id)
            tm++;
        tn = id - tm * (tm + 1) / 2;
    } else {
        const unsigned band = GROUP * tiles_n, first = id / band * GROUP;
        const unsigned high = tiles_m - first < GROUP ? tiles_m - first : GROUP;
        tm = first + id % band % high;
        tn = id % band / high;
    }
}

// EMIT neighbours of T and U, on their way while the sums are finished.
constexpr int EMIT = 8;

struct Addends {
    f16x8 th, tl, uh, ul;

    __device__ __forceinline__ void fetch(const PairArgs &p, int64_t b, int m, int n, bool any)
    {
        th = tl = uh = ul = f16x8{};
        const auto load = [&](const Planes &x, f16x8 &h, f16x8 &l) {
            const _Float16 *at = x.at(b, m, n);
            h = *reinterpret_cast<const f16x8 *>(at);
            l = *reinterpret_cast<const f16x8 *>(at + PAIR);
        };
        if (any && p.t.p)
            load(p.t, th, tl);
        if (any && p.u.p)
            load(p.u, uh, ul);
    }

    // v = q s + r U + p T
    __device__ __forceinline__ void finish(const PairArgs &p, float *v) const
    {
#pragma unroll
        for (int i = 0; i < EMIT; i++)
            v[i] = p.q * v[i];
        if (p.u.p)
#pragma unroll
            for (int i = 0; i < EMIT; i++)
                v[i] = __builtin_fmaf(p.r, (float)uh[i] + (float)ul[i], v[i]);
        if (p.t.p)
#pragma unroll
            for (int i = 0; i < EMIT; i++)
                v[i] = __builtin_fmaf(p.p, (float)th[i] + (float)tl[i], v[i]);
    }
};

// Stores EMIT neighbours of row m; n is a multiple of EMIT.
template <typename O>
__device__ __forceinline__ void emit(const PairArgs &p, int64_t b, int m, int n, const float *v)
{
    if (!p.out.p) {
        put_result<O, EMIT>(p.o, b, m, n, p.N - n < EMIT ? p.N - n : EMIT, v);
        return;
    }
    f16x8 h, l;
#pragma unroll
    for (int i = 0; i < EMIT; i++) {
        _Float16 hi, lw;
        split_value(v[i], hi, lw);
        h[i] = hi;
        l[i] = lw;
    }
    _Float16 *to = p.out.at(b, m, n);
    *reinterpret_cast<f16x8 *>(to) = h;
    *reinterpret_cast<f16x8 *>(to + PAIR) = l;
}

// Columns of a row that are written: planes also get the zeros behind the row.
__device__ __forceinline__ int64_t emit_columns(const PairArgs &p) { return p.out.p ? p.out.ld : p.N; }

// A workgroup's share: a tile of a matrix, whole or a split of it.
struct Share {
    int64_t b;
    unsigned tm, tn;
    int first, steps; // of k
    float *part;      // where a split's sums go
    // Of a symmetric product the lower side is written to the upper one too, where G is
    // carried through several steps also within the tiles of the diagonal: what it
    // differed by from its transpose, as the rounding of T Q does from that of Q T, would
    // grow with it (600 x 1000 of rank 2 in whole numbers, 5 steps: an error of 4e-3 of
    // the result, so 2e-4; T, H and K need not).
    bool mirror, diagonal;
};

template <bool SYM, int BM, int BN> __device__ __forceinline__ Share share_of(const PairArgs &p, int all)
{
    Share s{0, 0, 0, 0, all, nullptr, false, false};
    unsigned id;
    if (blockIdx.x < p.whole) {
        id = xcd_order(blockIdx.x, p.whole);
    } else {
        // splits of one range of k run together: they share what they read
        const unsigned at = xcd_order(blockIdx.x - p.whole, p.rest * p.splits), split = at / p.rest;
        id = p.whole + at % p.rest;
        if (p.splits > 1) {
            s.first = (int)split * p.per;
            s.steps = all - s.first < p.per ? all - s.first : p.per;
            s.part = p.part + ((int64_t)(id - p.whole) * p.splits + split) * (BM * BN);
        }
    }
    s.b = id / (unsigned)p.tiles;
    pair_tile<SYM>(id % (unsigned)p.tiles, p.tiles_m, p.tiles_n, s.tm, s.tn);
    s.diagonal = SYM && s.tm == s.tn && p.even;
    s.mirror = SYM && (s.tm != s.tn || p.even);
    return s;
}

// Rows i of the wavefronts' fragments, which lie in LDS at `o`, 16 of each row
// of wavefronts: whole rows are read and written.  A symmetric product's upper
// side is the finished values of the lower, read along the columns.
template <int BM, int BN, int WM, int WN> struct Rows {
    static constexpr int THREADS = WM * WN * WAVE, ROWS = WM * 16, CHUNKS = ROWS * BN / EMIT, PER = CHUNKS / THREADS;
    static_assert(CHUNKS % THREADS == 0, "every thread writes as much");
    Addends add[PER];

    static __device__ __forceinline__ int row(const Share &s, int i, int r)
    {
        return (int)s.tm * BM + r / 16 * (BM / WM) + i * 16 + r % 16;
    }

    __device__ __forceinline__ void fetch(const PairArgs &p, const Share &s, int i, int thread)
    {
        const int64_t cols = emit_columns(p);
#pragma unroll
        for (int e = 0; e < PER; e++) {
            const int at = thread + e * THREADS, m = row(s, i, at / (BN / EMIT)), n = (int)s.tn * BN + at % (BN / EMIT) * EMIT;
            add[e].fetch(p, s.b, m, n, m < p.M && n < cols);
        }
    }

    template <typename O>
    __device__ __forceinline__ void emit_all(const PairArgs &p, const Share &s, int i, float *o, int thread) const
    {
        const int64_t cols = emit_columns(p);
        const int n0 = (int)s.tn * BN;
#pragma unroll
        for (int e = 0; e < PER; e++) {
            const int at = thread + e * THREADS, r = at / (BN / EMIT), c = at % (BN / EMIT) * EMIT;
            const int m = row(s, i, r), n = n0 + c;
            float v[EMIT];
#pragma unroll
            for (int g = 0; g < EMIT; g += 4)
                __builtin_memcpy(v + g, o + write_tile_at<BN>(r, c + g), 16);
            add[e].finish(p, v);
            if (m < p.M && n < cols && !(s.diagonal && n + EMIT > m))
                emit<O>(p, s.b, m, n, v);
            if (s.mirror && p.t.p)
#pragma unroll
                for (int g = 0; g < EMIT; g += 4)
                    __builtin_memcpy(o + write_tile_at<BN>(r, c + g), v + g, 16);
        }
        if (s.mirror) {
            const float q = p.t.p ? 1.f : p.q; // without T and U the sums are still there
            if (p.t.p)
                __syncthreads();
#pragma unroll
            for (int e = 0; e < PER; e++) {
                const int at = thread + e * THREADS, c = at / (ROWS / EMIT), r = at % (ROWS / EMIT) * EMIT;
                const int n = n0 + c, m = row(s, i, r);
                if (n < p.N && m < cols && !(s.diagonal && m + EMIT <= n)) {
                    float v[EMIT];
#pragma unroll
                    for (int g = 0; g < EMIT; g++)
                        v[g] = q * o[write_tile_at<BN>(r + g, c & ~3) + (c & 3)];
                    // on the diagonal the row's own values up to it, which lie among these rows
                    if (s.diagonal && n > m)
#pragma unroll
                        for (int g = 0; g < EMIT; g++)
                            if (g < n - m)
                                v[g] = q * o[write_tile_at<BN>(r + n - m, (c - n + m + g) & ~3) + ((c - n + m + g) & 3)];
                    emit<O>(p, s.b, n, m, v);
                }
            }
        }
    }
};


template <int BN, int WN> __device__ __forceinline__ int fragment_at(int j, int thread)
{
    const int wave = thread / WAVE, lane = thread % WAVE;
    return write_tile_at<BN>((wave / WN) * 16 + (lane & 15), (wave % WN) * (BN / WN) + j * 16 + (lane >> 4) * 4);
}

// The finished tile, through LDS in two buffers that take turns; a split's sums
// go to memory as the threads hold them.
template <typename O, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void emit_tile(const PairArgs &p, const Share &s, const f32x4 (&acc)[BM / WM / 16][BN / WN / 16],
                                          char *b0, char *b1)
{
    constexpr int THREADS = WM * WN * WAVE, FM = BM / WM / 16, FN = BN / WN / 16;
    if (s.part) {
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < FN; j++)
                reinterpret_cast<f32x4 *>(s.part)[(i * FN + j) * THREADS + threadIdx.x] = acc[i][j];
        return;
    }
    Rows<BM, BN, WM, WN> rows[2];
    rows[0].fetch(p, s, 0, threadIdx.x);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < FM; i++) {
        float *o = reinterpret_cast<float *>(i & 1 ? b1 : b0);
        if (i + 1 < FM)
            rows[(i + 1) & 1].fetch(p, s, i + 1, threadIdx.x);
#pragma unroll
        for (int j = 0; j < FN; j++)
            *reinterpret_cast<f32x4 *>(o + fragment_at<BN, WN>(j, threadIdx.x)) = acc[i][j];
        __syncthreads();
        rows[i & 1].template emit_all<O>(p, s, i, o, threadIdx.x);
    }
}

// Joins the splits' sums in their order: workgroup (split tile, rows i of its
// fragments).
template <typename O, int BM, int BN, int WM, int WN, bool SYM>
__global__ __launch_bounds__(WM *WN *WAVE) void pair_join_kernel(PairArgs p)
{
    constexpr int THREADS = WM * WN * WAVE, FM = BM / WM / 16, FN = BN / WN / 16;
    __shared__ __attribute__((aligned(16))) float o[WM * 16 * BN];
    const unsigned tile = blockIdx.x / FM;
    const int i = blockIdx.x % FM;
    Share s{0, 0, 0, 0, 0, nullptr, false, false};
    s.b = (p.whole + tile) / (unsigned)p.tiles;
    pair_tile<SYM>((p.whole + tile) % (unsigned)p.tiles, p.tiles_m, p.tiles_n, s.tm, s.tn);
    s.diagonal = SYM && s.tm == s.tn && p.even;
    s.mirror = SYM && (s.tm != s.tn || p.even);
    const f32x4 *from = reinterpret_cast<const f32x4 *>(p.part + (int64_t)tile * p.splits * (BM * BN)) + i * FN * THREADS + threadIdx.x;
    Rows<BM, BN, WM, WN> rows;
    rows.fetch(p, s, i, threadIdx.x);
    f32x4 sum[FN];
#pragma unroll
    for (int j = 0; j < FN; j++)
        sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (unsigned z = 0; z < p.splits; z++)
#pragma unroll
        for (int j = 0; j < FN; j++)
            sum[j] += from[z * (BM * BN / 4) + j * THREADS];
#pragma unroll
    for (int j = 0; j < FN; j++)
        *reinterpret_cast<f32x4 *>(o + fragment_at<BN, WN>(j, threadIdx.x)) = sum[j];
    __syncthreads();
    rows.template emit_all<O>(p, s, i, o, threadIdx.x);
}

// A step's tile of one operand, hi and lo: STEP bytes of k of each.  An inner
// operand's rows of 128 bytes are PAIR values of k (a step of more has several
// such tiles), an outer one's rows are the 2 ROWS values of one k, as they lie in
// memory or (halves) hi before lo: a fragment's two addresses are then a constant
// apart, without which two outer operands need more registers than two workgroups
// a CU have (X^T X of 14336 x 4096: 601 us, with one workgroup 757).
// Matrices are padded with zeros, rows and columns, to whole steps, so only the
// tile's own edge is checked, once.
template <bool OUTER, int ROWS, int THREADS, int STEP> struct PairCopy {
    static constexpr int PARTS = OUTER ? 1 : STEP / 2 / PAIR, BYTES = 2 * ROWS * STEP / PARTS;
    typedef Direct<_Float16, OUTER, OUTER ? 2 * ROWS : ROWS, THREADS, OUTER ? STEP : 4 * PAIR> Copies;
    Copies d;

    // r0: the tile's first row, of `rows`; first: its first step
    __device__ __forceinline__ void init(const Planes &x, int64_t b, int r0, int rows, int first, bool halves)
    {
        d.init(x.p + b * x.stride, 2 * x.ld, OUTER ? 2 * r0 : r0, OUTER ? (int)(2 * x.ld) : rows, 0);
        d.base += first * (PARTS * d.advance);
        if (OUTER && halves)
            d.halves(2 * x.ld, r0, PAIR);
    }

    __device__ __forceinline__ void start(char *tile)
    {
        if constexpr (OUTER) {
            // rows that far apart have their chunks in the same order; past the last
            // column the sum stays out of range
            static_assert(2 * THREADS / Copies::CPR % 16 == 0 || Copies::CH <= 2, "two offsets are enough");
            d.start_apart(tile, (uint32_t)(d.advance / Copies::BK) * (2 * THREADS / Copies::CPR));
        } else {
#pragma unroll
            for (int q = 0; q < PARTS; q++)
                d.start_at(tile + q * BYTES, q * d.advance, Copies::BK);
        }
        d.base += PARTS * d.advance;
    }

    // Fragment of the rows from r0 at the 32 values kk of the step's k; lo: 0 or 1
    static __device__ __forceinline__ Frag read(const char *tile, int r0, int kk, int lo, int lane, bool halves)
    {
        if constexpr (OUTER)
            return read_frag<_Float16, true, 2 * ROWS, STEP>(tile, halves ? lo * ROWS + r0 : r0 + r0 / PAIR * PAIR + lo * PAIR, kk, lane);
        else
            return read_frag<_Float16, false, ROWS, 4 * PAIR>(tile + kk * BYTES, r0, lo, lane);
    }
};

// acc += the three products of one pair of fragments.
__device__ __forceinline__ f32x4 mma_pair(const Frag &bh, const Frag &bl, const Frag &ah, const Frag &al, f32x4 acc)
{
    acc = mma<_Float16>(bl, ah, acc);
    acc = mma<_Float16>(bh, al, acc);
    return mma<_Float16>(bh, ah, acc);
}

// Small products: 64 x 64 tiles, steps of 128 bytes of k.  Two groups of four
// wavefronts take half a step's k each, since one wavefront a SIMD leaves the
// matrix cores idle while it reads LDS; their sums are joined at the end.  With
// a tile a CU or fewer a step waits for memory, and four buffers (DEEP) let three
// steps be on their way; with more tiles two workgroups a CU, with two buffers
// each, hide it.  All of a 1000 x 1000 call's 15 products: 252 us with one group
// and two buffers, 226 with four, 202 with two groups and four; XX^T of 1000 x 1000
// alone 12 us.
template <typename O, bool AO, bool BO, bool SYM, bool DEEP>
__global__ __launch_bounds__(512) void pair_kernel(PairArgs p)
{
    constexpr int BM = 64, WM = 2, WN = 2, GROUP_THREADS = WM * WN * WAVE, THREADS = 2 * GROUP_THREADS;
    constexpr int BK = STEP_BYTES / 2, F = 2;
    constexpr int AB = BM * STEP_BYTES; // one plane of one operand
    constexpr int COPIES = 4 * AB / 16 / THREADS; // per thread and step
    __shared__ __attribute__((aligned(1024))) char l0[4 * AB];
    __shared__ __attribute__((aligned(1024))) char l1[4 * AB];
    __shared__ __attribute__((aligned(1024))) char l2[DEEP ? 4 * AB : 16];
    __shared__ __attribute__((aligned(1024))) char l3[DEEP ? 4 * AB : 16];
    const Share sh = share_of<SYM, BM, BM>(p, (p.K + BK - 1) / BK);
    const int m0 = (int)sh.tm * BM, n0 = (int)sh.tn * BM, steps = sh.steps;
    const int group = threadIdx.x / GROUP_THREADS, thread = threadIdx.x % GROUP_THREADS;
    const int wave = thread / WAVE, lane = thread % WAVE;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BM / WN);
    f32x4 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; i++)
#pragma unroll
        for (int j = 0; j < F; j++)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    PairCopy<AO, BM, THREADS, STEP_BYTES> a;
    PairCopy<BO, BM, THREADS, STEP_BYTES> b;
    a.init(p.a, sh.b, m0, p.M, sh.first, AO && BO);
    b.init(p.b, sh.b, n0, p.N, sh.first, AO && BO);
    const auto copy = [&](char *l) {
        a.start(l);
        b.start(l + 2 * AB);
    };
    const auto step = [&](const char *l) {
        Frag ah[F], al[F], bh[F], bl[F];
#pragma unroll
        for (int i = 0; i < F; i++) {
            ah[i] = a.read(l, wm + i * 16, group, 0, lane, AO && BO);
            al[i] = a.read(l, wm + i * 16, group, 1, lane, AO && BO);
            bh[i] = b.read(l + 2 * AB, wn + i * 16, group, 0, lane, AO && BO);
            bl[i] = b.read(l + 2 * AB, wn + i * 16, group, 1, lane, AO && BO);
        }
#pragma unroll
        for (int i = 0; i < F; i++)
#pragma unroll
            for (int j = 0; j < F; j++)
                acc[i][j] = mma_pair(bh[j], bl[j], ah[i], al[i], acc[i][j]);
    };
    if constexpr (DEEP) {
        // step t from `cur`; `free` held step t - 1 and takes step t + 3
        const auto turn = [&](const char *cur, char *free, int t) {
            if (t + 2 < steps)
                copies_done<2 * COPIES, true>();
            else if (t + 1 < steps)
                copies_done<COPIES, true>();
            else
                copies_done<0, true>();
            if (t + 3 < steps)
                copy(free);
            step(cur);
        };
        copy(l0);
        if (steps > 1)
            copy(l1);
        if (steps > 2)
            copy(l2);
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
        copy(l0);
        int s = 0;
        for (; s + 1 < steps; s += 2) {
            copies_done<0, true>();
            copy(l1);
            step(l0);
            copies_done<0, true>();
            if (s + 2 < steps)
                copy(l0);
            step(l1);
        }
        copies_done<0, true>();
        if (s < steps)
            step(l0);
    }
    Rows<BM, BM, WM, WN> rows;
    if (!sh.part)
        rows.fetch(p, sh, group, thread);
    // the second group's sums of fragments i = 0 go to the first, the first's of
    // i = 1 to the second, and each finishes its own
    __syncthreads();
    f32x4 *give = reinterpret_cast<f32x4 *>(l0), mine[F];
#pragma unroll
    for (int j = 0; j < F; j++)
        give[(group * F + j) * GROUP_THREADS + thread] = group == 0 ? acc[1][j] : acc[0][j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < F; j++) {
        const f32x4 other = give[((group ^ 1) * F + j) * GROUP_THREADS + thread];
        mine[j] = (group == 0 ? acc[0][j] : acc[1][j]) + other;
    }
    if (sh.part) {
#pragma unroll
        for (int j = 0; j < F; j++)
            reinterpret_cast<f32x4 *>(sh.part)[(group * F + j) * GROUP_THREADS + thread] = mine[j];
        return;
    }
    float *o = reinterpret_cast<float *>(l1 + group * 2 * AB);
#pragma unroll
    for (int j = 0; j < F; j++)
        *reinterpret_cast<f32x4 *>(o + fragment_at<BM, WN>(j, thread)) = mine[j];
    __syncthreads();
    rows.template emit_all<O>(p, sh, group, o, thread);
}

// Larger products, bound by the matrix cores: steps of 64 bytes of k in BUFS
// buffers.  A step is walked by rows of fragments of A.  Row i + 3's are read
// from LDS while row i's products run; two rows before the step's end all its
// reads are done, so after a barrier the copies of step t + BUFS take its buffer,
// and the next step's first fragments are read behind those two rows.  Two
// 128 x 128 tiles share a CU with two buffers each; one alone takes four, since
// its step is shorter than the way from memory: XX^T of 2048 x 2048, half of its
// tiles, 44 us with four buffers and 51 with two, 52 with four wavefronts of
// 64 x 64 instead of eight.  14336 x 4096 by 4096 x 4096 in 256 x 256 tiles takes
// 1.06 ms, 1.36 PFLOP/s over the three products.
constexpr int PAIR_SLOTS = 4;

// Tiles that share a CU have half of its registers each.
template <typename O, int BM, int BN, int WM, int WN, bool AO, bool BO, bool SYM, int BUFS>
__global__ __launch_bounds__(WM *WN *WAVE, BM * BN * BUFS <= 2 * 128 * 128 ? 4 : 2) void pair_pipe_kernel(PairArgs p)
{
    constexpr int THREADS = WM * WN * WAVE, BK = PIPE_STEP / 2, STEP = PIPE_STEP;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    constexpr int AB = BM * STEP, BB = BN * STEP; // one plane of each operand
    static_assert(FM % PAIR_SLOTS == 0, "a row keeps its registers from step to step");
    __shared__ __attribute__((aligned(1024))) char l0[2 * (AB + BB)];
    __shared__ __attribute__((aligned(1024))) char l1[2 * (AB + BB)];
    __shared__ __attribute__((aligned(1024))) char l2[BUFS == 4 ? 2 * (AB + BB) : 16];
    __shared__ __attribute__((aligned(1024))) char l3[BUFS == 4 ? 2 * (AB + BB) : 16];
    constexpr int COPIES = 2 * (AB + BB) / 16 / THREADS; // per thread and step
    static_assert(BUFS == 2 || BUFS == 4, "the buffers above");
    const Share sh = share_of<SYM, BM, BN>(p, (p.K + BK - 1) / BK);
    const int m0 = (int)sh.tm * BM, n0 = (int)sh.tn * BN, steps = sh.steps;
    const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE;
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);
    PairCopy<AO, BM, THREADS, STEP> a;
    PairCopy<BO, BN, THREADS, STEP> b;
    a.init(p.a, sh.b, m0, p.M, sh.first, AO && BO);
    b.init(p.b, sh.b, n0, p.N, sh.first, AO && BO);
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    Frag ah[PAIR_SLOTS], al[PAIR_SLOTS], bh[2][FN], bl[2][FN];
    const auto copy = [&](char *l) {
        a.start(l);
        b.start(l + 2 * AB);
    };
    const auto read_a = [&](const char *l, int i) {
        ah[i % PAIR_SLOTS] = a.read(l, wm + i * 16, 0, 0, lane, AO && BO);
        al[i % PAIR_SLOTS] = a.read(l, wm + i * 16, 0, 1, lane, AO && BO);
    };
    const auto read_b = [&](const char *l, int s) {
#pragma unroll
        for (int j = 0; j < FN; j++) {
            bh[s][j] = b.read(l + 2 * AB, wn + j * 16, 0, 0, lane, AO && BO);
            bl[s][j] = b.read(l + 2 * AB, wn + j * 16, 0, 1, lane, AO && BO);
        }
    };
    // step t; inner: steps t + 1 .. t + BUFS are there
    const auto step = [&](char *cur, const char *next, int s, int t, bool inner) {
#pragma unroll
        for (int i = 0; i < FM; i++) {
            if (i == FM - 2) {
                if (inner || t + BUFS - 1 < steps)
                    copies_done<(BUFS - 2) * COPIES, true>();
                else
                    copies_done<0, true>();
                __builtin_amdgcn_sched_barrier(0);
                if (inner || t + BUFS < steps)
                    copy(cur);
                if (inner || t + 1 < steps)
                    read_b(next, s ^ 1);
            }
            if (i < FM - 3) {
                read_a(cur, i + 3);
            } else if (i >= FM - 2 && (inner || t + 1 < steps)) {
                if (i == FM - 2) {
                    read_a(next, 0);
                } else {
                    read_a(next, 1);
                    read_a(next, 2);
                }
            }
#pragma unroll
            for (int j = 0; j < FN; j++)
                acc[i][j] = mma_pair(bh[s][j], bl[s][j], ah[i % PAIR_SLOTS], al[i % PAIR_SLOTS], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    copy(l0);
    if (steps > 1)
        copy(l1);
    if constexpr (BUFS == 4) {
        if (steps > 2)
            copy(l2);
        if (steps > 3)
            copy(l3);
    }
    if (steps >= BUFS)
        copies_done<(BUFS - 1) * COPIES, true>();
    else
        copies_done<0, true>();
    read_b(l0, 0);
    read_a(l0, 0);
    read_a(l0, 1);
    read_a(l0, 2);
    int t = 0;
    if constexpr (BUFS == 4) {
        for (; t + 2 * BUFS - 1 < steps; t += BUFS) {
            step(l0, l1, 0, t, true);
            step(l1, l2, 1, t + 1, true);
            step(l2, l3, 0, t + 2, true);
            step(l3, l0, 1, t + 3, true);
        }
        for (; t < steps; t += BUFS) {
            step(l0, l1, 0, t, false);
            if (t + 1 < steps)
                step(l1, l2, 1, t + 1, false);
            if (t + 2 < steps)
                step(l2, l3, 0, t + 2, false);
            if (t + 3 < steps)
                step(l3, l0, 1, t + 3, false);
        }
    } else {
        for (; t + 2 * BUFS - 1 < steps; t += BUFS) {
            step(l0, l1, 0, t, true);
            step(l1, l0, 1, t + 1, true);
        }
        for (; t < steps; t += BUFS) {
            step(l0, l1, 0, t, false);
            if (t + 1 < steps)
                step(l1, l0, 1, t + 1, false);
        }
    }
    emit_tile<O, BM, BN, WM, WN>(p, sh, acc, l0, l1);
}

// ------------------------------------------------------------ short sides, in fp64
// Three stages: the Gram matrix G, its polynomial P, the product with X.  A
// workgroup has a part of the long side; with s <= 32 a call whose matrices have one
// part each runs all three in one launch.  Else G's parts go through memory, and
// for s <= 32, where that is cheap, every workgroup of the last stage forms P.
// 128 matrices of 16 x 4096 fp32 (67 MB): 12 us for the Gram matrices, 24 for P and
// the product.  One of 64 x 1000: 111 us in one launch, 68 in three; P of 64 x 64 by
// itself, 15 products one after another on one CU, takes 51 us with 8 wavefronts and
// 40 with 16.
constexpr int SHORT_MAX = 64, SHORT_THREADS = 512, SHORT_WAVES = SHORT_THREADS / WAVE, SHORT_STEP = 64;
constexpr int64_t SHORT_ALONE = 256;
enum { STAGE_GRAM = 1, STAGE_POLY = 2, STAGE_APPLY = 4 };

// Fragments of the matrix cores' 16x16x4 product in fp64: lane l holds row
// l % 16 of the one operand and column l % 16 of the other, both at k = l / 16,
// and of the result column l % 16, rows l / 16 + 4 r.
__device__ __forceinline__ f64x4 mma64(double a, double b, f64x4 c)
{
    return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}

// A symmetric matrix as its blocks of 16 x 16 on and below the diagonal, row by
// row; rows are spread over the banks.
constexpr int blocks_of(int t) { return t * (t + 1) / 2; }
typedef double Block[16][18];

__device__ __forceinline__ void block_at(int e, int &r, int &c)
{
    r = (e >= 1) + (e >= 3) + (e >= 6);
    c = e - r * (r + 1) / 2;
}

// Element (16 r + i, 16 c + k).
__device__ __forceinline__ double symmetric_at(const Block *m, int r, int i, int c, int k)
{
    return c <= r ? m[r * (r + 1) / 2 + c][i][k] : m[c * (c + 1) / 2 + r][k][i];
}

// Four values of short row i at k .. k + 3 of the long side, 0 where there are none.
template <typename T, bool WIDE>
__device__ __forceinline__ void short_values(const OrthoArgs &p, int64_t b, int i, int64_t k, int64_t s, int64_t l,
                                             typename value<T>::type *t)
{
    const int valid = (int)(i >= s || k >= l ? 0 : l - k < 4 ? l - k : 4);
    if constexpr (WIDE) {
        values_at<T, 4>(p, b, i, k, true, valid, t);
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
            values_at<T, 1>(p, b, k + j, i, true, j < valid, t + j);
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
        t[j] = j < valid ? t[j] : 0;
}

// G of the columns (rows) [k0, k1) of the long side into `to`, with `scratch` of
// SHORT_WAVES * 256 doubles.
template <typename T, int SB, bool WIDE, typename PUT>
__device__ __forceinline__ void short_gram(const OrthoArgs &p, int64_t b, int64_t k0, int64_t k1, double *scratch, PUT put)
{
    constexpr int NB = blocks_of(SB), U = SB <= 2 ? 4 : 2;
    const int64_t s = WIDE ? p.m : p.n;
    const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE, i = lane & 15, g = lane >> 4;
    f64x4 acc[NB];
#pragma unroll
    for (int e = 0; e < NB; e++)
        acc[e] = f64x4{0, 0, 0, 0};
    // 16 of the long side a wavefront, U such pieces on their way
    for (int64_t k = k0 + wave * 16; k < k1; k += SHORT_WAVES * 16 * U) {
        typename value<T>::type t[U][SB][4];
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int r = 0; r < SB; r++)
                short_values<T, WIDE>(p, b, r * 16 + i, k + u * SHORT_WAVES * 16 + g * 4, s, k1, t[u][r]);
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (u > 0 && k + u * SHORT_WAVES * 16 >= k1)
                break;
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int r = 0; r < SB; r++)
#pragma unroll
                    for (int c = 0; c <= r; c++)
                        acc[r * (r + 1) / 2 + c] = mma64(t[u][r][j], t[u][c][j], acc[r * (r + 1) / 2 + c]);
        }
    }
#pragma unroll
    for (int e = 0; e < NB; e++) {
        __syncthreads();
#pragma unroll
        for (int z = 0; z < 4; z++)
            scratch[wave * 256 + (g + 4 * z) * 16 + i] = acc[e][z];
        __syncthreads();
        if (threadIdx.x < 256) {
            double sum = scratch[threadIdx.x];
#pragma unroll
            for (int w = 1; w < SHORT_WAVES; w++)
                sum += scratch[w * 256 + threadIdx.x];
            put(e, (int)threadIdx.x, sum);
        }
    }
}

// Block e of A B for symmetric A and B that commute: its four values of a lane.
template <int SB> __device__ __forceinline__ f64x4 block_product(const Block *a, const Block *b, int e, int s)
{
    const int lane = threadIdx.x % WAVE, i = lane & 15, g = lane >> 4;
    int r, c;
    block_at(e, r, c);
    // all fragments first: the products then wait for LDS once.  Blocks above the
    // diagonal are read across; e is the same for a wavefront.
    double av[SB * 4], bv[SB * 4];
    const auto fetch = [&](const Block *m, int row, double *v) {
#pragma unroll
        for (int kb = 0; kb < SB; kb++) {
            if (kb <= row) {
                const double *at = &m[row * (row + 1) / 2 + kb][i][g];
#pragma unroll
                for (int q = 0; q < 4; q++)
                    v[kb * 4 + q] = at[q * 4];
            } else {
                const double *at = &m[kb * (kb + 1) / 2 + row][g][i];
#pragma unroll
                for (int q = 0; q < 4; q++)
                    v[kb * 4 + q] = at[q * 4 * 18];
            }
        }
    };
    fetch(a, r, av);
    fetch(b, c, bv);
    f64x4 acc = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < SB * 4; k++)
        if (k * 4 < s)
            acc = mma64(av[k], bv[k], acc);
    return acc;
}

// P from G, both in m: m[0] holds G at the start, the result is the index of P.
// Q = a + b G + c G^2; P <- Q P; G <- (Q G) Q.  Per step three rounds of block
// products, independent within a round.
template <int SB, int THREADS>
__device__ __forceinline__ int short_poly(const OrthoArgs &p, Block (*m)[blocks_of(SB)], double *norm)
{
    constexpr int NB = blocks_of(SB), WAVES = THREADS / WAVE;
    const int s = (int)(p.m < p.n ? p.m : p.n);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE), lane = threadIdx.x % WAVE, i = lane & 15, g = lane >> 4;
    __syncthreads();
    if (threadIdx.x < WAVE) {
        double t = (int)threadIdx.x < s ? m[0][blocks_of((threadIdx.x >> 4) % SB + 1) - 1][threadIdx.x & 15][threadIdx.x & 15] : 0.0;
#pragma unroll
        for (int d = 1; d < WAVE; d *= 2)
            t += __shfl_xor(t, d);
        if (threadIdx.x == 0)
            *norm = p.unit ? 1.0 : inverse_norm(t);
    }
    __syncthreads();
    const double f = *norm;
    for (int e = threadIdx.x; e < NB * 256; e += THREADS)
        m[0][e / 256][e / 16 % 16][e % 16] *= f * f;
    constexpr int G = 0, Q = 1, T = 2;
    int P = 3, N = 4;
    const auto put = [&](Block *to, int e, auto value) {
#pragma unroll
        for (int z = 0; z < 4; z++)
            to[e][g + 4 * z][i] = value(z);
    };
    for (int k = 0; k < p.steps; k++) {
        const double ca = p.coef[k][0], cb = p.coef[k][1], cc = p.coef[k][2];
        const bool last = k + 1 == p.steps;
        __syncthreads();
        for (int e = wave; e < NB; e += WAVES) {
            const f64x4 v = block_product<SB>(m[G], m[G], e, s);
            int r, c;
            block_at(e, r, c);
            const auto q = [&](int z) { return cc * v[z] + cb * m[G][e][g + 4 * z][i] + (r == c && g + 4 * z == i ? ca : 0.0); };
            put(m[Q], e, q);
            if (k == 0) // P was the norm's inverse
                put(m[P], e, [&](int z) { return f * q(z); });
        }
        __syncthreads();
        for (int e = wave + (k == 0 ? NB : 0); e < (last ? NB : 2 * NB); e += WAVES) {
            const bool first = e < NB;
            const f64x4 v = block_product<SB>(m[Q], first ? m[P] : m[G], first ? e : e - NB, s);
            put(first ? m[N] : m[T], first ? e : e - NB, [&](int z) { return v[z]; });
        }
        if (k > 0) {
            const int swap = P;
            P = N;
            N = swap;
        }
        if (last)
            break;
        __syncthreads();
        for (int e = wave; e < NB; e += WAVES) {
            const f64x4 v = block_product<SB>(m[T], m[Q], e, s);
            int r, c;
            block_at(e, r, c);
            // The diagonal's blocks get their lower side twice: what G differed by from its
            // transpose would grow with it (64 x 1000 of rank 3, 8 steps: an error of 1e-6,
            // so 2e-11; the others need not).  What is left out goes to the padding, without
            // a branch of single lanes.
#pragma unroll
            for (int z = 0; z < 4; z++) {
                const int row = g + 4 * z;
                m[G][e][row][r == c && row < i ? 16 : i] = v[z];
                m[G][e][r == c ? i : row][r == c && row > i ? row : 16] = v[z];
            }
        }
    }
    __syncthreads();
    return P;
}

// P X (wide) or X P (tall) for the columns (rows) [k0, k1) of the long side, a piece
// of SHORT_STEP columns or 16 rows a wavefront.
template <typename T, typename O, int SB, bool WIDE>
__device__ __forceinline__ void short_apply(const OrthoArgs &p, int64_t b, int64_t k0, int64_t k1, const Block *P)
{
    const int64_t s = WIDE ? p.m : p.n;
    const int wave = threadIdx.x / WAVE, lane = threadIdx.x % WAVE, i = lane & 15, g = lane >> 4;
    if constexpr (WIDE) {
        // Where there are fewer pieces than wavefronts, SB of these share a piece,
        // 16 rows of the result each; X is then read before any of it is written,
        // as the result may lie in its place.
        const int64_t pieces = (k1 - k0 + SHORT_STEP - 1) / SHORT_STEP;
        const bool shared = SB > 1 && pieces < SHORT_WAVES;
        constexpr int SHARES = SHORT_WAVES / SB;
        const int first = shared ? wave / SB : wave, stride = shared ? SHARES : SHORT_WAVES;
        for (int64_t q0 = 0; q0 < pieces; q0 += stride) {
            const int64_t piece = q0 + first;
            const bool mine = first < stride && piece < pieces;
            // t[r][j][q]: short index 16 r + 4 g + j at long index at + q
            const int64_t at = k0 + piece * SHORT_STEP + 4 * i;
            const int valid = (int)(!mine || at >= k1 ? 0 : k1 - at < 4 ? k1 - at : 4);
            typename value<T>::type t[SB][4][4];
#pragma unroll
            for (int r = 0; r < SB; r++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int row = r * 16 + g * 4 + j, n = row < s ? valid : 0;
                    values_at<T, 4>(p, b, row, at, false, n, t[r][j]);
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        t[r][j][q] = q < n ? t[r][j][q] : 0;
                }
            if (shared)
                __syncthreads();
            const int c0 = shared ? wave % SB : 0, c1 = !mine ? 0 : shared ? c0 + 1 : SB;
#pragma unroll 1 // unrolled, the fragments of P of all c are held at once
            for (int c = c0; c < c1; c++) {
                f64x4 acc[4];
#pragma unroll
                for (int q = 0; q < 4; q++)
                    acc[q] = f64x4{0, 0, 0, 0};
#pragma unroll
                for (int r = 0; r < SB; r++)
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const double w = symmetric_at(P, c, i, r, g * 4 + j);
#pragma unroll
                        for (int q = 0; q < 4; q++)
                            acc[q] = mma64(w, t[r][j][q], acc[q]);
                    }
#pragma unroll
                for (int z = 0; z < 4; z++) {
                    typedef typename value<O>::type V;
                    const V v[4] = {(V)acc[0][z], (V)acc[1][z], (V)acc[2][z], (V)acc[3][z]};
                    const int row = c * 16 + g + 4 * z;
                    if (row < s)
                        put_values<O, 4>(p, b, row, at, valid, v);
                }
            }
        }
    } else {
        for (int64_t k = k0 + wave * 16; k < k1; k += SHORT_WAVES * 16 * 4) {
            // t[u][r][j]: long index k + 128 (u0 + u) + i at short index 16 r + 4 g + j
            constexpr int U = SB <= 2 ? 4 : 2;
#pragma unroll 1
            for (int u0 = 0; u0 < 4; u0 += U) {
                if (k + u0 * SHORT_WAVES * 16 >= k1)
                    break;
                typename value<T>::type t[U][SB][4];
#pragma unroll
                for (int u = 0; u < U; u++)
#pragma unroll
                    for (int r = 0; r < SB; r++) {
                        const int64_t at = k + (u0 + u) * SHORT_WAVES * 16 + i, first = r * 16 + g * 4;
                        const int n = (int)(at >= k1 || first >= s ? 0 : s - first < 4 ? s - first : 4);
                        values_at<T, 4>(p, b, at, first, false, n, t[u][r]);
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            t[u][r][j] = j < n ? t[u][r][j] : 0;
                    }
                // lane i gives short indices SB i .. SB i + SB - 1
                const int col = SB * i, valid = (int)(col >= s ? 0 : s - col < SB ? s - col : SB);
                f64x4 acc[U][SB];
#pragma unroll
                for (int u = 0; u < U; u++)
#pragma unroll
                    for (int c = 0; c < SB; c++)
                        acc[u][c] = f64x4{0, 0, 0, 0};
#pragma unroll
                for (int r = 0; r < SB; r++)
#pragma unroll
                    for (int j = 0; j < 4; j++)
#pragma unroll
                        for (int c = 0; c < SB; c++) {
                            const double w = symmetric_at(P, (col + c) >> 4, (col + c) & 15, r, g * 4 + j);
#pragma unroll
                            for (int u = 0; u < U; u++)
                                acc[u][c] = mma64(t[u][r][j], w, acc[u][c]);
                        }
#pragma unroll
                for (int u = 0; u < U; u++)
#pragma unroll
                    for (int z = 0; z < 4; z++) {
                        typename value<O>::type v[SB];
#pragma unroll
                        for (int c = 0; c < SB; c++)
                            v[c] = (typename value<O>::type)acc[u][c][z];
                        const int64_t row = k + (u0 + u) * SHORT_WAVES * 16 + g + 4 * z;
                        if (row < k1 && valid > 0)
                            put_values<O, SB>(p, b, row, col, valid, v);
                    }
            }
        }
    }
}

// P alone runs on more wavefronts: four a SIMD hide each other's reads of LDS.
template <int STAGES> constexpr int short_threads() { return STAGES == STAGE_POLY ? 1024 : SHORT_THREADS; }

// Workgroup (matrix, part of the long side).  `part` [matrix][parts][block][256]
// holds G's parts, `poly` [matrix][block] P between the stages' launches.
template <typename T, typename O, int SB, bool WIDE, int STAGES>
__global__ __launch_bounds__(short_threads<STAGES>()) void short_kernel(OrthoArgs p, int parts, int64_t per, int sums, double *part,
                                                                        Block *poly)
{
    constexpr int NB = blocks_of(SB), MATRICES = STAGES & STAGE_POLY ? 5 : 1, THREADS = short_threads<STAGES>();
    constexpr bool GRAM = STAGES & STAGE_GRAM, POLY = STAGES & STAGE_POLY, APPLY = STAGES & STAGE_APPLY;
    constexpr int GROUPS = THREADS / 256;
    __shared__ __attribute__((aligned(16))) Block m[MATRICES][NB];
    __shared__ double scratch[GRAM ? SHORT_WAVES * 256 : POLY ? THREADS : 1];
    __shared__ double norm;
    int64_t b = blockIdx.x;
    int q = 0;
    if (GRAM || APPLY)
        matrix_of(blockIdx.x, parts, b, q);
    const int64_t l = WIDE ? p.n : p.m, k0 = q * per, k1 = k0 + per < l ? k0 + per : l;
    if constexpr (GRAM) {
        double *to = part + (b * parts + q) * (NB * 256);
        short_gram<T, SB, WIDE>(p, b, k0, k1, scratch, [&](int e, int at, double v) {
            if constexpr (POLY)
                m[0][e][at / 16][at % 16] = v;
            else
                to[e * 256 + at] = v;
        });
    } else if constexpr (POLY) {
        // groups of 256 threads take the parts in turn
        const double *from = part + b * sums * (NB * 256);
        const int at = threadIdx.x % 256, group = threadIdx.x / 256;
        for (int e = 0; e < NB; e++) {
            double sum = 0;
#pragma unroll 8
            for (int z = group; z < sums; z += GROUPS)
                sum += from[(int64_t)z * (NB * 256) + e * 256 + at];
            __syncthreads();
            scratch[threadIdx.x] = sum;
            __syncthreads();
            if (group == 0) {
#pragma unroll
                for (int z = 1; z < GROUPS; z++)
                    sum += scratch[z * 256 + at];
                m[0][e][at / 16][at % 16] = sum;
            }
        }
    }
    int P = 0;
    if constexpr (POLY)
        P = short_poly<SB, THREADS>(p, m, &norm);
    double *flat = reinterpret_cast<double *>(poly + b * NB);
    constexpr int SIZE = sizeof(Block) / sizeof(double) * NB;
    if constexpr (POLY && !APPLY)
        for (int e = threadIdx.x; e < SIZE; e += THREADS)
            flat[e] = reinterpret_cast<const double *>(m[P])[e];
    if constexpr (APPLY && !POLY) {
        for (int e = threadIdx.x; e < SIZE; e += THREADS)
            reinterpret_cast<double *>(m[0])[e] = flat[e];
        __syncthreads();
    }
    if constexpr (APPLY)
        short_apply<T, O, SB, WIDE>(p, b, k0, k1, m[P]);
}

// t in fp64 into p.out, of calls whose steps go in groups; the momentum is stepped.
template <typename T> __global__ __launch_bounds__(256) void short_lift_kernel(OrthoArgs p)
{
    const int64_t wide = (p.n + 3) / 4, all = p.B * p.m * wide;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < all; at += (int64_t)gridDim.x * 256) {
        const int64_t b = at / wide / p.m, r = at / wide % p.m, c = at % wide * 4;
        const int valid = (int)(p.n - c < 4 ? p.n - c : 4);
        float t[4];
        values_at<T, 4>(p, b, r, c, true, valid, t);
        const double v[4] = {t[0], t[1], t[2], t[3]};
        put_values<double, 4>(p, b, r, c, valid, v);
    }
}

// Sums of up to JOIN_PARTS of G's parts, for calls with many.
constexpr int JOIN_PARTS = 32;

__global__ __launch_bounds__(256) void short_join_kernel(const double *part, int parts, int sums, int blocks, double *out)
{
    const int e = blockIdx.x % blocks;
    const int64_t q = blockIdx.x / blocks % sums, b = blockIdx.x / blocks / sums;
    const int first = (int)q * JOIN_PARTS, end = first + JOIN_PARTS < parts ? first + JOIN_PARTS : parts;
    double sum = 0;
#pragma unroll 8
    for (int z = first; z < end; z++)
        sum += part[((b * parts + z) * blocks + e) * 256 + threadIdx.x];
    out[((b * sums + q) * blocks + e) * 256 + threadIdx.x] = sum;
}

// ------------------------------------------------------------ launches

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// What the steps can make of X, whose singular values v begin within 0 and 1 (and
// a margin): v = 0 stays and the steps are continuous, so after each they fill
// [0, top] with the largest |a v + b v^3 + c v^5| over the last such range, which is
// found exactly.  No margin is added to it here: a step would enlarge that too,
// and the next one what came of it (1.05 a step, with the default coefficients:
// 1.2, 1.3, 1.8, 16, 2e6).
struct Spectrum {
    double top;
    double least, most, alpha; // the group's product P: its range, and at v = 0

    void start(double t)
    {
        top = t;
        group();
    }
    void group() { least = most = alpha = 1; }

    // Takes f(w) at the ends of w = v^2 and where k0 + k1 w + k2 w^2 = 0, f's turns.
    template <typename F, typename TAKE> void visit(double k0, double k1, double k2, F f, TAKE take) const
    {
        const double end = top * top, size = std::max({std::fabs(k0), std::fabs(k1), std::fabs(k2)});
        take(f(0.0));
        take(f(end));
        if (!(size > 0))
            return;
        k0 /= size;
        k1 /= size;
        k2 /= size;
        const double square = k1 * k1 - 4 * k0 * k2, sum = -0.5 * (k1 + std::copysign(std::sqrt(std::max(square, 0.0)), k1));
        for (const double w : {sum / k2, k0 / sum})
            if (square >= 0 && w > 0 && w < end)
                take(f(w));
    }
    template <typename F> double largest(double k0, double k1, double k2, F f) const
    {
        double most = 0;
        visit(k0, k1, k2, f, [&](double v) { most = std::max(most, std::fabs(v)); });
        return most;
    }

    double h(const double *c) const
    {
        return largest(c[1], 2 * c[2], 0, [&](double w) { return (c[1] + c[2] * w) * w; });
    }
    double t(const double *c) const
    {
        return largest(c[0], 2 * c[1], 3 * c[2], [&](double w) { return (c[0] + (c[1] + c[2] * w) * w) * w; });
    }
    double k() const { return std::max(std::fabs(most - alpha), std::fabs(least - alpha)); }
    double growth(const double *c) const
    {
        const double q = 1.05 * largest(c[1], 2 * c[2], 0, [&](double w) { return c[0] + (c[1] + c[2] * w) * w; });
        return std::max(1.0, q * q);
    }

    void step(const double *c)
    {
        double q0 = c[0], q1 = c[0];
        visit(c[1], 2 * c[2], 0, [&](double w) { return c[0] + (c[1] + c[2] * w) * w; }, [&](double q) {
            q0 = std::min(q0, q);
            q1 = std::max(q1, q);
        });
        const auto ends = {least * q0, least * q1, most * q0, most * q1};
        least = std::min(ends);
        most = std::max(ends);
        alpha *= c[0];
        top = largest(c[0], 3 * c[1], 5 * c[2], [&](double w) { return (c[0] + (c[1] + c[2] * w) * w) * std::sqrt(w); });
    }
};

constexpr double START_TOP = 1.01, GROWTH_MAX = 3e4;

// Exponent of the power of two that brings values of up to `top`, and 5% more for
// rounding, near 2^15, below fp16's largest.
int exponent_for(double top)
{
    int e;
    std::frexp(std::max(1.05 * top, 1e-30), &e); // below 2^e
    return 15 - e;
}

double power(int e) { return std::ldexp(1.0, e); }

int norm_across(int64_t n)
{
    int a = 1;
    while (a < 64 && (int64_t)a * NORM_W < n)
        a *= 2;
    return a;
}

// A step on long sides with its scales: X, G, H, K are held times powers of two
// that bring their bounds near fp16's largest.
struct LongStep {
    bool first, more;     // of its group; whether the group goes on
    float gram;           // first: G = gram (X X^T)
    float hh, h;          // H = hh G^2 + h G
    float tt, t, gg, g;   // more: T = tt H G + t G = Q G, then G = gg T H + g T = T Q
    float kk, k, kh;      // not first: K = kk H K + k K + kh H, where P = alpha + K
    float xx, x;          // not more: X = xx K X + x X
};

// The steps of a call and the exponent of the first X.  False where a scale or
// a coefficient times it leaves fp32.
bool long_steps(const double (*coef)[3], int steps, bool grouped, LongStep *out, int &start)
{
    Spectrum z;
    z.start(START_TOP);
    int ex = start = exponent_for(z.top), eg = 0, ek = 0;
    double growth = 1;
    bool first = true, ok = true;
    const auto fp32 = [&](double v) {
        ok = ok && std::fabs(v) <= (double)FLT_MAX;
        return (float)v;
    };
    for (int i = 0; i < steps; i++) {
        const double *c = coef[i];
        LongStep &s = out[i] = {};
        const bool last = i + 1 == steps;
        if (first) {
            z.group();
            growth = 1;
            eg = exponent_for(z.top * z.top);
            s.gram = fp32(power(eg - 2 * ex));
        }
        growth *= z.growth(c);
        s.first = first;
        s.more = grouped && !last && growth <= GROWTH_MAX;
        const int eh = exponent_for(z.h(c)), et = exponent_for(z.t(c));
        const double alpha = z.alpha;
        z.step(c);
        // H = b G + c G^2
        s.hh = fp32(c[2] * power(eh - 2 * eg));
        s.h = fp32(c[1] * power(eh - eg));
        if (s.more) {
            // T = Q G = a G + H G, then G = T Q = a T + T H
            const int en = exponent_for(z.top * z.top);
            s.tt = fp32(power(et - eh - eg));
            s.t = fp32(c[0] * power(et - eg));
            s.gg = fp32(power(en - et - eh));
            s.g = fp32(c[0] * power(en - et));
            eg = en;
        }
        // P = alpha + K: Q P = a alpha + (alpha H + a K + H K)
        if (first) {
            ek = eh;
        } else {
            const int en = exponent_for(z.k());
            s.kk = fp32(power(en - eh - ek));
            s.k = fp32(c[0] * power(en - ek));
            s.kh = fp32(alpha * power(en - eh));
            ek = en;
        }
        if (!s.more) {
            // X = alpha X + K X, or alpha X + X K; the last X is the result's
            const int en = last ? 0 : exponent_for(z.top);
            s.x = fp32(z.alpha * power(en - ex));
            s.xx = fp32(power(en - ek - ex));
            ex = en;
        }
        first = !s.more;
    }
    return ok;
}

struct LongPlan {
    int64_t pitch_x, pitch_s, plane_x, plane_s; // elements of a row, of one plane of one matrix
    int64_t rows_per; // rows of a part in the passes over t, none empty
    int parts;
    bool groups; // whether groups of steps on the Gram matrix pay
    size_t sums, x, g, part;
    int squares() const { return groups ? 5 : 2; } // s x s matrices: G, H; T, K and the next K
    size_t total() const { return sums + 2 * x + squares() * g + part; }
};

bool groups_pay(int64_t s, int64_t l) { return 4 * l >= 5 * s; }

int64_t pair_tiles(int64_t M, int64_t N, int64_t t, bool sym)
{
    const int64_t tm = ceil_div(M, t), tn = ceil_div(N, t);
    return sym ? tm * (tm + 1) / 2 : tm * tn;
}

// The tiles that do not fill a round of workgroups are split along k.
struct PairPlan {
    int tile;
    int64_t whole, rest;
    int splits, per;
    size_t part_bytes() const { return splits > 1 ? (size_t)rest * splits * tile * tile * 4 : 0; }
};

PairPlan pair_plan(int64_t B, int64_t M, int64_t N, int64_t K, bool sym, bool outer, int cus)
{
    // tile, bytes of k of a step, tiles at once on a CU, us of a step of a round
    // of them and of one workgroup a CU.  Measured, us of a product (which is
    // between 4 and 6 longer than its steps): 4096 x 4096 by 4096 in 256, 128: 308,
    // 357; symmetric 2048, K = 2048 in 256, 128, 64: 130, 44, 54; symmetric 1000,
    // K = 1000: 75, 24, 12.  Splits cost their sums' way to memory and back:
    // symmetric 4096 in 256, 3 splits, 202 + 36 against 271 whole; symmetric 2048 in
    // 128, 2 splits, 38 + 8 against 44.
    static const struct {
        int tile, step, at_once;
        double full, alone;
    } kinds[] = {{256, PIPE_STEP, 1, 2.36, 2.05}, {128, PIPE_STEP, 2, 1.35, 0.62}, {64, STEP_BYTES, 2, 0.94, 0.5}};
    PairPlan best{};
    double least = 0;
    for (const auto &k : kinds) {
        // two outer operands' addresses do not fit into the registers beside 256 x 256 sums
        if (outer && k.tile == 256)
            continue;
        const int64_t count = B * pair_tiles(M, N, k.tile, sym), steps = ceil_div(2 * K, k.step), slots = (int64_t)cus * k.at_once;
        const int64_t whole = count / slots * slots, rest = count - whole;
        for (int s = 1; s <= 16 && (s == 1 || (rest > 0 && steps >= 4 * s)); s++) {
            const int64_t per = ceil_div(steps, s), used = ceil_div(steps, per), groups = rest * used;
            const double step = groups > 0 && groups <= cus ? k.alone : k.full;
            double t = (double)(whole / slots * steps) * k.full + (double)(ceil_div(groups, slots) * per) * step;
            if (used > 1)
                t += 4 + (double)(groups * k.tile * k.tile) * 8 / 7e6;
            if (!best.tile || t < least) {
                best = {k.tile, whole, rest, (int)used, (int)per};
                least = t;
            }
        }
    }
    return best;
}

LongPlan long_plan(int64_t B, int64_t m, int64_t n, int cus)
{
    const int64_t s = std::min(m, n), l = std::max(m, n);
    LongPlan p;
    p.pitch_x = round_up(n, PAD);
    p.pitch_s = round_up(s, PAD);
    p.plane_x = round_up(m, PAD) * p.pitch_x;
    p.plane_s = s * p.pitch_s;
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>({NORM_MAX_PARTS, ceil_div(4 * cus, B), ceil_div(m * n, 4096), m}));
    p.rows_per = ceil_div(m, parts);
    p.parts = (int)ceil_div(m, p.rows_per);
    const auto bytes = [](int64_t b) { return (size_t)round_up(b, 256); };
    p.sums = bytes(B * p.parts * 8);
    p.groups = groups_pay(s, l);
    p.x = bytes(2 * B * p.plane_x * 2);
    p.g = bytes(2 * B * p.plane_s * 2);
    const PairPlan gram = pair_plan(B, s, s, l, true, m > n, cus), square = pair_plan(B, s, s, s, true, false, cus),
                   apply = pair_plan(B, m, n, s, false, false, cus);
    p.part = bytes((int64_t)std::max({gram.part_bytes(), square.part_bytes(), apply.part_bytes()}));
    return p;
}

template <typename O, int BM, int WM, int WN, bool SYM> hipError_t join_pair(const PairArgs &a, hipStream_t st)
{
    if (a.splits > 1)
        pair_join_kernel<O, BM, BM, WM, WN, SYM><<<a.rest * (BM / WM / 16), WM * WN * WAVE, 0, st>>>(a);
    return hipGetLastError();
}

template <typename O, bool AO, bool BO, bool SYM>
hipError_t pair_product(PairArgs a, int64_t B, float *part, int cus, hipStream_t st)
{
    const PairPlan p = pair_plan(B, a.M, a.N, a.K, SYM, AO && BO, cus);
    a.tiles_m = (int)ceil_div(a.M, p.tile);
    a.tiles_n = (int)ceil_div(a.N, p.tile);
    a.tiles = (int)pair_tiles(a.M, a.N, p.tile, SYM);
    a.whole = (unsigned)p.whole;
    a.rest = (unsigned)p.rest;
    a.splits = (unsigned)p.splits;
    a.per = p.per;
    a.part = part;
    const unsigned grid = a.whole + a.rest * a.splits;
    const bool alone = grid <= (unsigned)cus; // a workgroup a CU
    if (p.tile == 64 && alone)
        pair_kernel<O, AO, BO, SYM, true><<<grid, 512, 0, st>>>(a);
    else if (p.tile == 64)
        pair_kernel<O, AO, BO, SYM, false><<<grid, 512, 0, st>>>(a);
    else if (p.tile == 128 && alone)
        pair_pipe_kernel<O, 128, 128, 2, 4, AO, BO, SYM, 4><<<grid, 512, 0, st>>>(a);
    else if (p.tile == 128)
        pair_pipe_kernel<O, 128, 128, 2, 4, AO, BO, SYM, 2><<<grid, 512, 0, st>>>(a);
    else if constexpr (!(AO && BO))
        pair_pipe_kernel<O, 256, 256, 2, 4, AO, BO, SYM, 2><<<grid, 512, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    return p.tile == 64    ? join_pair<O, 64, 2, 2, SYM>(a, st)
           : p.tile == 128 ? join_pair<O, 128, 2, 4, SYM>(a, st)
                           : join_pair<O, 256, 2, 4, SYM>(a, st);
}

template <typename T, typename O> hipError_t run_long(const OrthoArgs &o, int cus, hipStream_t st)
{
    const int64_t m = o.m, n = o.n, s = std::min(m, n), B = o.B;
    const bool wide = m <= n;
    const LongPlan plan = long_plan(B, m, n, cus);
    char *ws = static_cast<char *>(o.ws);
    double *sums = reinterpret_cast<double *>(ws);
    ws += plan.sums;
    const auto planes = [&](size_t bytes, int64_t ld, int64_t plane) {
        const Planes p{reinterpret_cast<_Float16 *>(ws), ld, 2 * plane};
        ws += bytes;
        return p;
    };
    Planes x = planes(plan.x, plan.pitch_x, plan.plane_x), y = planes(plan.x, plan.pitch_x, plan.plane_x), sq[5]{};
    for (int i = 0; i < plan.squares(); i++)
        sq[i] = planes(plan.g, plan.pitch_s, plan.plane_s);
    Planes &g = sq[0], &h = sq[1], &t = sq[2], &kp = sq[3], &next = sq[4];
    float *part = reinterpret_cast<float *>(ws);
    LongStep list[FA_MAX_ORTHO_STEPS];
    int start;
    if (!long_steps(o.coef, o.steps, plan.groups && sizeof(O) == 2, list, start))
        return hipErrorInvalidValue;
    const int across = norm_across(n);
    const unsigned grid = (unsigned)(B * plan.parts);
    norm_kernel<T><<<grid, NORM_THREADS, 0, st>>>(o, plan.parts, plan.rows_per, across, sums);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    split_kernel<T><<<grid, NORM_THREADS, 0, st>>>(o, plan.parts, plan.rows_per, across, sums, (float)power(start), x, y, round_up(m, PAD));
    e = hipGetLastError();

    // out = q A B + p T + r U of symmetric s x s matrices
    const auto square = [&](const Planes &a, const Planes &b, float q, const Planes &t, float p, const Planes &u, float r,
                            const Planes &out, bool even = false) {
        PairArgs v{};
        v.even = even;
        v.a = a;
        v.b = b;
        v.M = v.N = v.K = (int)s;
        v.q = q;
        v.t = t;
        v.p = p;
        v.u = u;
        v.r = r;
        v.out = out;
        return pair_product<float, false, false, true>(v, B, part, cus, st);
    };
    for (int i = 0; i < o.steps && e == hipSuccess; i++) {
        const LongStep &l = list[i];
        if (l.first) {
            if (!h.p) // without groups, the last step's K has H's place
                std::swap(kp, h);
            PairArgs v{};
            v.a = v.b = x;
            v.M = v.N = (int)s;
            v.K = (int)std::max(m, n);
            v.q = l.gram;
            v.out = g;
            v.even = l.more;
            e = wide ? pair_product<float, false, false, true>(v, B, part, cus, st) : pair_product<float, true, true, true>(v, B, part, cus, st);
        }
        if (e == hipSuccess)
            e = square(g, g, l.hh, g, l.h, {}, 0, h);
        if (l.more && e == hipSuccess) {
            e = square(h, g, l.tt, g, l.t, {}, 0, t);
            if (e == hipSuccess)
                e = square(t, h, l.gg, t, l.g, {}, 0, g, true);
        }
        if (l.first) {
            std::swap(kp, h);
        } else if (e == hipSuccess) {
            e = square(h, kp, l.kk, kp, l.k, h, l.kh, next);
            std::swap(kp, next);
        }
        if (l.more || e != hipSuccess)
            continue;
        PairArgs v{};
        v.o = o;
        v.a = wide ? kp : x;
        v.b = wide ? x : kp;
        v.t = x;
        v.M = (int)m;
        v.N = (int)n;
        v.K = (int)s;
        v.p = l.x;
        v.q = l.xx;
        v.out = i + 1 == o.steps ? Planes{} : y;
        e = wide ? pair_product<O, false, true, false>(v, B, part, cus, st) : pair_product<O, false, false, false>(v, B, part, cus, st);
        std::swap(x, y);
    }
    return e;
}

struct ShortPlan {
    int sb, parts, sums; // sums: parts of G that P is formed from
    int64_t per;
    size_t part, joined, poly;
    size_t total() const { return part + joined + poly; }
};

// `apart`: each stage in a launch of its own.
ShortPlan short_plan(int64_t B, int64_t m, int64_t n, int cus, bool apart = false)
{
    const int64_t s = std::min(m, n), l = std::max(m, n);
    ShortPlan p{};
    p.sb = (int)ceil_div(s, 16);
    // with s <= 32 and up to SHORT_ALONE of the long side a workgroup takes a
    // matrix to the end
    const int64_t want = p.sb <= 2 && l <= SHORT_ALONE ? 1 : std::max<int64_t>(1, ceil_div(2 * cus, B));
    p.per = std::max<int64_t>(SHORT_STEP, round_up(ceil_div(l, want), SHORT_STEP));
    p.parts = (int)ceil_div(l, p.per);
    p.sums = p.parts;
    const int64_t matrix = blocks_of(p.sb) * 256 * 8;
    if (p.parts > 1 || p.sb > 2 || apart) {
        p.part = (size_t)(B * p.parts * matrix);
        if (p.parts > JOIN_PARTS) {
            p.sums = (int)ceil_div(p.parts, JOIN_PARTS);
            p.joined = (size_t)(B * p.sums * matrix);
        }
        if (p.sb > 2 || apart)
            p.poly = (size_t)(B * blocks_of(p.sb)) * sizeof(Block);
    }
    return p;
}

// Rounding of G, 2^-53 of its largest eigenvalue, grows by a step's largest Q^2 until G
// is formed anew.  A singular value that grew as much has it as an error, and
// directions that X does not have end as eigenvalues of either sign on which the
// steps have no hold: singular values spread from 1 to 1e-9 in 64 x 1000, the default
// coefficients, are off by 7e-10 after 8 steps, 7e-9 after 9, 8e-6 after 12, and rank 2
// is lost from 16 on.  A group ends when that growth has passed SHORT_GROWTH_MAX:
// 2^-53 1e8 = 1e-8, below fp32's half step.
constexpr double SHORT_GROWTH_MAX = 1e8;

// Steps of the group that begins with step k.
int short_group(const OrthoArgs &o, int k)
{
    Spectrum z;
    z.start(START_TOP);
    for (int i = 0; i < k; i++)
        z.step(o.coef[i]);
    double growth = 1;
    int end = k;
    do {
        growth *= z.growth(o.coef[end]);
        z.step(o.coef[end++]);
    } while (end < o.steps && growth <= SHORT_GROWTH_MAX);
    return end - k;
}

// Calls of several groups hold the X of as many matrices as have SHORT_HELD elements
// (at least one) in fp64, with G and P of up to SHORT_BLOCKS blocks, and take their
// batch in such passes: 128 MB, or one matrix.
constexpr int64_t SHORT_HELD = 1ll << 23, SHORT_BLOCKS = 1ll << 14;

struct ShortGroups {
    int64_t matrices;
    ShortPlan p;
    size_t total() const { return p.total() + x; }
    size_t x;
};

ShortGroups short_groups(int64_t B, int64_t m, int64_t n, int cus)
{
    ShortGroups g{};
    g.matrices = std::min({B, std::max<int64_t>(1, SHORT_HELD / (m * n)), SHORT_BLOCKS / blocks_of((int)ceil_div(std::min(m, n), 16))});
    g.p = short_plan(g.matrices, m, n, cus, true);
    g.x = (size_t)(g.matrices * m * n) * sizeof(double);
    return g;
}

template <typename O, int SB, bool WIDE> hipError_t run_short_groups(const OrthoArgs &o, int update_dt, int cus, hipStream_t st)
{
    const ShortGroups plan = short_groups(o.B, o.m, o.n, cus);
    const ShortPlan &p = plan.p;
    char *ws = static_cast<char *>(o.ws);
    double *part = reinterpret_cast<double *>(ws), *joined = reinterpret_cast<double *>(ws + p.part);
    Block *poly = reinterpret_cast<Block *>(ws + p.part + p.joined);
    double *x = reinterpret_cast<double *>(ws + p.total());
    const size_t es = update_dt == FA_BF16 ? 2 : 4;
    hipError_t e = hipSuccess;
    for (int64_t b = 0; b < o.B && e == hipSuccess; b += plan.matrices) {
        OrthoArgs t = o;
        t.B = std::min(plan.matrices, o.B - b);
        t.x = static_cast<const char *>(o.x) + b * o.stride_x * es;
        t.momentum = o.momentum ? o.momentum + b * o.stride_m : nullptr;
        t.out = x;
        t.ldo = o.n;
        t.stride_o = o.m * o.n;
        const int64_t pieces = t.B * t.m * ceil_div(t.n, 4);
        const unsigned lift = (unsigned)std::min<int64_t>(ceil_div(pieces, 256), 1 << 16), grid = (unsigned)(t.B * p.parts);
        if (update_dt == FA_BF16)
            short_lift_kernel<__bf16><<<lift, 256, 0, st>>>(t);
        else
            short_lift_kernel<float><<<lift, 256, 0, st>>>(t);
        e = hipGetLastError();
        for (int k = 0, steps; k < o.steps && e == hipSuccess; k += steps) {
            steps = short_group(o, k);
            OrthoArgs g = t;
            g.x = x;
            g.ldx = o.n;
            g.stride_x = o.m * o.n;
            g.momentum = nullptr;
            g.unit = k > 0;
            g.steps = steps;
            std::copy(o.coef[k], o.coef[k] + 3 * steps, g.coef[0]);
            short_kernel<double, float, SB, WIDE, STAGE_GRAM><<<grid, SHORT_THREADS, 0, st>>>(g, p.parts, p.per, p.sums, part, poly);
            e = hipGetLastError();
            const double *sums = part;
            if (e == hipSuccess && p.sums < p.parts) {
                short_join_kernel<<<(unsigned)(t.B * p.sums * blocks_of(SB)), 256, 0, st>>>(part, p.parts, p.sums, blocks_of(SB), joined);
                e = hipGetLastError();
                sums = joined;
            }
            if (e == hipSuccess) {
                short_kernel<float, float, SB, true, STAGE_POLY>
                    <<<(unsigned)t.B, short_threads<STAGE_POLY>(), 0, st>>>(g, p.parts, p.per, p.sums, const_cast<double *>(sums), poly);
                e = hipGetLastError();
            }
            if (e != hipSuccess)
                break;
            if (k + steps < o.steps) {
                short_kernel<double, double, SB, WIDE, STAGE_APPLY><<<grid, SHORT_THREADS, 0, st>>>(g, p.parts, p.per, p.sums, part, poly);
            } else {
                g.out = static_cast<char *>(o.out) + b * o.stride_o * sizeof(O);
                g.ldo = o.ldo;
                g.stride_o = o.stride_o;
                short_kernel<double, O, SB, WIDE, STAGE_APPLY><<<grid, SHORT_THREADS, 0, st>>>(g, p.parts, p.per, p.sums, part, poly);
            }
            e = hipGetLastError();
        }
    }
    return e;
}

template <typename O> hipError_t run_short_passes(const OrthoArgs &o, int update_dt, int cus, hipStream_t st)
{
    const bool wide = o.m <= o.n;
    switch (ceil_div(std::min(o.m, o.n), 16)) {
    case 1:
        return wide ? run_short_groups<O, 1, true>(o, update_dt, cus, st) : run_short_groups<O, 1, false>(o, update_dt, cus, st);
    case 2:
        return wide ? run_short_groups<O, 2, true>(o, update_dt, cus, st) : run_short_groups<O, 2, false>(o, update_dt, cus, st);
    case 3:
        return wide ? run_short_groups<O, 3, true>(o, update_dt, cus, st) : run_short_groups<O, 3, false>(o, update_dt, cus, st);
    default:
        return wide ? run_short_groups<O, 4, true>(o, update_dt, cus, st) : run_short_groups<O, 4, false>(o, update_dt, cus, st);
    }
}

template <typename T, typename O, int SB, bool WIDE> hipError_t run_short_form(const OrthoArgs &o, const ShortPlan &p, hipStream_t st)
{
    char *ws = static_cast<char *>(o.ws);
    double *part = reinterpret_cast<double *>(ws), *joined = reinterpret_cast<double *>(ws + p.part);
    Block *poly = reinterpret_cast<Block *>(ws + p.part + p.joined);
    const unsigned grid = (unsigned)(o.B * p.parts);
    if constexpr (SB <= 2)
        if (p.parts == 1) {
            short_kernel<T, O, SB, WIDE, STAGE_GRAM | STAGE_POLY | STAGE_APPLY><<<grid, SHORT_THREADS, 0, st>>>(o, 1, p.per, 1, part, poly);
            return hipGetLastError();
        }
    short_kernel<T, float, SB, WIDE, STAGE_GRAM><<<grid, SHORT_THREADS, 0, st>>>(o, p.parts, p.per, p.sums, part, poly);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.sums < p.parts) {
        short_join_kernel<<<(unsigned)(o.B * p.sums * blocks_of(SB)), 256, 0, st>>>(part, p.parts, p.sums, blocks_of(SB), joined);
        e = hipGetLastError();
        part = joined;
    }
    if (e != hipSuccess)
        return e;
    if constexpr (SB <= 2) {
        short_kernel<T, O, SB, WIDE, STAGE_POLY | STAGE_APPLY><<<grid, SHORT_THREADS, 0, st>>>(o, p.parts, p.per, p.sums, part, poly);
    } else {
        short_kernel<float, float, SB, true, STAGE_POLY>
            <<<(unsigned)o.B, short_threads<STAGE_POLY>(), 0, st>>>(o, p.parts, p.per, p.sums, part, poly);
        e = hipGetLastError();
        if (e == hipSuccess)
            short_kernel<T, O, SB, WIDE, STAGE_APPLY><<<grid, SHORT_THREADS, 0, st>>>(o, p.parts, p.per, p.sums, part, poly);
    }
    return e == hipSuccess ? hipGetLastError() : e;
}

template <typename T, typename O, int SB> hipError_t run_short_sb(const OrthoArgs &o, const ShortPlan &p, hipStream_t st)
{
    return o.m <= o.n ? run_short_form<T, O, SB, true>(o, p, st) : run_short_form<T, O, SB, false>(o, p, st);
}

template <typename T, typename O> hipError_t run_short(const OrthoArgs &o, int cus, hipStream_t st)
{
    const ShortPlan p = short_plan(o.B, o.m, o.n, cus);
    switch (p.sb) {
    case 1:
        return run_short_sb<T, O, 1>(o, p, st);
    case 2:
        return run_short_sb<T, O, 2>(o, p, st);
    case 3:
        return run_short_sb<T, O, 3>(o, p, st);
    default:
        return run_short_sb<T, O, 4>(o, p, st);
    }
}

template <typename T, typename O> hipError_t run(const OrthoArgs &o, int cus, hipStream_t st)
{
    return std::min(o.m, o.n) <= SHORT_MAX ? run_short<T, O>(o, cus, st) : run_long<T, O>(o, cus, st);
}

} // namespace

bool ortho_reach_ok(const OrthoArgs &o, int dt)
{
    Spectrum z;
    z.start(START_TOP);
    for (int k = 0; k < o.steps; k++) {
        const double *c = o.coef[k];
        if (!std::isfinite(c[0] + c[1] + c[2]) || !(z.h(c) < 1e9))
            return false;
        z.step(c);
        if (!(z.top < 1e9))
            return false;
    }
    const int64_t s = std::min(o.m, o.n);
    LongStep list[FA_MAX_ORTHO_STEPS];
    int start;
    return s <= SHORT_MAX || long_steps(o.coef, o.steps, groups_pay(s, std::max(o.m, o.n)) && dt == FA_BF16, list, start);
}

size_t ortho_workspace_bytes(int64_t B, int64_t m, int64_t n, int cus)
{
    if (B == 0 || m == 0 || n == 0)
        return 0;
    // A call that takes one launch needs none; it asks for some all the same, so that a
    // missing workspace shows at every size.
    if (std::min(m, n) <= SHORT_MAX)
        return std::max({(size_t)256, short_plan(B, m, n, cus).total(), short_groups(B, m, n, cus).total()});
    return long_plan(B, m, n, cus).total();
}

size_t ortho_workspace_needed(const OrthoArgs &o, int cus)
{
    if (o.B > 0 && o.m > 0 && o.n > 0 && std::min(o.m, o.n) <= SHORT_MAX && short_group(o, 0) == o.steps)
        return std::max<size_t>(256, short_plan(o.B, o.m, o.n, cus).total());
    return ortho_workspace_bytes(o.B, o.m, o.n, cus);
}

hipError_t launch_ortho(const OrthoArgs &o, int update_dt, int dt, int cus, hipStream_t s)
{
    if (std::min(o.m, o.n) <= SHORT_MAX && short_group(o, 0) < o.steps)
        return dt == FA_BF16 ? run_short_passes<__bf16>(o, update_dt, cus, s) : run_short_passes<float>(o, update_dt, cus, s);
    if (update_dt == FA_BF16)
        return dt == FA_BF16 ? run<__bf16, __bf16>(o, cus, s) : run<__bf16, float>(o, cus, s);
    return dt == FA_BF16 ? run<float, __bf16>(o, cus, s) : run<float, float>(o, cus, s);
}

} // namespace fa
