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
#include "tiles.h"

#include <algorithm>

namespace fa {
namespace {

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
    t.clear();

    if constexpr (DIRECT) {
        Direct<T, AO, BM, THREADS, STEP_BYTES> da;
        Direct<T, BO, BN, THREADS, STEP_BYTES> db;
        da.init(a, p.lda, m0, p.M, k0);
        db.init(b, p.ldb, n0, p.N, k0);
        t.run(l0, l1, steps, wm, wn, lane, [&](char *l, int s) {
            da.start(l, kend - k0 - s * BK);
            db.start(l + AB, kend - k0 - s * BK);
        });
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
// the 1.66 GHz that the card holds under this load).
template <typename T, int BM, int BN, int WM, int WN, bool AO, bool BO>
__global__ __launch_bounds__(WM *WN *WAVE) void pipe_kernel(GemmArgs p, int tiles_m, int tiles_n)
{
    constexpr int THREADS = WM * WN * WAVE;
    constexpr int BK = PIPE_STEP / (int)sizeof(T);
    constexpr int AB = BM * PIPE_STEP, BB = BN * PIPE_STEP;
    __shared__ __attribute__((aligned(1024))) char l0[AB + BB];
    __shared__ __attribute__((aligned(1024))) char l1[AB + BB];
    __shared__ __attribute__((aligned(1024))) char l2[AB + BB];
    __shared__ __attribute__((aligned(1024))) char l3[AB + BB];

    unsigned tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int m0 = (int)tm * BM, n0 = (int)tn * BN;
    Pipe<T, BM, BN, WM, WN, AO, BO> t;
    Direct<T, AO, BM, THREADS, PIPE_STEP> da;
    Direct<T, BO, BN, THREADS, PIPE_STEP> db;
    da.init(static_cast<const T *>(p.a), p.lda, m0, p.M, 0);
    db.init(static_cast<const T *>(p.b), p.ldb, n0, p.N, 0);
    int left = p.K; // of the next step to copy; steps past the end copy zeros
    t.run(l0, l1, l2, l3, (p.K + BK - 1) / BK, [&](char *l) {
        da.start(l, left);
        db.start(l + AB, left);
        left -= BK;
    });
    write_tile<T, BM, BN, WM, WN, AB + BB>(p, m0, n0, t.acc, l0, l1, nullptr);
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
        f.blocks[j] = finish_blocks(a.M, a.N);
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

// An fp32 as a + 2^-8 b + 2^-16 c of bf16: 8 bits each, cut off rather than
// rounded, so that the first stays finite; the others are scaled so that small
// values keep their bits.  NaN and infinities have the first alone.
__device__ __forceinline__ void store_planes(__bf16 *to, int64_t plane, const float *v)
{
    __bf16 e[3][AG_W];
#pragma unroll
    for (int i = 0; i < AG_W; i++) {
        const auto cut = [](float x) { return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & 0xffff0000u); };
        const bool finite = fabsf(v[i]) < INFINITY;
        const float hi = finite ? cut(v[i]) : v[i], rest = finite ? (v[i] - hi) * 256.f : 0.f, mid = cut(rest);
        e[0][i] = (__bf16)hi;
        e[1][i] = (__bf16)mid;
        e[2][i] = (__bf16)((rest - mid) * 256.f);
    }
#pragma unroll
    for (int q = 0; q < 3; q++)
        __builtin_memcpy(to + q * plane, e[q], sizeof e[q]);
}

// SCALED: with column factors, for the layers on 8-bit weights.  They are a form of
// their own: asked for at run time, they and fp32's three parts take 12 registers
// and with them a wavefront a SIMD (1594 x 2440 fp32, GELU, column sums: 13.1 us
// against 11.3; 4096 x 8192 51.8 against 48.9, bf16 35.6 against 34.9).
template <typename T, bool SCALED>
__global__ __launch_bounds__(AG_THREADS) void act_grad_kernel(ActGradArgs p, int64_t rows_per, int across)
{
    __shared__ float sums[AG_THREADS][AG_W + 1];
    const int col = threadIdx.x & (across - 1), group = threadIdx.x / across, groups = AG_THREADS / across;
    const int64_t n = ((int64_t)blockIdx.x * across + col) * AG_W;
    const int valid = (int)(p.N - n < AG_W ? p.N - n : AG_W);
    const int64_t r0 = (int64_t)blockIdx.y * rows_per, r1 = r0 + rows_per < p.M ? r0 + rows_per : p.M;
    float sum[AG_W] = {}, scale[AG_W];
    if constexpr (SCALED)
        load_n<float, AG_W>(p.col_scale + n, valid, scale);
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
#pragma unroll
            for (int i = 0; i < AG_W; i++)
                sum[i] += d[u][i];
            if constexpr (SCALED) {
#pragma unroll
                for (int i = 0; i < AG_W; i++)
                    d[u][i] *= scale[i];
            }
            if constexpr (SCALED && sizeof(T) == 4)
                store_planes(static_cast<__bf16 *>(p.dz) + m * p.lddz + n, p.plane, d[u]);
            else if (p.dz)
                store_n<T, AG_W>(static_cast<T *>(p.dz) + m * p.lddz + n, AG_W, d[u]);
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
    bool ok_a = direct_ok(a.a, a.lda, row_a, a.a_padded, sizeof(T)), ok_b = direct_ok(a.b, a.ldb, row_b, a.b_padded, sizeof(T));
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

int64_t finish_blocks(int64_t M, int64_t N)
{
    return (M * ((N + JOIN_W - 1) / JOIN_W) + FINISH_THREADS - 1) / FINISH_THREADS;
}

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
    const auto kernel = dt == FA_BF16 ? (a.col_scale ? act_grad_kernel<__bf16, true> : act_grad_kernel<__bf16, false>)
                                      : (a.col_scale ? act_grad_kernel<float, true> : act_grad_kernel<float, false>);
    kernel<<<grid, AG_THREADS, 0, s>>>(a, rows_per, across);
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
