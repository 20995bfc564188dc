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
constexpr int WAIT_LOADS = 0x0f70; // s_waitcnt vmcnt(0), the other counters as they are

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

// out(m, n..n+W-1) from the finished sums: z = alpha s + bias, then the
// activation, then the residual, all in fp32, each result rounded once.
template <typename T, int W>
__device__ __forceinline__ void epilogue(const GemmArgs &p, int64_t m, int n, const float *s)
{
    const int valid = p.N - n;
    float z[W], b[W];
#pragma unroll
    for (int i = 0; i < W; i++)
        b[i] = 0.f;
    if (p.bias)
        load_n<T, W>(static_cast<const T *>(p.bias) + n, valid, b);
#pragma unroll
    for (int i = 0; i < W; i++)
        z[i] = __builtin_fmaf(p.alpha, s[i], b[i]);
    if (p.pre)
        store_n<T, W>(static_cast<T *>(p.pre) + m * p.ldp + n, valid, z);
    if (p.act != FA_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < W; i++)
            z[i] = act_of(z[i], p.act);
    }
    if (p.res) {
        load_n<T, W>(static_cast<const T *>(p.res) + m * p.ldr + n, valid, b);
#pragma unroll
        for (int i = 0; i < W; i++)
            z[i] += b[i];
    }
    store_n<T, W>(static_cast<T *>(p.out) + m * p.ldo + n, valid, z);
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

// The same moved straight from memory into LDS (16 bytes a lane, no
// registers), for operands whose rows start on 16 bytes and end on a whole
// chunk.  The hardware places a wavefront's 64 chunks one after another, so
// the exchange of chunks within a row is made on the addresses read.  A chunk
// outside the operand gets an offset past the buffer's range, which reads 0.
constexpr uint32_t OUT_OF_RANGE = 0x80000000u;

template <typename T, bool OUTER, int ROWS, int THREADS> struct Direct {
    static constexpr int EPC = traits<T>::EPC;
    static constexpr int BK = STEP_BYTES / (int)sizeof(T);
    static constexpr int CHUNKS = ROWS * STEP_BYTES / 16;
    static constexpr int CH = (CHUNKS + THREADS - 1) / THREADS;
    static constexpr int CPR = OUTER ? ROWS / EPC : 8;
    uint32_t off[CH]; // byte offset of each chunk from the tile's base
    const char *base;
    int64_t advance; // bytes from one step to the next

    __device__ __forceinline__ void init(const T *p, int64_t ld, int r0, int rows, int k0)
    {
        base = reinterpret_cast<const char *>(OUTER ? p + (int64_t)k0 * ld + r0 : p + (int64_t)r0 * ld + k0);
        advance = OUTER ? BK * ld * (int64_t)sizeof(T) : STEP_BYTES;
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int q = threadIdx.x + c * THREADS;
            if constexpr (!OUTER) {
                const int r = q / 8, ch = (q % 8) ^ (r & 7);
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
                const int k = OUTER ? q / CPR : ((q % 8) ^ ((q / 8) & 7)) * EPC;
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
    }
};

// Waits for this wavefront's copies into LDS, then for the other wavefronts;
// no access to memory moves across.
__device__ __forceinline__ void copies_done()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(WAIT_LOADS);
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

// Workgroup (tile, split): the sums over k in [split * kper, + kper).  With
// more than one split they go to `part` [split][M][N], else to the epilogue.
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
        Direct<T, AO, BM, THREADS> da;
        Direct<T, BO, BN, THREADS> db;
        da.init(a, p.lda, m0, p.M, k0);
        db.init(b, p.ldb, n0, p.N, k0);
        if (steps > 0) {
            da.start(l0, kend - k0);
            db.start(l0 + AB, kend - k0);
        }
        int s = 0;
        for (; s + 1 < steps; s += 2) {
            copies_done();
            da.start(l1, kend - k0 - (s + 1) * BK);
            db.start(l1 + AB, kend - k0 - (s + 1) * BK);
            t.step(l0, l0 + AB, wm, wn, lane);
            copies_done();
            if (s + 2 < steps) {
                da.start(l0, kend - k0 - (s + 2) * BK);
                db.start(l0 + AB, kend - k0 - (s + 2) * BK);
            }
            t.step(l1, l1 + AB, wm, wn, lane);
        }
        copies_done();
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
    // The finished tile goes through LDS, 16 rows of each row of wavefronts at
    // a time, so that whole rows are read and written from consecutive lanes.
    constexpr int W = 8, PITCH = BN + 4, ROWS = WM * 16;
    static_assert(ROWS * PITCH * 4 <= AB + BB, "a pass of the epilogue fits one buffer");
#pragma unroll
    for (int i = 0; i < FM; i++) {
        float *o = reinterpret_cast<float *>(i & 1 ? l1 : l0);
#pragma unroll
        for (int j = 0; j < FN; j++)
            *reinterpret_cast<f32x4 *>(o + ((wave / WN) * 16 + (lane & 15)) * PITCH + wn + j * 16 + (lane >> 4) * 4) =
                t.acc[i][j];
        __syncthreads();
#pragma unroll 1
        for (int q = threadIdx.x; q < ROWS * BN / W; q += THREADS) {
            const int r = q / (BN / W), n = n0 + q % (BN / W) * W;
            const int m = m0 + r / 16 * (BM / WM) + i * 16 + r % 16;
            if (m < p.M && n < p.N) {
                float v[W];
                __builtin_memcpy(v, o + r * PITCH + n - n0, sizeof v);
                if (part)
                    store_n<float, W>(part + ((int64_t)blockIdx.y * p.M + m) * p.N + n, p.N - n, v);
                else
                    epilogue<T, W>(p, m, n, v);
            }
        }
    }
}

// Joins the splits' sums in split order and finishes them.
constexpr int JOIN_THREADS = 256, JOIN_W = 4;

template <typename T> __global__ __launch_bounds__(JOIN_THREADS) void join_kernel(GemmArgs p, const float *part, int splits)
{
    const int64_t groups = (p.N + JOIN_W - 1) / JOIN_W, at = (int64_t)blockIdx.x * JOIN_THREADS + threadIdx.x;
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
    epilogue<T, JOIN_W>(p, m, n, s);
}

template <typename T, int BM, int BN, int WM, int WN, bool DIRECT>
hipError_t run_tile(const GemmArgs &a, int layout, int splits, float *ws, hipStream_t s)
{
    constexpr int BK = STEP_BYTES / (int)sizeof(T);
    const int64_t tm = ((int64_t)a.M + BM - 1) / BM, tn = ((int64_t)a.N + BN - 1) / BN;
    const int steps = std::max(1, (a.K + BK - 1) / BK), per = (steps + splits - 1) / splits;
    splits = (steps + per - 1) / per;
    float *part = splits > 1 ? ws : nullptr;
    const dim3 grid((unsigned)(tm * tn), (unsigned)splits), block(WM * WN * WAVE);
    if (layout == 0)
        gemm_kernel<T, BM, BN, WM, WN, false, false, DIRECT><<<grid, block, 0, s>>>(a, (int)tm, (int)tn, per * BK, part);
    else if (layout == GEMM_B_OUTER)
        gemm_kernel<T, BM, BN, WM, WN, false, true, DIRECT><<<grid, block, 0, s>>>(a, (int)tm, (int)tn, per * BK, part);
    else
        gemm_kernel<T, BM, BN, WM, WN, true, true, DIRECT><<<grid, block, 0, s>>>(a, (int)tm, (int)tn, per * BK, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !part)
        return e;
    const int64_t groups = (int64_t)a.M * ((a.N + JOIN_W - 1) / JOIN_W);
    join_kernel<T><<<(unsigned)((groups + JOIN_THREADS - 1) / JOIN_THREADS), JOIN_THREADS, 0, s>>>(a, part, splits);
    return hipGetLastError();
}

// ------------------------------------------------------------ dz and db
// Eight columns a thread, a workgroup's rows in order: a column's partial sum
// is added in fp32 in row order, and the partials in a fixed order, so db is
// the same bits on every call.
constexpr int AG_THREADS = 256, AG_W = 8, AG_U = 4;
constexpr int AG_COLS = AG_THREADS * AG_W;
constexpr int AG_MIN_ROWS = 16;

template <typename T> __global__ __launch_bounds__(AG_THREADS) void act_grad_kernel(ActGradArgs p, int64_t rows_per)
{
    const int64_t n = ((int64_t)blockIdx.x * AG_THREADS + threadIdx.x) * AG_W;
    if (n >= p.N)
        return;
    const int valid = (int)(p.N - n < AG_W ? p.N - n : AG_W);
    const int64_t r0 = (int64_t)blockIdx.y * rows_per, r1 = r0 + rows_per < p.M ? r0 + rows_per : p.M;
    float sum[AG_W] = {};
    for (int64_t m0 = r0; m0 < r1; m0 += AG_U) {
        float d[AG_U][AG_W], z[AG_U][AG_W];
#pragma unroll
        for (int u = 0; u < AG_U; u++) { // rows past the end read nothing and add 0
            const int v = m0 + u < r1 ? valid : 0;
            load_n<T, AG_W>(static_cast<const T *>(p.dy) + (m0 + u) * p.lddy + n, v, d[u]);
            if (p.act != FA_ACT_NONE)
                load_n<T, AG_W>(static_cast<const T *>(p.pre) + (m0 + u) * p.ldp + n, v, z[u]);
        }
#pragma unroll
        for (int u = 0; u < AG_U; u++) {
            if (p.act != FA_ACT_NONE) {
#pragma unroll
                for (int i = 0; i < AG_W; i++)
                    d[u][i] *= act_slope(z[u][i], p.act);
            }
            if (p.dz)
                store_n<T, AG_W>(static_cast<T *>(p.dz) + (m0 + u) * p.N + n, m0 + u < r1 ? valid : 0, d[u]);
#pragma unroll
            for (int i = 0; i < AG_W; i++)
                sum[i] += d[u][i];
        }
    }
    if (p.db)
        store_n<float, AG_W>(p.part + (int64_t)blockIdx.y * p.N + n, valid, sum);
}

// 64 columns a workgroup: each wavefront adds every CJ_WAVES-th partial, and
// the wavefronts' sums are added in order.
constexpr int CJ_WAVES = 8;

template <typename T> __global__ __launch_bounds__(CJ_WAVES *WAVE) void column_join_kernel(ActGradArgs p, int64_t parts)
{
    __shared__ float sums[CJ_WAVES][WAVE];
    const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
    const int64_t n = (int64_t)blockIdx.x * WAVE + lane;
    float s = 0.f;
    if (n < p.N) {
#pragma unroll 8
        for (int64_t q = wave; q < parts; q += CJ_WAVES)
            s += p.part[q * p.N + n];
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && n < p.N) {
#pragma unroll
        for (int w = 1; w < CJ_WAVES; w++)
            s += sums[w][lane];
        static_cast<T *>(p.db)[n] = (T)s;
    }
}

} // namespace

namespace {

// Whether an operand's rows start on 16 bytes and end on a whole chunk, and a
// tile of it stays within the 31 bits of a buffer offset.
bool direct_ok(const void *p, int64_t ld, int64_t row, size_t es)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld * (int64_t)es % 16 == 0 && row * (int64_t)es % 16 == 0 &&
           ld * (int64_t)es * 257 < (int64_t)OUT_OF_RANGE;
}

enum { TILE_256, TILE_128, TILE_64, TILE_THIN_N, TILE_THIN_M };

struct Plan {
    int tile, splits;
};

int64_t tiles(int64_t M, int64_t N, int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

Plan plan_of(int64_t M, int64_t N, int64_t K, size_t es, int cus)
{
    if (tiles(M, N, 256, 256) * 4 >= 3 * cus)
        return {TILE_256, 1};
    int tile = TILE_64;
    int64_t count = tiles(M, N, 64, 64);
    if (N <= 16) {
        tile = TILE_THIN_N;
        count = tiles(M, N, 128, 16);
    } else if (M <= 16) {
        tile = TILE_THIN_M;
        count = tiles(M, N, 16, 128);
    } else if (tiles(M, N, 128, 128) >= cus) {
        tile = TILE_128;
        count = tiles(M, N, 128, 128);
    }
    // fill the chip, at least 4 steps of k a split
    const int64_t steps = K * (int64_t)es / STEP_BYTES;
    const int64_t want = tile == TILE_128 ? 2 * cus : 4 * cus;
    const int64_t splits = std::min<int64_t>(std::min<int64_t>(want / std::max<int64_t>(count, 1), steps / 4), 64);
    return {tile, (int)std::max<int64_t>(1, splits)};
}

template <typename T, bool DIRECT> hipError_t run_plan(const GemmArgs &a, int layout, Plan p, float *ws, hipStream_t s)
{
    switch (p.tile) {
    case TILE_256:
        if constexpr (DIRECT)
            return run_tile<T, 256, 256, 2, 4, true>(a, layout, 1, ws, s);
        [[fallthrough]];
    case TILE_128:
        return run_tile<T, 128, 128, 2, 2, DIRECT>(a, layout, p.splits, ws, s);
    case TILE_64:
        return run_tile<T, 64, 64, 2, 2, DIRECT>(a, layout, p.splits, ws, s);
    case TILE_THIN_N:
        return run_tile<T, 128, 16, 4, 1, DIRECT>(a, layout, p.splits, ws, s);
    default:
        return run_tile<T, 16, 128, 1, 4, DIRECT>(a, layout, p.splits, ws, s);
    }
}

template <typename T> hipError_t gemm_of(const GemmArgs &a, int layout, float *ws, int cus, hipStream_t s)
{
    const Plan p = plan_of(a.M, a.N, a.K, sizeof(T), cus);
    if (direct_ok(a.a, a.lda, layout & GEMM_A_OUTER ? a.M : a.K, sizeof(T)) &&
        direct_ok(a.b, a.ldb, layout & GEMM_B_OUTER ? a.N : a.K, sizeof(T)))
        return run_plan<T, true>(a, layout, p, ws, s);
    return run_plan<T, false>(a, layout, p, ws, s);
}

} // namespace

size_t gemm_workspace_bytes(int dt, int64_t M, int64_t N, int64_t K, int, int cus)
{
    const Plan p = plan_of(M, N, K, dt == FA_BF16 ? 2 : 4, cus);
    return p.splits > 1 ? (size_t)p.splits * M * N * sizeof(float) : 0;
}

hipError_t launch_gemm(const GemmArgs &a, int dt, int layout, void *ws, int cus, hipStream_t s)
{
    if (a.M == 0 || a.N == 0)
        return hipSuccess;
    float *part = static_cast<float *>(ws);
    return dt == FA_BF16 ? gemm_of<__bf16>(a, layout, part, cus, s) : gemm_of<float>(a, layout, part, cus, s);
}

int64_t act_grad_partials(int64_t M, int64_t N, int cus)
{
    // enough workgroups for the chip, at least AG_MIN_ROWS rows each
    const int64_t across = (N + AG_COLS - 1) / AG_COLS;
    const int64_t want = std::max<int64_t>(1, 4 * (int64_t)cus / std::max<int64_t>(across, 1));
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
    const unsigned g = (unsigned)((a.N + WAVE - 1) / WAVE);
    if (dt == FA_BF16)
        column_join_kernel<__bf16><<<g, CJ_WAVES * WAVE, 0, s>>>(a, parts);
    else
        column_join_kernel<float><<<g, CJ_WAVES * WAVE, 0, s>>>(a, parts);
    return hipGetLastError();
}

} // namespace fa
