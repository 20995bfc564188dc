// A client's top logits of each row (token), and the loss and gradient of a
// student distilled from several clients' top logits.
//
// All of it is bound by reading the logits (and writing the gradient): rows
// are read in 16-byte vectors, whatever their alignment, with the softmax's
// running maximum and sum kept per thread in the same pass.
#include "learn_internal.h"

#include <algorithm>

namespace fa {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int WAVE = 64;
constexpr float NEG_INF = -__builtin_inff();
constexpr float LOG2E = 1.44269504088896341f;

// ------------------------------------------------------------ reductions
// Butterflies over a wavefront, then over the wavefronts in order: the same
// bits on every call.  `lds` holds one float per wavefront.
__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int o = WAVE / 2; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor(v, o));
    return v;
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = WAVE / 2; o > 0; o >>= 1)
        v += __shfl_xor(v, o);
    return v;
}

template <int THREADS> __device__ __forceinline__ float block_max(float v, float *lds)
{
    v = wave_max(v);
    if (threadIdx.x % WAVE == 0)
        lds[threadIdx.x / WAVE] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < THREADS / WAVE; w++)
        v = fmaxf(v, lds[w]);
    __syncthreads();
    return v;
}

template <int THREADS> __device__ __forceinline__ float block_sum(float v, float *lds)
{
    v = wave_sum(v);
    if (threadIdx.x % WAVE == 0)
        lds[threadIdx.x / WAVE] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < THREADS / WAVE; w++)
        v += lds[w];
    __syncthreads();
    return v;
}

// ------------------------------------------------------------ rows
// 16 bytes of a row as EPC floats.  Rows start at any element; the hardware
// takes vector accesses of that alignment.
template <typename T> struct Chunk;

template <> struct Chunk<__bf16> {
    static constexpr int EPC = 8;
    u32x4 v;
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t w = v[i >> 1];
        return __uint_as_float((i & 1) ? w & 0xffff0000u : w << 16);
    }
};
template <> struct Chunk<float> {
    static constexpr int EPC = 4;
    u32x4 v;
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(v[i]); }
};

// Elements [i, i + EPC) of the row, -inf past `end`.
template <typename T> __device__ __forceinline__ Chunk<T> load_row(const T *x, int i, int end)
{
    constexpr int EPC = Chunk<T>::EPC;
    Chunk<T> c;
    if (i + EPC <= end) {
        __builtin_memcpy(&c.v, x + i, 16);
    } else {
        T e[EPC];
#pragma unroll
        for (int j = 0; j < EPC; j++)
            e[j] = i + j < end ? x[i + j] : (T)NEG_INF;
        __builtin_memcpy(&c.v, e, 16);
    }
    return c;
}

// A softmax's running maximum (of x, before the temperature) and sum of
// exp((x - max) / tau), c = log2(e) / tau.  The difference is taken before the
// scaling, so the type's lowest values neither overflow nor lose digits.  A
// maximum of -inf is taken off as 0, so that -inf entries add 0; NaN and +inf
// turn the sum into NaN.  v_exp_f32 flushes results below 2^-126, far under
// the sum's rounding.
struct Softmax {
    float m = NEG_INF, s = 0.f;

    // Returns the chunk's maximum (of its numbers); `special` is set when it
    // holds NaN or +inf.
    template <typename T> __device__ __forceinline__ float add(const Chunk<T> &k, float c, bool &special)
    {
        constexpr int EPC = Chunk<T>::EPC;
        float t = k.get(0);
#pragma unroll
        for (int j = 1; j < EPC; j++)
            t = fmaxf(t, k.get(j));
        const float mn = fmaxf(m, t);
        const float b = mn == NEG_INF ? 0.f : mn;
        s *= __builtin_amdgcn_exp2f((m - b) * c);
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < EPC; j++)
            a += __builtin_amdgcn_exp2f((k.get(j) - b) * c);
        s += a;
        m = mn;
        special = a != a;
        return t;
    }

    __device__ __forceinline__ float scaled_to(float M, float c) const
    {
        return s * __builtin_amdgcn_exp2f((m - (M == NEG_INF ? 0.f : M)) * c);
    }
};

// log sum exp(x / tau) from the row's maximum and sum
__device__ __forceinline__ float lse_of(float m, float s, float inv_tau)
{
    return m == NEG_INF && s == 0.f ? NEG_INF : m * inv_tau + logf(s);
}

// Partial results of one piece of a row, when rows are split.
struct TopPiece {
    float m, s;
};
constexpr int SPLIT_MAX = WAVE; // pieces of a row

// The pieces' sums joined, one lane a piece, to every lane.
__device__ __forceinline__ float lse_of_pieces(const TopPiece *t, int pieces, float c, float inv_tau)
{
    const int lane = threadIdx.x % WAVE;
    const TopPiece q = lane < pieces ? t[lane] : TopPiece{NEG_INF, 0.f};
    const float M = wave_max(q.m);
    return lse_of(M, wave_sum(Softmax{q.m, q.s}.scaled_to(M, c)), inv_tau);
}

// The threads' sums joined, to every thread.
template <int THREADS> __device__ __forceinline__ void join_block(Softmax &t, float c, float *lds)
{
    const float M = block_max<THREADS>(t.m, lds);
    t.s = block_sum<THREADS>(t.scaled_to(M, c), lds);
    t.m = M;
}

// Softmax sums of elements [i0, i1) of a row, to every thread; each thread
// keeps UNROLL loads in flight.
template <typename T, int THREADS>
__device__ __forceinline__ Softmax row_softmax(const T *x, int i0, int i1, float c, float *lds)
{
    constexpr int EPC = Chunk<T>::EPC, UNROLL = 4;
    constexpr int STEP = THREADS * EPC;
    Softmax t;
    bool special;
    int i = i0 + threadIdx.x * EPC;
    for (; i + (UNROLL - 1) * STEP + EPC <= i1; i += UNROLL * STEP) {
        Chunk<T> k[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; u++)
            __builtin_memcpy(&k[u].v, x + i + u * STEP, 16);
#pragma unroll
        for (int u = 0; u < UNROLL; u++)
            t.add(k[u], c, special);
    }
    for (; i < i1; i += STEP)
        t.add(load_row(x, i, i1), c, special);
    join_block<THREADS>(t, c, lds);
    return t;
}

// ------------------------------------------------------------ top logits
// Unsigned keys in the order of the values: NaN of either sign highest, then
// descending numbers, -0 and +0 equal.  bf16 keys have 16 bits.  No value has
// key 0.
template <typename T> struct Key;
template <> struct Key<float> {
    static constexpr int BITS = 32;
    static constexpr uint32_t NAN_KEY = 0xffffffffu;
    static __device__ __forceinline__ uint32_t of(float x)
    {
        const uint32_t b = __float_as_uint(x + 0.f);
        return x != x ? NAN_KEY : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    }
    static __device__ __forceinline__ float value(uint32_t k)
    {
        return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
    }
};
template <> struct Key<__bf16> {
    static constexpr int BITS = 16;
    static constexpr uint32_t NAN_KEY = 0xffffu;
    static __device__ __forceinline__ uint32_t of(float x) { return Key<float>::of(x) >> 16; }
    static __device__ __forceinline__ float value(uint32_t k) { return Key<float>::value(k << 16 | 0xffffu * !(k & 0x8000u)); }
};

constexpr int TR_SMALL = 256, TR_LARGE = 1024, TR_JOIN = 512; // threads
constexpr int TR_U = 2;                        // chunks a thread takes per block
constexpr int TR_PRUNE = 1024;                 // candidates from which on they are cut down to k
// A block adds at most FA_MAX_TOP - 1 threads' worth above its bound and
// FA_MAX_TOP equal to it (see gather_top).
constexpr int TR_CAP = TR_PRUNE + (FA_MAX_TOP - 1) * 8 * TR_U + FA_MAX_TOP + 16;

struct TopLds {
    uint32_t key[TR_CAP];
    int32_t idx[TR_CAP];
    float val[TR_CAP]; // the value itself: keys do not tell -0 or a NaN's bits
    uint32_t out_key[FA_MAX_TOP];
    int32_t out_idx[FA_MAX_TOP];
    float out_val[FA_MAX_TOP];
    uint32_t best[TR_LARGE];
    int n, hits, kept;
    int count[8][16];
    int wave[TR_LARGE / WAVE];
    float red[TR_LARGE / WAVE];
};

// The largest t with at least k of the n keys at or above it, four bits of t
// a step: each wavefront counts the keys at or above the 15 values tried by
// ballot, lane b adds the b-th count, and as the counts fall with b the next
// digit is how many of them reach k.  (Two bits a step took twice the
// barriers: 27.5 and 24.4 us for a row of 151936 fp32 in two kernels.)
template <typename T, int THREADS>
__device__ __forceinline__ uint32_t kth_key(TopLds &l, const uint32_t *keys, int n, int k)
{
    constexpr int STEPS = Key<T>::BITS / 4;
    const int lane = threadIdx.x % WAVE;
    if (threadIdx.x < STEPS * 16)
        (&l.count[0][0])[threadIdx.x] = 0;
    __syncthreads();
    uint32_t cut = 0;
#pragma unroll 1
    for (int step = 0; step < STEPS; step++) {
        const int s = Key<T>::BITS - 4 - 4 * step;
        int mine = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += THREADS) {
            const int i = i0 + threadIdx.x;
            const uint32_t key = i < n ? keys[i] : 0u; // 0 is below every value tried
#pragma unroll
            for (int b = 1; b < 16; b++) {
                const int c = __popcll(__ballot(key >= (cut | ((uint32_t)b << s))));
                mine += lane == b ? c : 0;
            }
        }
        if (mine)
            atomicAdd(&l.count[step][lane], mine);
        __syncthreads();
        const int c = l.count[step][lane & 15];
        const uint32_t digit = __popcll(__ballot(lane > 0 && lane < 16 && c >= k));
        cut |= digit << s;
    }
    return cut;
}

// Cuts the n >= k candidates down to the k largest (ties to the lower index),
// in index order: an entry's place is the number of kept ones before it.
// Returns the k-th largest key.
template <typename T, int THREADS> __device__ __forceinline__ uint32_t prune(TopLds &l, int n, int k)
{
    const uint32_t cut = kth_key<T, THREADS>(l, l.key, n, k);
    if (threadIdx.x == 0)
        l.n = l.kept = 0;
    __syncthreads();
    // first those at or above the cut, in any order, moved to the front: an
    // entry never moves past the tiles that have been read
    for (int i0 = 0; i0 < n; i0 += THREADS) {
        const int i = i0 + threadIdx.x;
        uint32_t key = 0;
        int32_t idx = 0;
        float val = 0.f;
        if (i < n) {
            key = l.key[i];
            idx = l.idx[i];
            val = l.val[i];
        }
        __syncthreads();
        if (i < n && key >= cut) {
            const int at = atomicAdd(&l.n, 1);
            l.key[at] = key;
            l.idx[at] = idx;
            l.val[at] = val;
            if (key > cut)
                atomicAdd(&l.kept, 1);
        }
    }
    __syncthreads();
    const int m = l.n, ties = k - l.kept;
    for (int i = threadIdx.x; i < m; i += THREADS) {
        const uint32_t key = l.key[i];
        const int32_t idx = l.idx[i];
        int gt = 0, eq = 0;
#pragma unroll 4
        for (int j = 0; j < m; j++) {
            const bool before = l.idx[j] < idx, above = l.key[j] > cut;
            gt += before && above;
            eq += before && !above;
        }
        if (key > cut || eq < ties) {
            const int at = gt + (eq < ties ? eq : ties);
            l.out_key[at] = key;
            l.out_idx[at] = idx;
            l.out_val[at] = l.val[i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < k; i += THREADS) {
        l.key[i] = l.out_key[i];
        l.idx[i] = l.out_idx[i];
        l.val[i] = l.out_val[i];
    }
    if (threadIdx.x == 0)
        l.n = k;
    __syncthreads();
    return cut;
}

// Entry b of a thread's U chunks (b counts through them in order), and masks
// over those entries, bit b for entry b.
template <typename T, int U> __device__ __forceinline__ float select(const Chunk<T> *c, int b)
{
    constexpr int EPC = Chunk<T>::EPC;
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < EPC * U; j++)
        v = b == j ? c[j / EPC].get(j % EPC) : v;
    return v;
}

template <typename T, int U> __device__ __forceinline__ bool select_nan(const Chunk<T> *c)
{
    constexpr int EPC = Chunk<T>::EPC;
    bool n = false;
#pragma unroll
    for (int j = 0; j < EPC * U; j++)
        n |= c[j / EPC].get(j % EPC) != c[j / EPC].get(j % EPC);
    return n;
}

template <typename T, int U> __device__ __forceinline__ uint32_t equal_mask(const Chunk<T> *c, uint32_t key)
{
    constexpr int EPC = Chunk<T>::EPC;
    const float t = Key<T>::value(key);
    const bool nan = key == Key<T>::NAN_KEY;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < EPC * U; j++) {
        const float v = c[j / EPC].get(j % EPC);
        m |= (uint32_t)(nan ? v != v : v == t) << j;
    }
    return m;
}

// Entries with keys above `key`; all for 0, none for a NaN's.
template <typename T, int U> __device__ __forceinline__ uint32_t above_mask(const Chunk<T> *c, uint32_t key)
{
    constexpr int EPC = Chunk<T>::EPC;
    if (key == 0)
        return ~0u;
    if (key == Key<T>::NAN_KEY)
        return 0;
    const float t = Key<T>::value(key);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < EPC * U; j++)
        m |= (uint32_t)(!(c[j / EPC].get(j % EPC) <= t)) << j;
    return m;
}

// Entries inside the row: `left` of them from the first chunk's start on,
// chunks `next` entries apart.
template <typename T, int U> __device__ __forceinline__ uint32_t valid_mask(int left, int next)
{
    constexpr int EPC = Chunk<T>::EPC;
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int v = left - u * next;
        m |= (v >= EPC ? (1u << EPC) - 1 : v > 0 ? (1u << v) - 1 : 0u) << (u * EPC);
    }
    return m;
}

// One pass over elements [i0, i1) of a row (at least one) that leaves in `l`
// the min(k, i1 - i0) largest, in index order, and the softmax sums of the
// thread's share in `sm`.  Candidates are the entries above a bound that k
// earlier entries reach (an equal one has k before it and cannot matter).  The
// bound is 0 at first and rises in two ways: when TR_PRUNE candidates have
// gathered they are cut down to k; and when a block's candidates might not fit
// (always in a long row's first block), to the k-th largest of the threads'
// own maxima, above which fewer than k threads have entries.  Entries equal to
// that are taken in index order, k of them at most.
template <typename T, int THREADS>
__device__ __forceinline__ void gather_top(const T *row, int i0, int i1, int k, float c, TopLds &l, Softmax &sm)
{
    constexpr int EPC = Chunk<T>::EPC, U = TR_U;
    constexpr int BLOCK = THREADS * EPC * U, NEXT = THREADS * EPC;
    const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
    const T *x = row + i0;
    const int len = i1 - i0;
    const int mine = threadIdx.x * EPC;
    if (threadIdx.x == 0)
        l.n = l.hits = 0;
    Chunk<T> next[U];
#pragma unroll
    for (int u = 0; u < U; u++)
        next[u] = load_row(x, mine + u * NEXT, len);
    uint32_t bound = 0;
    float bound_value = NEG_INF;
    int n = 0;
    __syncthreads();
    for (int b0 = 0; b0 < len; b0 += BLOCK) {
        Chunk<T> cur[U];
        bool hit;
#pragma unroll
        for (int u = 0; u < U; u++)
            cur[u] = next[u];
        if (b0 + BLOCK < len) {
#pragma unroll
            for (int u = 0; u < U; u++)
                next[u] = load_row(x, mine + b0 + BLOCK + u * NEXT, len);
        }
        float top = NEG_INF;
        bool odd = false;
#pragma unroll
        for (int u = 0; u < U; u++) {
            bool special;
            top = fmaxf(top, sm.add(cur[u], c, special));
            odd |= special;
        }
        hit = top > bound_value || odd || bound == 0;
        const uint64_t hits = __ballot(hit);
        if (lane == 0 && hits)
            atomicAdd(&l.hits, __popcll(hits));
        __syncthreads();
        const int threads_hit = l.hits;
        uint32_t t = bound;
        const int left = len - (mine + b0);
        if (threads_hit * EPC * U > TR_CAP - n) {
            uint32_t best = left > 0 ? Key<T>::of(top) : 0; // 0: no entries
            if (odd && select_nan<T, U>(cur))
                best = Key<T>::NAN_KEY;
            l.best[threadIdx.x] = best;
            // more threads than k have entries above the old bound, so t > bound
            t = kth_key<T, THREADS>(l, l.best, THREADS, k);
            // places of the entries equal to t in index order: chunk u = 0 of
            // all threads comes before u = 1; both counts travel in one word
            uint32_t ties = equal_mask<T, U>(cur, t) & valid_mask<T, U>(left, NEXT);
            const uint32_t cnt = __popc(ties & ((1u << EPC) - 1)) | (uint32_t)__popc(ties >> EPC) << 16;
            uint32_t upto = cnt;
#pragma unroll
            for (int o = 1; o < WAVE; o <<= 1) {
                const uint32_t v = __shfl_up(upto, o);
                upto += lane >= o ? v : 0;
            }
            if (lane == WAVE - 1)
                l.wave[wave] = (int)upto;
            __syncthreads();
            uint32_t before = upto - cnt, total = 0;
#pragma unroll 1
            for (int w = 0; w < THREADS / WAVE; w++) {
                const uint32_t v = (uint32_t)l.wave[w];
                before += w < wave ? v : 0;
                total += v;
            }
            int place0 = (int)(before & 0xffff), place1 = (int)((total & 0xffff) + (before >> 16));
            while (ties) {
                const int b = __builtin_ctz(ties);
                ties &= ties - 1;
                if ((b < EPC ? place0++ : place1++) < k) {
                    const int p = atomicAdd(&l.n, 1);
                    l.key[p] = t;
                    l.idx[p] = i0 + mine + b0 + (b / EPC) * NEXT + b % EPC;
                    l.val[p] = select<T, U>(cur, b);
                }
            }
        }
        if (hit) {
            uint32_t mask = above_mask<T, U>(cur, t) & valid_mask<T, U>(left, NEXT);
            while (mask) {
                const int b = __builtin_ctz(mask);
                mask &= mask - 1;
                const float v = select<T, U>(cur, b);
                const int p = atomicAdd(&l.n, 1);
                l.key[p] = Key<T>::of(v);
                l.idx[p] = i0 + mine + b0 + (b / EPC) * NEXT + b % EPC;
                l.val[p] = v;
            }
        }
        __syncthreads();
        n = l.n;
        if (threadIdx.x == 0)
            l.hits = 0;
        if (n > TR_PRUNE) {
            t = prune<T, THREADS>(l, n, k);
            n = k;
        } else {
            __syncthreads();
        }
        bound = t;
        bound_value = t == 0 ? NEG_INF : t == Key<T>::NAN_KEY ? __builtin_inff() : Key<T>::value(t);
    }
    prune<T, THREADS>(l, n, n < k ? n : k);
}

__device__ __forceinline__ float *piece_vals(const TopRowsArgs &p, int pieces)
{
    return reinterpret_cast<float *>(static_cast<TopPiece *>(p.ws) + p.R * pieces);
}

// A workgroup per row (pieces = 1) or per piece of a row; a piece's results go
// to the workspace, unused places with index -1.
template <typename T, int THREADS>
__global__ __launch_bounds__(THREADS, THREADS == TR_LARGE ? 8 : 4) void top_rows_kernel(TopRowsArgs p, int pieces, int64_t len)
{
    __shared__ TopLds l;
    const float c = p.inv_tau * LOG2E;
    for (int64_t w = blockIdx.x; w < p.R * pieces; w += gridDim.x) {
        const int64_t r = w / pieces;
        const int i0 = (int)((w % pieces) * len), i1 = (int)(i0 + len < p.V ? i0 + len : p.V);
        const T *x = static_cast<const T *>(p.x) + r * p.ldx;
        Softmax sm;
        int n = 0;
        if (p.k > 0) {
            gather_top<T, THREADS>(x, i0, i1, p.k, c, l, sm);
            n = l.n;
        } else {
            bool special;
            for (int i = i0 + threadIdx.x * Chunk<T>::EPC; i < i1; i += THREADS * Chunk<T>::EPC)
                sm.add(load_row(x, i, i1), c, special);
        }
        join_block<THREADS>(sm, c, l.red);
        int32_t *idx = p.idx + w * p.k;
        float *val = p.val + w * p.k;
        if (pieces > 1) {
            val = piece_vals(p, pieces) + w * p.k;
            idx = reinterpret_cast<int32_t *>(piece_vals(p, pieces) + p.R * pieces * p.k) + w * p.k;
            if (threadIdx.x == 0)
                static_cast<TopPiece *>(p.ws)[w] = TopPiece{sm.m, sm.s};
        } else if (threadIdx.x == 0 && p.lse) {
            p.lse[r] = lse_of(sm.m, sm.s, p.inv_tau);
        }
        for (int j = threadIdx.x; j < p.k; j += THREADS) {
            idx[j] = j < n ? l.idx[j] : -1;
            val[j] = j < n ? l.val[j] : 0.f;
        }
        __syncthreads();
    }
}

// Joins a row's pieces: their entries are the candidates, their softmax sums
// are added in piece order.
template <typename T> __global__ __launch_bounds__(TR_JOIN) void top_join_kernel(TopRowsArgs p, int pieces)
{
    __shared__ TopLds l;
    const float c = p.inv_tau * LOG2E;
    for (int64_t r = blockIdx.x; r < p.R; r += gridDim.x) {
        const float *val = piece_vals(p, pieces) + r * pieces * p.k;
        const int32_t *idx = reinterpret_cast<const int32_t *>(piece_vals(p, pieces) + p.R * pieces * p.k) + r * pieces * p.k;
        if (threadIdx.x == 0)
            l.n = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < pieces * p.k; j += TR_JOIN) {
            const int32_t i = idx[j];
            const float v = val[j];
            if (i >= 0) {
                const int at = atomicAdd(&l.n, 1);
                l.key[at] = Key<T>::of(v);
                l.idx[at] = i;
                l.val[at] = v;
            }
        }
        const TopPiece *t = static_cast<const TopPiece *>(p.ws) + r * pieces;
        if (threadIdx.x < WAVE && p.lse) {
            const float lse = lse_of_pieces(t, pieces, c, p.inv_tau);
            if (threadIdx.x == 0)
                p.lse[r] = lse;
        }
        __syncthreads();
        prune<T, TR_JOIN>(l, l.n, p.k);
        for (int j = threadIdx.x; j < p.k; j += TR_JOIN) {
            p.idx[r * p.k + j] = l.idx[j];
            p.val[r * p.k + j] = l.val[j];
        }
        __syncthreads();
    }
}

// How rows are split: only while there are fewer rows than CUs, into pieces
// of at least SPLIT_MIN bytes whose entries the join can hold.
constexpr int64_t SPLIT_MIN = 16384;

void split_rows(int64_t R, int64_t V, size_t es, int64_t most, int cus, int &pieces, int64_t &len)
{
    const int64_t unit = 64; // elements: pieces start on a vector of an aligned row
    int64_t s = R > 0 && R < cus ? (2 * cus + R - 1) / R : 1;
    s = std::min(s, std::min<int64_t>(most, V * (int64_t)es / SPLIT_MIN));
    s = std::max<int64_t>(1, std::min<int64_t>(s, SPLIT_MAX));
    len = (((V + s - 1) / s + unit - 1) / unit) * unit;
    len = std::max(len, unit);
    pieces = (int)std::max<int64_t>(1, (V + len - 1) / len);
}

// ------------------------------------------------------------ distillation
constexpr int DI_SMALL = 256, DI_LARGE = 512;
constexpr int64_t DI_SMALL_BYTES = 16384; // rows up to this take the small workgroup

// LDS of one row's lists, sized by the entries a row can have: per client its
// numbers, per entry its probability and its slot, and a table with a slot for
// each distinct index (open addressing, at most half full).
struct Lists {
    int *len;     // [clients] entries in use; 0: the client did not send the row
    float *mass;  // [clients] sum_j q_cj
    float *kl;    // [clients] sum_j q_cj (log q_cj - z_j / tau)
    float *share; // [clients] n_c over the sum of n of the clients that sent the row
    float *q;     // [entries]
    int *slot;    // [entries] -1: outside the piece
    int *index;   // [slots] -1: free
    float *sum;   // [slots]
    int slots;

    static __host__ __device__ int slots_for(int entries)
    {
        int n = 64;
        while (n < 2 * entries)
            n *= 2;
        return n;
    }
    static __host__ size_t bytes(int clients, int entries)
    {
        return (size_t)(4 * clients + 2 * entries + 2 * slots_for(entries)) * 4;
    }
    __device__ __forceinline__ void place(char *at, int clients, int entries)
    {
        slots = slots_for(entries);
        index = reinterpret_cast<int *>(at);
        sum = reinterpret_cast<float *>(index + slots);
        q = sum + slots;
        slot = reinterpret_cast<int *>(q + entries);
        len = slot + entries;
        mass = reinterpret_cast<float *>(len + clients);
        kl = mass + clients;
        share = kl + clients;
    }
};

// The row's lists: q_cj = exp(v/tau - L_c) and what is summed over them; with
// GRAD also each index in [i0, i1) once, with sum_c w_c q_c added up in client
// order.  One wavefront a client.  A list is used up to its first negative
// index; one that is not strictly increasing or passes V is left out whole and
// raises the flag.
template <typename T, int THREADS, bool LOSS>
__device__ __forceinline__ void load_lists(const DistillArgs &p, int64_t r, const T *z, int i0, int i1, bool grad, Lists &l)
{
    const int lane = threadIdx.x % WAVE;
    if (grad) {
        for (int i = threadIdx.x; i < l.slots; i += THREADS) {
            l.index[i] = -1;
            l.sum[i] = 0.f;
        }
        __syncthreads();
    }
    for (int c = threadIdx.x / WAVE; c < p.clients; c += THREADS / WAVE) {
        const int k = p.k[c], at = p.first[c];
        const int32_t *idx = p.idx[c] + r * k;
        const float *val = p.val[c] + r * k;
        const float given = p.has_tlse ? p.tlse[c][r] : 0.f;
        constexpr int PER = FA_MAX_TOP / WAVE;
        int32_t ix[PER];
        float y[PER];
#pragma unroll
        for (int e = 0; e < PER; e++) {
            const int j = e * WAVE + lane;
            ix[e] = j < k ? idx[j] : -1;
            y[e] = j < k ? val[j] * p.inv_tau : NEG_INF;
        }
        int len = k;
        bool bad = false;
#pragma unroll
        for (int e = PER - 1; e >= 0; e--) {
            const uint64_t b = __ballot(e * WAVE + lane < k && ix[e] < 0);
            len = b ? e * WAVE + __builtin_ctzll(b) : len;
        }
        int32_t last = -1; // the entry before this group's first
        float m = NEG_INF;
#pragma unroll
        for (int e = 0; e < PER; e++) {
            int32_t before = __shfl_up(ix[e], 1);
            before = lane == 0 ? last : before;
            last = __shfl(ix[e], WAVE - 1);
            if (e * WAVE + lane < len) {
                bad |= ix[e] >= p.V || before >= ix[e];
                m = fmaxf(m, y[e]);
            }
        }
        if (__ballot(bad)) {
            if (lane == 0 && p.err)
                *p.err = FA_ERR_INDEX;
            len = 0;
        }
        m = wave_max(m);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < PER; e++)
            if (e * WAVE + lane < len)
                s += y[e] == NEG_INF ? 0.f : expf(y[e] - m);
        s = wave_sum(s);
        if (m == NEG_INF && s == 0.f)
            len = 0; // nothing, or only -inf
        const float L = p.has_tlse ? given : m + logf(s);
        float mass = 0.f, kl = 0.f;
#pragma unroll
        for (int e = 0; e < PER; e++) {
            const int j = e * WAVE + lane;
            if (j >= len)
                continue;
            const float lq = y[e] - L;
            const float q = expf(lq);
            mass += q;
            if (LOSS && q != 0.f)
                kl += q * (lq - (float)z[ix[e]] * p.inv_tau);
            if (grad) {
                int slot = -1;
                if (ix[e] >= i0 && ix[e] < i1) {
                    slot = (uint32_t)ix[e] * 0x9E3779B1u >> 7 & (l.slots - 1);
                    // the table has more slots than entries: a free one, or
                    // the index's own, comes within one round
                    for (int tries = 0; tries < l.slots; tries++) {
                        const int was = atomicCAS(&l.index[slot], -1, ix[e]);
                        if (was == -1 || was == ix[e])
                            break;
                        slot = (slot + 1) & (l.slots - 1);
                    }
                }
                l.q[at + j] = q;
                l.slot[at + j] = slot;
            }
        }
        mass = wave_sum(mass);
        kl = wave_sum(kl);
        if (lane == 0) {
            l.len[c] = len;
            l.mass[c] = mass;
            l.kl[c] = kl;
        }
    }
    __syncthreads();
    // exact up to 2^24, and rounded no further than fp32 beyond
    float W = 0.f;
    for (int c = 0; c < p.clients; c++)
        W += l.len[c] ? p.n[c] : 0.f;
    for (int c = threadIdx.x; c < p.clients; c += THREADS)
        l.share[c] = l.len[c] ? p.n[c] / W : 0.f;
    if (grad)
        // a client has an index once, so its entries touch different slots
        for (int c = 0; c < p.clients; c++) {
            __syncthreads();
            const float w = l.len[c] ? p.n[c] / W : 0.f;
            for (int j = threadIdx.x; j < l.len[c]; j += THREADS) {
                const int s = l.slot[p.first[c] + j];
                if (s >= 0)
                    l.sum[s] = __builtin_fmaf(w, l.q[p.first[c] + j], l.sum[s]);
            }
        }
    __syncthreads();
}

// 16 bytes of gradient to elements [i, i + EPC) of a row, none past `end`
template <typename T> __device__ __forceinline__ void store_row(T *x, int i, int end, const float *v)
{
    constexpr int EPC = Chunk<T>::EPC;
    T e[EPC];
#pragma unroll
    for (int j = 0; j < EPC; j++)
        e[j] = (T)v[j]; // round to nearest even
    if (i + EPC <= end) {
        __builtin_memcpy(x + i, e, 16);
    } else {
#pragma unroll
        for (int j = 0; j < EPC; j++)
            if (i + j < end)
                x[i + j] = e[j];
    }
}

// Where a row's normaliser comes from.
enum { LSE_COMPUTE = 0, LSE_PIECES = 1, LSE_GIVEN = 2 };

// exp((z inv_tau - lse)) of the dense pass: one rounding of the scaled logit
// and one of the difference; v_exp_f32 flushes below 2^-126.
__device__ __forceinline__ float prob(float z, float inv_tau, float lse)
{
    return __builtin_amdgcn_exp2f((z * inv_tau - lse) * LOG2E);
}

// A workgroup per row, or per piece of a row's gradient.  LOSS: writes loss
// and lse (piece 0 does).
template <typename T, int THREADS, bool LOSS, int FROM>
__global__ __launch_bounds__(THREADS) void distill_kernel(DistillArgs p, int grad_pieces, int64_t len, int stat_pieces)
{
    constexpr int EPC = Chunk<T>::EPC;
    extern __shared__ __attribute__((aligned(16))) char dynamic[];
    __shared__ float fl[THREADS / WAVE];
    Lists l;
    l.place(dynamic, p.clients, p.first[p.clients]);
    const float c2 = p.inv_tau * LOG2E;
    for (int64_t w = blockIdx.x; w < p.R * grad_pieces; w += gridDim.x) {
        const int64_t r = w / grad_pieces;
        const int i0 = (int)((w % grad_pieces) * len), i1 = (int)(i0 + len < p.V ? i0 + len : p.V);
        const bool first = i0 == 0;
        const T *z = static_cast<const T *>(p.z) + r * p.ldz;
        T *dz = p.dz ? static_cast<T *>(p.dz) + r * p.lddz : nullptr;
        const float g = p.row_weight ? p.row_weight[r] : 1.f;
        float lse = 0.f, M = 0.f, kl = 0.f;
        bool sent = false;
        if (g != 0.f) {
            load_lists<T, THREADS, LOSS>(p, r, z, i0, i1, dz != nullptr, l);
            if (FROM == LSE_COMPUTE) {
                const Softmax t = row_softmax<T, THREADS>(z, 0, (int)p.V, c2, fl);
                lse = lse_of(t.m, t.s, p.inv_tau);
            } else if (FROM == LSE_PIECES) {
                lse = lse_of_pieces(static_cast<const TopPiece *>(p.ws) + r * stat_pieces, stat_pieces, c2, p.inv_tau);
            } else {
                lse = p.lse[r];
            }
            if (lse != NEG_INF)
                for (int c = 0; c < p.clients; c++)
                    if (l.len[c]) {
                        M = __builtin_fmaf(l.share[c], l.mass[c], M);
                        kl = __builtin_fmaf(l.share[c], __builtin_fmaf(lse, l.mass[c], l.kl[c]), kl);
                        sent = true;
                    }
        }
        if (LOSS && first && threadIdx.x == 0) {
            p.loss[r] = sent ? g * (p.tau * p.tau) * kl : 0.f;
            if (p.lse)
                p.lse[r] = lse;
        }
        if (dz && !sent) {
            const float zero[EPC] = {};
            for (int i = i0 + threadIdx.x * EPC; i < i1; i += THREADS * EPC)
                store_row(dz, i, i1, zero);
        } else if (dz) {
            // The listed entries' gradients are taken from z before the dense
            // pass, as dz may be z, and written after it.
            const float gt = g * p.tau, gm = gt * M;
            for (int i = threadIdx.x; i < l.slots; i += THREADS)
                if (l.index[i] >= 0)
                    l.sum[i] = gt * (M * prob((float)z[l.index[i]], p.inv_tau, lse) - l.sum[i]);
            __syncthreads();
            for (int i = i0 + threadIdx.x * EPC; i < i1; i += THREADS * EPC) {
                const Chunk<T> k = load_row(z, i, i1);
                float v[EPC];
#pragma unroll
                for (int j = 0; j < EPC; j++)
                    v[j] = gm * prob(k.get(j), p.inv_tau, lse);
                store_row(dz, i, i1, v);
            }
            __syncthreads();
            for (int i = threadIdx.x; i < l.slots; i += THREADS)
                if (l.index[i] >= 0)
                    dz[l.index[i]] = (T)l.sum[i];
        }
        __syncthreads();
    }
}

// Softmax sums of the pieces of each row (rows of weight 0 are not read).
template <typename T, int THREADS>
__global__ __launch_bounds__(THREADS) void row_stats_kernel(DistillArgs p, int pieces, int64_t len)
{
    __shared__ float fl[THREADS / WAVE];
    for (int64_t w = blockIdx.x; w < p.R * pieces; w += gridDim.x) {
        const int64_t r = w / pieces;
        const int i0 = (int)((w % pieces) * len), i1 = (int)(i0 + len < p.V ? i0 + len : p.V);
        if (p.row_weight && p.row_weight[r] == 0.f)
            continue;
        const T *z = static_cast<const T *>(p.z) + r * p.ldz;
        const Softmax t = row_softmax<T, THREADS>(z, i0, i1, p.inv_tau * LOG2E, fl);
        if (threadIdx.x == 0)
            static_cast<TopPiece *>(p.ws)[w] = TopPiece{t.m, t.s};
        __syncthreads();
    }
}

template <typename T, int THREADS, bool LOSS, int FROM>
hipError_t run_distill(const DistillArgs &a, int pieces, int64_t len, int stat_pieces, int cus, hipStream_t s)
{
    const unsigned grid = (unsigned)std::min<int64_t>(a.R * pieces, (int64_t)cus * 16);
    const size_t lds = Lists::bytes(a.clients, a.first[a.clients]);
    static_assert((4 * FA_MAX_CLIENTS + 2 * FA_MAX_LIST_ENTRIES + 4 * FA_MAX_LIST_ENTRIES) * 4 <= 128 << 10, "the largest lists fit in LDS");
    static const hipError_t allowed = hipFuncSetAttribute(reinterpret_cast<const void *>(&distill_kernel<T, THREADS, LOSS, FROM>),
                                                          hipFuncAttributeMaxDynamicSharedMemorySize, 128 << 10);
    (void)allowed; // a launch that needs more than the default then fails and says so
    distill_kernel<T, THREADS, LOSS, FROM><<<grid, THREADS, lds, s>>>(a, pieces, len, stat_pieces);
    return hipGetLastError();
}

template <typename T> hipError_t distill_of(const DistillArgs &a, bool loss, int cus, hipStream_t s)
{
    int pieces;
    int64_t len;
    split_rows(a.R, a.V, sizeof(T), SPLIT_MAX, cus, pieces, len);
    const bool small = a.V * (int64_t)sizeof(T) <= DI_SMALL_BYTES;
    if (!loss) {
        if (small)
            return run_distill<T, DI_SMALL, false, LSE_GIVEN>(a, pieces, len, 0, cus, s);
        return run_distill<T, DI_LARGE, false, LSE_GIVEN>(a, pieces, len, 0, cus, s);
    }
    if (pieces == 1) {
        if (small)
            return run_distill<T, DI_SMALL, true, LSE_COMPUTE>(a, 1, len, 0, cus, s);
        return run_distill<T, DI_LARGE, true, LSE_COMPUTE>(a, 1, len, 0, cus, s);
    }
    row_stats_kernel<T, DI_LARGE><<<(unsigned)(a.R * pieces), DI_LARGE, 0, s>>>(a, pieces, len);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    if (!a.dz)
        return run_distill<T, DI_LARGE, true, LSE_PIECES>(a, 1, a.V, pieces, cus, s);
    if (a.dz != a.z)
        return run_distill<T, DI_LARGE, true, LSE_PIECES>(a, pieces, len, pieces, cus, s);
    // In place: the loss reads listed logits of the whole row, so it is
    // finished before the pieces overwrite them.
    DistillArgs b = a;
    b.dz = nullptr;
    e = run_distill<T, DI_LARGE, true, LSE_PIECES>(b, 1, a.V, pieces, cus, s);
    if (e != hipSuccess)
        return e;
    return run_distill<T, DI_LARGE, false, LSE_PIECES>(a, pieces, len, pieces, cus, s);
}

template <typename T> hipError_t top_rows_of(const TopRowsArgs &a, int cus, hipStream_t s)
{
    int pieces;
    int64_t len;
    split_rows(a.R, a.V, sizeof(T), TR_CAP / std::max(a.k, 1), cus, pieces, len);
    const unsigned grid = (unsigned)std::min<int64_t>(a.R * pieces, (int64_t)cus * 16);
    if (len * (int64_t)sizeof(T) <= DI_SMALL_BYTES)
        top_rows_kernel<T, TR_SMALL><<<grid, TR_SMALL, 0, s>>>(a, pieces, len);
    else
        top_rows_kernel<T, TR_LARGE><<<grid, TR_LARGE, 0, s>>>(a, pieces, len);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || pieces == 1)
        return e;
    top_join_kernel<T><<<(unsigned)std::min<int64_t>(a.R, (int64_t)cus * 16), TR_JOIN, 0, s>>>(a, pieces);
    return hipGetLastError();
}

} // namespace

size_t top_rows_workspace_bytes(int dt, int64_t R, int64_t V, int64_t k, int cus)
{
    int pieces;
    int64_t len;
    split_rows(R, V, dt == FA_BF16 ? 2 : 4, TR_CAP / std::max<int64_t>(k, 1), cus, pieces, len);
    return pieces > 1 ? (size_t)(R * pieces) * (sizeof(TopPiece) + 8 * (size_t)k) : 0;
}

hipError_t launch_top_rows(const TopRowsArgs &a, int dt, int cus, hipStream_t s)
{
    if (a.R == 0)
        return hipSuccess;
    return dt == FA_BF16 ? top_rows_of<__bf16>(a, cus, s) : top_rows_of<float>(a, cus, s);
}

size_t distill_workspace_bytes(int dt, int64_t R, int64_t V, int cus)
{
    int pieces;
    int64_t len;
    split_rows(R, V, dt == FA_BF16 ? 2 : 4, SPLIT_MAX, cus, pieces, len);
    return pieces > 1 ? (size_t)(R * pieces) * sizeof(TopPiece) : 0;
}

hipError_t launch_distill(const DistillArgs &a, int dt, bool loss, int cus, hipStream_t s)
{
    if (a.R == 0)
        return hipSuccess;
    return dt == FA_BF16 ? distill_of<__bf16>(a, loss, cus, s) : distill_of<float>(a, loss, cus, s);
}

} // namespace fa
