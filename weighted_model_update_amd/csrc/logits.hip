// A client's top logits of each row (token), and the loss and gradient of a
// student distilled from several clients' top logits.
//
// Rows are read in 16-byte vectors, whatever their alignment, with the softmax's
// running maximum and sum kept per thread in the same pass.  The passes are
// bound by reading the logits (and writing the gradient) and, where a logit
// takes a dozen instructions, by the vector units.
#include "device_once.h"
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

// max of numbers, NaN aside.  (fmaxf costs two instructions more for each
// operand whose NaN might be signalling; where one is, the sum that a maximum
// belongs to is NaN whatever the maximum.)
__device__ __forceinline__ float max2(float a, float b)
{
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// Up to this size of max * c the exponent x * c - max * c is one fused
// multiply-add.  It exposes what the rounding of max * c left off, half a step
// of 64 .. 128 or 2^-18 at most: 2.6e-6 of an entry, below half a step of the
// normaliser.  Beyond, the difference comes first: from 2^31 on the fused
// form's exponent alone would leave the range of fp32 (rows under a mask of
// -1e10, small temperatures).
constexpr float FUSED_UP_TO = 128.f;

// A softmax's running maximum (of x, before the temperature) and sum of
// exp((x - max) / tau), c = log2(e) / tau.  A maximum of -inf is taken off as
// 0, so that -inf entries add 0; NaN and +inf turn the sum into NaN.  Each
// thread's sum refers to its own running maximum.  v_exp_f32 flushes results
// below 2^-126, far under the sum's rounding.  What bounds the pass beside the
// memory is the vector unit: about five instructions an entry.
struct Softmax {
    float m = NEG_INF, s = 0.f;

    // `tops` receives the maximum of each chunk's numbers; `special` is set
    // when the chunks hold NaN or +inf.
    template <typename T, int N>
    __device__ __forceinline__ void add(const Chunk<T> *k, float c, bool &special, float *tops)
    {
        constexpr int EPC = Chunk<T>::EPC;
        float mn = m;
#pragma unroll
        for (int u = 0; u < N; u++) {
            float t = max2(k[u].get(0), k[u].get(1));
#pragma unroll
            for (int j = 2; j < EPC; j += 2)
                t = max3(t, k[u].get(j), k[u].get(j + 1));
            tops[u] = t;
            mn = max2(mn, t);
        }
        const float b = mn == NEG_INF ? 0.f : mn, bc = b * c;
        float a = 0.f;
        s *= __builtin_amdgcn_exp2f((m - b) * c); // exactly 1 while the maximum stays
        if (__any(fabsf(bc) > FUSED_UP_TO)) {
#pragma unroll
            for (int j = 0; j < EPC * N; j++)
                a += __builtin_amdgcn_exp2f((k[j / EPC].get(j % EPC) - b) * c);
        } else {
#pragma unroll
            for (int j = 0; j < EPC * N; j++)
                a += __builtin_amdgcn_exp2f(__builtin_fmaf(k[j / EPC].get(j % EPC), c, -bc));
        }
        s += a;
        m = mn;
        special = a != a;
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
__device__ __forceinline__ Softmax join_lanes(const Softmax &q, float c)
{
    const float M = wave_max(q.m);
    return Softmax{M, wave_sum(q.scaled_to(M, c))};
}

__device__ __forceinline__ Softmax join_pieces(const TopPiece *t, int pieces, float c)
{
    const int lane = threadIdx.x % WAVE;
    return join_lanes(lane < pieces ? Softmax{t[lane].m, t[lane].s} : Softmax{}, c);
}

// The threads' sums joined, to every thread.
template <int THREADS> __device__ __forceinline__ void join_block(Softmax &t, float c, float *lds)
{
    const float M = block_max<THREADS>(t.m, lds);
    t.s = block_sum<THREADS>(t.scaled_to(M, c), lds);
    t.m = M;
}

// Softmax sums of elements [i0, i1) of a row and what t holds already, to every
// thread; each thread keeps UNROLL loads in flight.
template <typename T, int THREADS>
__device__ __forceinline__ Softmax row_softmax(const T *x, int i0, int i1, float c, float *lds, Softmax t = {})
{
    constexpr int EPC = Chunk<T>::EPC, UNROLL = 4;
    constexpr int STEP = THREADS * EPC;
    bool special;
    float tops[2];
    int i = i0 + threadIdx.x * EPC;
    for (; i + (UNROLL - 1) * STEP + EPC <= i1; i += UNROLL * STEP) {
        Chunk<T> k[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; u++)
            __builtin_memcpy(&k[u].v, x + i + u * STEP, 16);
#pragma unroll
        for (int u = 0; u < UNROLL; u += 2)
            t.add<T, 2>(k + u, c, special, tops);
    }
    // the rest in pairs too: a thread's chunks are then added the same way
    // wherever its loop starts, and the loss has the same bits with the
    // gradient and without
    for (; i < i1; i += 2 * STEP) {
        const Chunk<T> k[2] = {load_row(x, i, i1), load_row(x, i + STEP, i1)};
        t.add<T, 2>(k, c, special, tops);
    }
    join_block<THREADS>(t, c, lds);
    return t;
}

// The same of a whole row read piece by piece, with the bits that the pieces'
// sums joined from the workspace have.
template <typename T, int THREADS>
__device__ __forceinline__ Softmax row_by_pieces(const T *x, int V, int len, int pieces, float c, float *lds)
{
    Softmax mine;
    for (int q = 0; q < pieces; q++) {
        const Softmax t = row_softmax<T, THREADS>(x, q * len, V - q * len < len ? V : (q + 1) * len, c, lds);
        if ((int)threadIdx.x % WAVE == q)
            mine = t;
    }
    return join_lanes(mine, c);
}

// Whether a stored normaliser is so large that its own rounding would show in
// exp(z / tau - lse): then the row's maximum and sum are taken again.
__device__ __forceinline__ bool lse_too_coarse(float lse) { return !(fabsf(lse) * LOG2E <= FUSED_UP_TO); }

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

// A workgroup's shape and its LDS: THREADS_; QUEUE_, chunks it can hold; CAP_,
// candidates it can hold; U_, chunks a thread takes for the first bound.
template <int THREADS_, int QUEUE_, int CAP_, int U_> struct TopLds {
    static constexpr int THREADS = THREADS_, QUEUE = QUEUE_, CAP = CAP_, U = U_;
    static_assert(CAP >= 2 * FA_MAX_TOP, "the k largest and their ties fit");
    union {
        struct { // candidates
            uint32_t key[CAP];
            int32_t idx[CAP];
            float val[CAP]; // the value itself: keys do not tell -0 or a NaN's bits
        };
        struct { // chunks that hold candidates, and where they start in the row
            u32x4 chunk[QUEUE];
            int32_t at[QUEUE];
        };
    };
    int32_t out_idx[FA_MAX_TOP];
    float out_val[FA_MAX_TOP];
    uint32_t best[THREADS];
    int n, kept;
    int count[8][16];
    int wave[THREADS / WAVE];
    float red[THREADS / WAVE];
};

// The largest t with at least k of the n keys at or above it, four bits of t
// a step: each wavefront counts the keys at or above the 15 values tried by
// ballot, lane b adds the b-th count, and as the counts fall with b the next
// digit is how many of them reach k.  (Two bits a step took twice the
// barriers: 27.5 and 24.4 us for a row of 151936 fp32 in two kernels.)
// It stops where at most `spare` more than k reach it; the lower bits are 0
// then, which selects the same keys.  With n <= k + spare keys that is at once,
// and the result 0 bounds nothing: EXACT_KEY goes through all bits.
constexpr int EXACT_KEY = -1;

template <int BITS, typename L>
__device__ __forceinline__ uint32_t kth_key(L &l, const uint32_t *keys, int n, int k, int spare)
{
    constexpr int STEPS = BITS / 4;
    const int lane = threadIdx.x % WAVE;
    if (threadIdx.x < STEPS * 16)
        (&l.count[0][0])[threadIdx.x] = 0;
    __syncthreads();
    uint32_t cut = 0;
    int have = n; // keys at or above the cut
#pragma unroll 1
    for (int step = 0; step < STEPS && have > k + spare; step++) {
        const int s = BITS - 4 - 4 * step;
        int mine = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += L::THREADS) {
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
        have = digit > 0 ? __shfl(c, (int)digit) : have;
    }
    return cut;
}

// Moves the candidates with keys at or above `cut` to the front, in any order:
// an entry never moves past the tiles that have been read.  Returns how many
// there are; l.kept counts those above the cut.
template <typename L> __device__ __forceinline__ int keep_from(L &l, int n, uint32_t cut)
{
    if (threadIdx.x == 0)
        l.n = l.kept = 0;
    __syncthreads();
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += L::THREADS) {
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
    return l.n;
}

// Cuts the n >= k candidates down to the k largest (ties to the lower index),
// in index order: an entry's place is the number of kept ones before it.  Of
// their keys nothing is left.
template <typename T, typename L> __device__ __forceinline__ void prune(L &l, int n, int k)
{
    uint32_t cut = kth_key<Key<T>::BITS>(l, l.key, n, k, 0);
    int m = keep_from(l, n, cut);
    if (m > k + L::THREADS / 4) {
        // many equal to the cut: the first of them by index, found as the
        // largest keys again.  (Counting them out below took 0.5 ms for 2000.)
        for (int i = threadIdx.x; i < m; i += L::THREADS)
            l.key[i] = l.key[i] > cut ? ~0u : ~(uint32_t)l.idx[i];
        __syncthreads();
        cut = kth_key<32>(l, l.key, m, k, 0);
        m = keep_from(l, m, cut);
    }
    const int ties = k - l.kept;
#pragma unroll 1
    for (int i = threadIdx.x; i < m; i += L::THREADS) {
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
            l.out_idx[at] = idx;
            l.out_val[at] = l.val[i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < k; i += L::THREADS) {
        l.idx[i] = l.out_idx[i];
        l.val[i] = l.out_val[i];
    }
    if (threadIdx.x == 0)
        l.n = k;
    __syncthreads();
}

// One pass over elements [i0, i1) of a row that queues the chunks with entries
// above the key `bound` and adds up the softmax.  A chunk is
// queued whole, from its maximum alone, so that a wavefront in which some lane
// hits pays about as much as for two more entries a lane.  (Taking the entries
// out on the spot cost each wavefront several instructions an entry: 396 us
// where this took 334, 4096 rows of 128256 bf16, k = 64.)  Chunks are
// counted even where they no longer fit.  No barrier until the end.
template <typename T, typename L>
__device__ __forceinline__ int stream_above(const T *x, int i0, int i1, uint32_t bound, float c, L &l, Softmax &sm)
{
    constexpr int EPC = Chunk<T>::EPC, UNROLL = 4, STEP = L::THREADS * EPC;
    // above a NaN's key there is nothing; a NaN's place in a chunk is told by
    // the sum, or here, where +inf is told apart
    const bool none = bound == Key<T>::NAN_KEY, all = bound < Key<T>::of(NEG_INF);
    const float above = none ? __builtin_inff() : Key<T>::value(bound);
    const auto queue = [&](const Chunk<T> &k, bool hit, int i) {
        if ((hit || all) && !none) {
            const int p = atomicAdd(&l.n, 1);
            if (p < L::QUEUE) {
                l.chunk[p] = k.v;
                l.at[p] = i;
            }
        }
    };
    int i = i0 + threadIdx.x * EPC;
    for (; i + (UNROLL - 1) * STEP + EPC <= i1; i += UNROLL * STEP) {
        Chunk<T> k[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; u++)
            __builtin_memcpy(&k[u].v, x + i + u * STEP, 16);
#pragma unroll
        for (int u = 0; u < UNROLL; u += 2) {
            bool odd;
            float t[2];
            sm.add<T, 2>(k + u, c, odd, t);
            queue(k[u], t[0] > above || odd, i + u * STEP);
            queue(k[u + 1], t[1] > above || odd, i + (u + 1) * STEP);
        }
    }
    for (; i < i1; i += STEP) {
        const Chunk<T> k = load_row(x, i, i1);
        bool odd;
        float t;
        sm.add<T, 1>(&k, c, odd, &t);
        queue(k, t > above || odd, i);
    }
    __syncthreads();
    return l.n;
}

// The entries of the n queued chunks above `bound` become the candidates.
// Returns how many there are, even where they do not fit.
template <typename T, typename L>
__device__ __forceinline__ int take_queued(int n, int i1, uint32_t bound, L &l)
{
    constexpr int EPC = Chunk<T>::EPC, PER = (L::QUEUE + L::THREADS - 1) / L::THREADS;
    Chunk<T> k[PER];
    int at[PER];
#pragma unroll
    for (int e = 0; e < PER; e++) {
        const int q = e * L::THREADS + threadIdx.x;
        at[e] = q < n ? l.at[q] : -1;
        if (q < n)
            k[e].v = l.chunk[q];
    }
    __syncthreads();
    if (threadIdx.x == 0)
        l.n = 0;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < PER; e++) {
        if (at[e] < 0)
            continue;
#pragma unroll
        for (int j = 0; j < EPC; j++) {
            const float v = k[e].get(j);
            const uint32_t key = Key<T>::of(v);
            if (key > bound && at[e] + j < i1) {
                const int p = atomicAdd(&l.n, 1);
                if (p < L::CAP) {
                    l.key[p] = key;
                    l.idx[p] = at[e] + j;
                    l.val[p] = v;
                }
            }
        }
    }
    __syncthreads();
    return l.n;
}

// A pass that makes the entries above `bound` the candidates one by one, for
// the rare rows whose chunks do not fit the queue.
template <typename T, typename L>
__device__ __forceinline__ int list_above(const T *x, int i0, int i1, uint32_t bound, L &l)
{
#pragma unroll 1
    for (int i = i0 + threadIdx.x; i < i1; i += L::THREADS) {
        const float v = (float)x[i];
        const uint32_t key = Key<T>::of(v);
        if (key > bound) {
            const int p = atomicAdd(&l.n, 1);
            if (p < L::CAP) {
                l.key[p] = key;
                l.idx[p] = i;
                l.val[p] = v;
            }
        }
    }
    __syncthreads();
    return l.n;
}

// The first `need` entries with the key `tie`, in index order, join the
// candidates; the pass ends where they are complete.
template <typename T, typename L>
__device__ __forceinline__ void collect_ties(const T *x, int i0, int i1, uint32_t tie, int need, L &l)
{
    constexpr int EPC = Chunk<T>::EPC, STEP = L::THREADS * EPC;
    const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
    const float t = Key<T>::value(tie);
    const bool nan = tie == Key<T>::NAN_KEY;
    for (int b0 = i0; b0 < i1 && need > 0; b0 += STEP) {
        const int at = b0 + threadIdx.x * EPC;
        const Chunk<T> k = load_row(x, at, i1);
        uint32_t mask = 0;
#pragma unroll
        for (int j = 0; j < EPC; j++)
            mask |= (uint32_t)(at + j < i1 && (nan ? k.get(j) != k.get(j) : k.get(j) == t)) << j;
        int place = __popc(mask);
#pragma unroll
        for (int o = 1; o < WAVE; o <<= 1) {
            const int v = __shfl_up(place, o);
            place += lane >= o ? v : 0;
        }
        if (lane == WAVE - 1)
            l.wave[wave] = place;
        __syncthreads();
        place -= __popc(mask);
        int total = 0;
#pragma unroll 1
        for (int w = 0; w < L::THREADS / WAVE; w++) {
            place += w < wave ? l.wave[w] : 0;
            total += l.wave[w];
        }
#pragma unroll
        for (int j = 0; j < EPC; j++)
            if ((mask >> j & 1) && place++ < need) {
                const int p = atomicAdd(&l.n, 1);
                l.key[p] = tie;
                l.idx[p] = at + j;
                l.val[p] = k.get(j);
            }
        need -= total;
        __syncthreads();
    }
}

// The k-th largest key of a whole row by counting, a bit a pass.
template <typename T, typename L>
__device__ __forceinline__ uint32_t kth_of_row(const T *x, int i0, int i1, int k, L &l)
{
    uint32_t cut = 0;
#pragma unroll 1
    for (int bit = Key<T>::BITS - 1; bit >= 0; bit--) {
        const uint32_t t = cut | 1u << bit;
        int c = 0;
        for (int i = i0 + threadIdx.x; i < i1; i += L::THREADS)
            c += Key<T>::of((float)x[i]) >= t;
        if (threadIdx.x == 0)
            l.n = 0;
        __syncthreads();
        atomicAdd(&l.n, c);
        __syncthreads();
        cut = l.n >= k ? t : cut;
        __syncthreads();
    }
    return cut;
}

// Leaves in `l` the min(k, i1 - i0) largest of elements [i0, i1) of a row (at
// least one), in index order, and the softmax sums of the thread's share in
// `sm`.  A first block gives a bound that at least k entries reach, the k-th
// largest of the threads' own maxima; one pass then collects what is above it,
// a few times k entries for values in no particular order.  Should they not
// fit (values that rise along the row), the same bound is taken from the
// threads' maxima over the whole row, and should those above it still not fit,
// the k-th key itself is counted out.  Fewer than k above the bound (many
// equal values, masked rows): the missing ones equal it.
template <typename T, typename L>
__device__ __forceinline__ void row_top(const T *x, int i0, int i1, int k, float c, L &l, Softmax &sm)
{
    constexpr int EPC = Chunk<T>::EPC, STEP = L::THREADS * EPC;
    const int want = k < i1 - i0 ? k : i1 - i0;
    if (threadIdx.x == 0)
        l.n = 0;
    // short: all are candidates, also where fewer than k threads have entries
    const int share = (i1 - i0 + EPC - 1) / EPC;
    if (i1 - i0 <= 512 || share < k) {
        for (int i = i0 + threadIdx.x * EPC; i < i1; i += STEP) {
            const Chunk<T> e = load_row(x, i, i1);
            bool odd;
            float top;
            sm.add<T, 1>(&e, c, odd, &top);
#pragma unroll
            for (int j = 0; j < EPC; j++)
                if (i + j < i1) {
                    l.key[i - i0 + j] = Key<T>::of(e.get(j));
                    l.idx[i - i0 + j] = i + j;
                    l.val[i - i0 + j] = e.get(j);
                }
        }
        __syncthreads();
        prune<T, L>(l, i1 - i0, want);
        return;
    }
    const int at = i0 + threadIdx.x * EPC;
    // (a loop: the sample's chunks held at once cost registers, 434 us)
    float top = NEG_INF;
    bool nan = false;
#pragma unroll 2
    for (int u = 0; u < L::U; u++) {
        const Chunk<T> e = load_row(x, at + u * STEP, i1);
        float t = max2(e.get(0), e.get(1)), a = e.get(0) + e.get(1);
#pragma unroll
        for (int j = 2; j < EPC; j += 2) {
            t = max3(t, e.get(j), e.get(j + 1));
            a += e.get(j) + e.get(j + 1);
        }
        if (a != a)
#pragma unroll
            for (int j = 0; j < EPC; j++)
                nan |= e.get(j) != e.get(j);
        top = max2(top, t);
    }
    l.best[threadIdx.x] = at >= i1 ? 0u : nan ? Key<T>::NAN_KEY : Key<T>::of(top); // 0: no entries
    // A quarter more than k may reach it, or, where there are no more threads
    // than that, just k: 4096 rows of 8192 bf16, 256 threads, k = 204, 205, 256
    // 91, 89, 262 us (a quarter more for all: 90, 129, 571, the last two with a
    // bound of 0 and so with all entries for candidates).
    uint32_t bound = kth_key<Key<T>::BITS>(l, l.best, L::THREADS, k, L::THREADS > k + k / 4 ? k / 4 : EXACT_KEY);
    __syncthreads();
    int q = stream_above<T, L>(x, i0, i1, bound, c, l, sm);
    int n = q > L::QUEUE ? L::CAP + 1 : take_queued<T, L>(q, i1, bound, l);
#pragma unroll 1
    for (int again = 0; again < 2 && n > L::CAP; again++) {
        __syncthreads();
        if (again == 0) {
            l.best[threadIdx.x] = Key<T>::of(sm.m); // of the numbers: FA_MAX_TOP threads or more have some
            bound = max(bound, kth_key<Key<T>::BITS>(l, l.best, L::THREADS, k, EXACT_KEY));
        } else {
            bound = kth_of_row<T, L>(x, i0, i1, k, l);
        }
        __syncthreads();
        if (threadIdx.x == 0)
            l.n = 0;
        __syncthreads();
        n = list_above<T, L>(x, i0, i1, bound, l);
    }
    if (n < want) {
        __syncthreads();
        collect_ties<T, L>(x, i0, i1, bound, want - n, l);
        n = want;
    }
    prune<T, L>(l, n, want);
}

__device__ __forceinline__ float *piece_vals(const TopRowsArgs &p, int pieces)
{
    return reinterpret_cast<float *>(static_cast<TopPiece *>(p.ws) + p.R * pieces);
}

// A workgroup per row (pieces = 1) or per piece of a row; a piece's results go
// to the workspace, unused places with index -1.  Bound by the vector units,
// which issue in 76% of the cycles: 4096 x 128256 bf16, k = 64, in 247 us (1.05
// GB, 4.3 TB/s, whatever of it the caches hold), with 12 vector instructions a
// logit: the pass's five, a quarter of the row sampled before it, the selection,
// and 8 spilled registers (69 MB of writes).
template <typename T, typename L>
__global__ __launch_bounds__(L::THREADS, 8) void top_rows_kernel(TopRowsArgs p, int pieces, int64_t len)
{
    constexpr int THREADS = L::THREADS;
    __shared__ L l;
    const float c = p.inv_tau * LOG2E;
    for (int64_t w = blockIdx.x; w < p.R * pieces; w += gridDim.x) {
        const int64_t r = w / pieces;
        const int i0 = (int)((w % pieces) * len), i1 = (int)(i0 + len < p.V ? i0 + len : p.V);
        const T *x = static_cast<const T *>(p.x) + r * p.ldx;
        Softmax sm;
        int n = 0;
        if (p.k > 0) {
            row_top<T, L>(x, i0, i1, p.k, c, l, sm);
            n = l.n;
        } else {
            bool special;
            float top;
            for (int i = i0 + threadIdx.x * Chunk<T>::EPC; i < i1; i += THREADS * Chunk<T>::EPC) {
                const Chunk<T> e = load_row(x, i, i1);
                sm.add<T, 1>(&e, c, special, &top);
            }
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
// are added in piece order.  Bound by latency: about three eighths of the 23.4
// us of a call (one row of 151936 fp32, 32 pieces, k = 32).
using TopJoin = TopLds<512, 1, 4096, 1>;

template <typename T> __global__ __launch_bounds__(TopJoin::THREADS) void top_join_kernel(TopRowsArgs p, int pieces)
{
    __shared__ TopJoin l;
    const float c = p.inv_tau * LOG2E;
    for (int64_t r = blockIdx.x; r < p.R; r += gridDim.x) {
        const float *val = piece_vals(p, pieces) + r * pieces * p.k;
        const int32_t *idx = reinterpret_cast<const int32_t *>(piece_vals(p, pieces) + p.R * pieces * p.k) + r * pieces * p.k;
        if (threadIdx.x == 0)
            l.n = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < pieces * p.k; j += TopJoin::THREADS) {
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
            const Softmax row = join_pieces(t, pieces, c);
            if (threadIdx.x == 0)
                p.lse[r] = lse_of(row.m, row.s, p.inv_tau);
        }
        __syncthreads();
        prune<T, TopJoin>(l, l.n, p.k);
        for (int j = threadIdx.x; j < p.k; j += TopJoin::THREADS) {
            p.idx[r * p.k + j] = l.idx[j];
            p.val[r * p.k + j] = l.val[j];
        }
        __syncthreads();
    }
}

// How rows are split: while there are fewer rows than CUs, into pieces of at
// least SPLIT_MIN bytes, at most `most`; and into `least` in any case, while
// `most` allows.
constexpr int64_t SPLIT_MIN = 16384;

void split_rows(int64_t R, int64_t V, size_t es, int64_t most, int64_t least, int cus, int &pieces, int64_t &len)
{
    const int64_t unit = 64; // elements: pieces start on a vector of an aligned row
    int64_t s = R > 0 && R < cus ? (2 * cus + R - 1) / R : 1;
    s = std::max(std::min(s, V * (int64_t)es / SPLIT_MIN), least);
    s = std::max<int64_t>(1, std::min<int64_t>(s, std::min<int64_t>(most, SPLIT_MAX)));
    len = (((V + s - 1) / s + unit - 1) / unit) * unit;
    len = std::max(len, unit);
    pieces = (int)std::max<int64_t>(1, (V + len - 1) / len);
}

// ------------------------------------------------------------ distillation
constexpr int DI_SMALL = 256, DI_LARGE = 512;
constexpr int LISTS_LDS = 162816; // of a CU's 160 KB, 1 KB left to the kernel's own
constexpr int DI_KEEP_SMALL = 4, DI_KEEP_LARGE = 8; // a small row is kept whole
constexpr int64_t DI_SMALL_BYTES = 16384; // rows up to this take the small workgroup

// LDS of one row's lists, sized by the entries a row can have: per client its
// numbers, per entry its probability and its slot, a table with a slot for
// each distinct index (open addressing, at most four fifths full), and chains
// of the slots whose indices fall in the same 2^shift chunks of the piece.
struct Lists {
    int *len;     // [clients] entries in use; 0: the client did not send the row
    float *mass;  // [clients] sum_j q_cj
    float *kl;    // [clients] sum_j q_cj log q_cj; from finish_kl on tau / 4 sum_j q_cj (log q_cj - log p_j)
    float *share; // [clients] n_c over the sum of n of the clients that sent the row
    float *q;     // [entries]
    float *z;     // [entries] the listed logits, for the loss
    short *slot;  // [entries] -1: outside the piece
    int *index;   // [slots] -1: free
    float *sum;   // [slots]
    short *next;  // [slots] the chain's next slot + 1, or 0
    int *head;    // [heads] its first slot + 1, or 0
    int slots, heads, shift;

    static constexpr int MAX_HEADS = 8192;

    static __host__ __device__ int slots_for(int entries)
    {
        int n = 64;
        while (n < entries + entries / 4)
            n *= 2;
        return n;
    }
    static __host__ __device__ int shift_for(int chunks)
    {
        int s = 0;
        while (((chunks - 1) >> s) >= MAX_HEADS)
            s++;
        return s;
    }
    static __host__ size_t bytes(int clients, int entries, int chunks, bool loss)
    {
        const size_t heads = (size_t)((chunks - 1) >> shift_for(chunks)) + 1, slots = slots_for(entries);
        return (4 * (size_t)clients + (loss ? 2 : 1) * (size_t)entries + 2 * slots + heads) * 4 + (slots + entries) * 2;
    }
    __device__ __forceinline__ void place(char *at, int clients, int entries, int chunks, bool loss)
    {
        slots = slots_for(entries);
        shift = shift_for(chunks);
        heads = ((chunks - 1) >> shift) + 1;
        index = reinterpret_cast<int *>(at);
        sum = reinterpret_cast<float *>(index + slots);
        head = reinterpret_cast<int *>(sum + slots);
        q = reinterpret_cast<float *>(head + heads);
        z = q + entries;
        len = reinterpret_cast<int *>(loss ? z + entries : z);
        mass = reinterpret_cast<float *>(len + clients);
        kl = mass + clients;
        share = kl + clients;
        next = reinterpret_cast<short *>(share + clients);
        slot = next + slots;
    }
    // The slot of index i, made and chained to its chunk if need be.  There are
    // more slots than entries, so a free one, or the index's own, comes within
    // one round.
    __device__ __forceinline__ int insert(int i, int chunk)
    {
        int s = ((uint32_t)i * 0x9E3779B1u >> 7) & (slots - 1);
        for (int tries = 0; tries < slots; tries++) {
            const int was = atomicCAS(&index[s], -1, i);
            if (was == i)
                break;
            if (was == -1) {
                next[s] = (short)atomicExch(&head[chunk >> shift], s + 1);
                break;
            }
            s = (s + 1) & (slots - 1);
        }
        return s;
    }
};

// The row's lists: q_cj = exp(v/tau - L_c) and what is summed over them; with
// LOSS the listed logits, with `grad` also each index in [i0, i1) once, with
// sum_c w_c q_c added up in client order.  One wavefront a client.  A list is used up to its first negative
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
        for (int i = threadIdx.x; i < l.heads; i += THREADS)
            l.head[i] = 0;
        __syncthreads();
    }
    for (int c = threadIdx.x / WAVE; c < p.clients; c += THREADS / WAVE) {
        const int k = p.k[c], at = p.first[c];
        const int32_t *idx = p.idx[c] + r * k;
        const float *val = p.val[c] + r * k;
        const float given = p.has_tlse ? p.tlse[c][r] : 0.f;
        constexpr int PER = FA_MAX_TOP / WAVE;
        int32_t ix[PER];
        float v[PER];
#pragma unroll
        for (int e = 0; e < PER; e++) {
            const int j = e * WAVE + lane;
            ix[e] = j < k ? idx[j] : -1;
            v[e] = j < k ? val[j] : NEG_INF;
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
                m = fmaxf(m, v[e]);
            }
        }
        if (__ballot(bad)) {
            if (lane == 0 && p.err)
                *p.err = FA_ERR_INDEX;
            len = 0;
        }
        m = wave_max(m);
        // the largest value is taken off before the temperature, so the
        // exponents carry no rounding of an offset that the list has
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < PER; e++)
            if (e * WAVE + lane < len)
                s += v[e] == NEG_INF ? 0.f : expf((v[e] - m) * p.inv_tau);
        s = wave_sum(s);
        if (m == NEG_INF && s == 0.f)
            len = 0; // nothing, or only -inf
        const float base = p.has_tlse ? 0.f : m, L = p.has_tlse ? given : logf(s);
        float mass = 0.f, kl = 0.f;
#pragma unroll
        for (int e = 0; e < PER; e++) {
            const int j = e * WAVE + lane;
            if (j >= len)
                continue;
            const float lq = __builtin_fmaf(v[e] - base, p.inv_tau, -L);
            const float q = expf(lq);
            mass += q;
            if (LOSS) {
                kl += q != 0.f ? q * lq : 0.f;
                l.z[at + j] = (float)z[ix[e]];
            }
            if (LOSS || grad)
                l.q[at + j] = q;
            if (grad)
                l.slot[at + j] = (short)(ix[e] >= i0 && ix[e] < i1 ? l.insert(ix[e], (ix[e] - i0) / Chunk<T>::EPC) : -1);
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

// l.kl = tau / 4 sum_j q_cj (log q_cj - log p_j) with the row's maximum and sum t:
//     tau log p_j = (z_j - max) - tau log s,
// where the maximum is taken off first, so that the difference holds whatever
// the row's offset is, and not divided by tau, which might pass fp32 where its
// product with tau does not; as neither does a quarter of the type's lowest
// value.  Each lane has the entries that it stored.
template <int THREADS> __device__ __forceinline__ void finish_kl(const DistillArgs &p, const Softmax &t, Lists &l)
{
    const int lane = threadIdx.x % WAVE;
    const float log_s = logf(t.s);
    for (int c = threadIdx.x / WAVE; c < p.clients; c += THREADS / WAVE) {
        float s = 0.f;
        for (int j = p.first[c] + lane; j < p.first[c] + l.len[c]; j += WAVE)
            s += l.q[j] != 0.f ? l.q[j] * (0.25f * l.z[j] - 0.25f * t.m) : 0.f;
        s = wave_sum(s);
        if (lane == 0)
            l.kl[c] = __builtin_fmaf(0.25f * p.tau, __builtin_fmaf(log_s, l.mass[c], l.kl[c]), -s);
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
        // past the caches, which then keep more of z for its second reading:
        // 350 -> 333 us (2048 rows of 128256 bf16, 8 clients)
        typedef uint32_t unaligned __attribute__((ext_vector_type(4), aligned(2)));
        unaligned v16;
        __builtin_memcpy(&v16, e, 16);
        __builtin_nontemporal_store(v16, reinterpret_cast<unaligned *>(x + i));
    } else {
#pragma unroll
        for (int j = 0; j < EPC; j++)
            if (i + j < end)
                x[i + j] = e[j];
    }
}

// Where a row's normaliser comes from.
enum { LSE_COMPUTE = 0, LSE_PIECES = 1, LSE_GIVEN = 2 };

// A workgroup per row, or per piece of a row's gradient.  LOSS: writes loss
// and lse (piece 0 does).  KEEP: chunks of the row that each thread keeps in
// registers from the softmax's pass for the gradient's.  Loss of 1024 x 151936
// bf16, an eighth of them of weight 0, one list a row, 60 us (272 MB, 4.5 TB/s;
// 53 of inputs that the last-level cache holds in part): all rows are resident
// at once, and CUs with four live rows end after those with three.  Loss and
// gradient of 2048 x 128256, an eighth of weight 0, with 8 lists 244 us (0.99
// GB, 4.1 TB/s; vector units 53% busy): half of each row is read twice.
// Gradient of 1000 x 32003 fp32 with 16 lists of 100 in 84 us (66 of inputs in
// the last-level cache): its lists, read before the row, cost about 30, which
// the two workgroups that 62 KB of lists leave a CU do not hide.
template <typename T, int THREADS, bool LOSS, int FROM, int KEEP>
__global__ __launch_bounds__(THREADS, KEEP ? 4 : 1) void distill_kernel(DistillArgs p, int grad_pieces, int64_t len, int stat_pieces)
{
    constexpr int EPC = Chunk<T>::EPC, STEP = THREADS * EPC;
    static_assert(KEEP % 2 == 0 && (KEEP == 0 || FROM == LSE_COMPUTE), "pairs, and of the pass that reads the row");
    extern __shared__ __attribute__((aligned(16))) char dynamic[];
    __shared__ float fl[THREADS / WAVE];
    Lists l;
    l.place(dynamic, p.clients, p.first[p.clients], p.dz ? (int)((len + EPC - 1) / EPC) : 1, LOSS);
    const float c2 = p.inv_tau * LOG2E;
    for (int64_t w = blockIdx.x; w < p.R * grad_pieces; w += gridDim.x) {
        const int64_t r = w / grad_pieces;
        const int i0 = (int)((w % grad_pieces) * len), i1 = (int)(i0 + len < p.V ? i0 + len : p.V);
        const bool first = i0 == 0;
        const T *z = static_cast<const T *>(p.z) + r * p.ldz;
        T *dz = p.dz ? static_cast<T *>(p.dz) + r * p.lddz : nullptr;
        const float g = p.row_weight ? p.row_weight[r] : 1.f;
        float lse = 0.f, M = 0.f, kl = 0.f;
        Softmax t;         // the row's, unless its stored normaliser serves
        bool stored = false;
        bool sent = false;
        Chunk<T> keep[KEEP > 0 ? KEEP : 1];
        if (g != 0.f) {
#pragma unroll
            for (int u = 0; u < KEEP; u++) // on their way while the lists are read
                keep[u] = load_row(z, threadIdx.x * EPC + u * STEP, (int)p.V);
            load_lists<T, THREADS, LOSS>(p, r, z, i0, i1, dz != nullptr, l);
            if (FROM == LSE_COMPUTE) {
#pragma unroll
                for (int u = 0; u < KEEP; u += 2) {
                    bool special;
                    float tops[2];
                    t.add<T, 2>(keep + u, c2, special, tops);
                }
                t = row_softmax<T, THREADS>(z, KEEP * STEP, (int)p.V, c2, fl, t);
            } else if (FROM == LSE_PIECES) {
                t = join_pieces(static_cast<const TopPiece *>(p.ws) + r * stat_pieces, stat_pieces, c2);
            } else {
                lse = p.lse ? p.lse[r] : NEG_INF; // none where V is 0
                stored = !lse_too_coarse(lse);
                if (!stored && stat_pieces > 0)
                    t = join_pieces(static_cast<const TopPiece *>(p.ws) + r * stat_pieces, stat_pieces, c2);
                else if (!stored)
                    t = row_by_pieces<T, THREADS>(z, (int)p.V, (int)len, grad_pieces, c2, fl);
            }
            if (FROM != LSE_GIVEN)
                lse = lse_of(t.m, t.s, p.inv_tau);
            if (LOSS)
                finish_kl<THREADS>(p, t, l);
            if (stored || t.m != NEG_INF || t.s != 0.f) // anything but -inf in the row
                for (int c = 0; c < p.clients; c++)
                    if (l.len[c]) {
                        M = __builtin_fmaf(l.share[c], l.mass[c], M);
                        if (LOSS)
                            kl = __builtin_fmaf(l.share[c], l.kl[c], kl);
                        sent = true;
                    }
        }
        if (LOSS && first && threadIdx.x == 0) {
            // kl is tau / 4 times it: tau^2 may pass fp32 where tau kl does not
            p.loss[r] = sent ? g * p.tau * kl * 4.f : 0.f;
            if (p.lse)
                p.lse[r] = lse;
        }
        if (dz && !sent) {
            const float zero[EPC] = {};
            for (int i = i0 + threadIdx.x * EPC; i < i1; i += THREADS * EPC)
                store_row(dz, i, i1, zero);
        } else if (dz) {
            // One pass that also takes off the listed entries' shares, found
            // through their chunk's chain.  (Gathering their logits before the
            // pass and writing their places after it touched most lines of a
            // row twice more: 93 us where this takes 77, 1000 rows of
            // 32003 fp32, 16 clients of 100.)
            const float gt = g * p.tau, gm = gt * M;
            // m p_i = scale * 2^(z c2 - base).  From the row's maximum and sum
            // rather than the normaliser, whose rounding relative to max / tau
            // would be a factor of every p.  The fused form's base is rounded,
            // and what that left off goes into the scale.
            const float top = stored ? lse : t.m, unit = stored ? LOG2E : c2, base = top * unit;
            const bool fused = fabsf(base) <= FUSED_UP_TO;
            const float rest = fused ? __builtin_amdgcn_exp2f(__builtin_fmaf(-top, unit, base)) : 1.f;
            const float scale = (stored ? gm : gm / t.s) * rest;
            const auto grad = [&](const Chunk<T> &k, int i) {
                float v[EPC];
                if (fused) {
#pragma unroll
                    for (int j = 0; j < EPC; j++)
                        v[j] = scale * __builtin_amdgcn_exp2f(__builtin_fmaf(k.get(j), c2, -base));
                } else {
#pragma unroll
                    for (int j = 0; j < EPC; j++)
                        v[j] = scale * __builtin_amdgcn_exp2f((k.get(j) - top) * c2);
                }
                for (int h = l.head[(uint32_t)(i - i0) / EPC >> l.shift]; h;) {
                    const int at = l.index[h - 1] - i;
                    const float Q = gt * l.sum[h - 1];
                    h = l.next[h - 1];
#pragma unroll
                    for (int j = 0; j < EPC; j++)
                        v[j] -= at == j ? Q : 0.f;
                }
                store_row(dz, i, i1, v);
            };
#pragma unroll
            for (int u = 0; u < KEEP; u++) {
                if (threadIdx.x * EPC + u * STEP < i1)
                    grad(keep[u], threadIdx.x * EPC + u * STEP);
                __builtin_amdgcn_sched_barrier(0); // one chunk's values at a time
            }
#pragma unroll 2
            for (int i = i0 + KEEP * STEP + threadIdx.x * EPC; i < i1; i += STEP)
                grad(load_row(z, i, i1), i);
        }
        __syncthreads();
    }
}

// Softmax sums of the pieces of each row.  Rows of weight 0 are not read, nor,
// in the gradient alone (`stored`: its normalisers), those that need no sums.
// 4 us for 3 rows of 128256 bf16 in 15 pieces each.
template <typename T, int THREADS>
__global__ __launch_bounds__(THREADS) void row_stats_kernel(DistillArgs p, int pieces, int64_t len, const float *stored)
{
    __shared__ float fl[THREADS / WAVE];
    for (int64_t w = blockIdx.x; w < p.R * pieces; w += gridDim.x) {
        const int64_t r = w / pieces;
        const int i0 = (int)((w % pieces) * len), i1 = (int)(i0 + len < p.V ? i0 + len : p.V);
        if ((p.row_weight && p.row_weight[r] == 0.f) || (stored && !lse_too_coarse(stored[r])))
            continue;
        const T *z = static_cast<const T *>(p.z) + r * p.ldz;
        const Softmax t = row_softmax<T, THREADS>(z, i0, i1, p.inv_tau * LOG2E, fl);
        if (threadIdx.x == 0)
            static_cast<TopPiece *>(p.ws)[w] = TopPiece{t.m, t.s};
        __syncthreads();
    }
}

template <typename T, int THREADS, bool LOSS, int FROM, int KEEP = 0>
hipError_t run_distill(const DistillArgs &a, int pieces, int64_t len, int stat_pieces, int cus, hipStream_t s)
{
    const unsigned grid = (unsigned)std::min<int64_t>(a.R * pieces, (int64_t)cus * 16);
    // without a gradient there is no table
    const int64_t chunks = a.dz ? (len + Chunk<T>::EPC - 1) / Chunk<T>::EPC : 1;
    const size_t lds = Lists::bytes(a.clients, a.first[a.clients], (int)chunks, LOSS);
    static_assert((4 * FA_MAX_CLIENTS + (2 + 4) * FA_MAX_LIST_ENTRIES + Lists::MAX_HEADS) * 4 + 3 * FA_MAX_LIST_ENTRIES * 2 <= LISTS_LDS,
                  "the largest lists fit in LDS, with two slots an entry");
    if (lds > 64 << 10) { // more than a kernel gets without asking
        static DeviceOnce limit;
        int device = 0;
        hipError_t e = hipGetDevice(&device);
        if (e == hipSuccess)
            e = (hipError_t)limit.run(device, [] {
                return (int)hipFuncSetAttribute(reinterpret_cast<const void *>(&distill_kernel<T, THREADS, LOSS, FROM, KEEP>),
                                                hipFuncAttributeMaxDynamicSharedMemorySize, LISTS_LDS);
            });
        if (e != hipSuccess)
            return e;
    }
    distill_kernel<T, THREADS, LOSS, FROM, KEEP><<<grid, THREADS, lds, s>>>(a, pieces, len, stat_pieces);
    return hipGetLastError();
}

template <typename T> hipError_t distill_of(const DistillArgs &a, bool loss, int cus, hipStream_t s)
{
    int pieces;
    int64_t len;
    split_rows(a.R, a.V, sizeof(T), SPLIT_MAX, 1, cus, pieces, len);
    const bool small = a.V * (int64_t)sizeof(T) <= DI_SMALL_BYTES;
    const auto stats = [&](const float *stored) {
        row_stats_kernel<T, DI_LARGE><<<(unsigned)(a.R * pieces), DI_LARGE, 0, s>>>(a, pieces, len, stored);
        return hipGetLastError();
    };
    if (!loss) {
        if (small)
            return run_distill<T, DI_SMALL, false, LSE_GIVEN>(a, pieces, len, 0, cus, s);
        if (pieces == 1 || a.dz != a.z)
            return run_distill<T, DI_LARGE, false, LSE_GIVEN>(a, pieces, len, 0, cus, s);
        // in place: what a piece may need of the whole row is read before
        // others overwrite it
        const hipError_t e = stats(a.lse);
        return e != hipSuccess ? e : run_distill<T, DI_LARGE, false, LSE_GIVEN>(a, pieces, len, pieces, cus, s);
    }
    if (pieces == 1) {
        if (!a.dz)
            return small ? run_distill<T, DI_SMALL, true, LSE_COMPUTE>(a, 1, len, 0, cus, s)
                         : run_distill<T, DI_LARGE, true, LSE_COMPUTE>(a, 1, len, 0, cus, s);
        return small ? run_distill<T, DI_SMALL, true, LSE_COMPUTE, DI_KEEP_SMALL>(a, 1, len, 0, cus, s)
                     : run_distill<T, DI_LARGE, true, LSE_COMPUTE, DI_KEEP_LARGE>(a, 1, len, 0, cus, s);
    }
    hipError_t e = stats(nullptr);
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

// The workgroups of the top logits.  Rows of up to 16 KB take the small one,
// whose queue holds the whole row.  Four workgroups of the large one fit a
// CU and hide each other's selection: 263 us against 334 us with two of twice
// the threads and the queue (4096 rows of 128256 bf16, k = 64).  Its sample of 8
// chunks a thread against 4: 263 us either way at k = 64, 292 against 337 at
// k = 128.  A pass finds about k times the row's length over the sample's, and
// top_longest counts a quarter more; longer rows are split, and where the
// pieces are as many as the join takes, another pass may follow.
using TopSmall = TopLds<256, 1024, 2048, 4>;
using TopLarge = TopLds<512, 1536, 2560, 8>;
constexpr int64_t TOP_SMALL_BYTES = 16384;

// The longest piece of a row whose candidates the queue is expected to hold.
int64_t top_longest(int64_t k, size_t es)
{
    using L = TopLarge;
    return (int64_t)L::QUEUE * L::THREADS * L::U * 16 / (int64_t)es * 4 / (5 * std::max<int64_t>(k, 1));
}

void split_top_rows(int64_t R, int64_t V, int64_t k, size_t es, int cus, int &pieces, int64_t &len)
{
    // with few rows the pieces' entries are kept to about two a thread of the
    // join, which is as long as a piece takes
    const int64_t least = V / top_longest(k, es) + 1, kk = std::max<int64_t>(k, 1);
    const int64_t most = std::min<int64_t>(TopJoin::CAP / kk, std::max({2 * TopJoin::THREADS / kk, least, (int64_t)8}));
    split_rows(R, V, es, most, least, cus, pieces, len);
}

template <typename T> hipError_t top_rows_of(const TopRowsArgs &a, int cus, hipStream_t s)
{
    int pieces;
    int64_t len;
    split_top_rows(a.R, a.V, a.k, sizeof(T), cus, pieces, len);
    const unsigned grid = (unsigned)std::min<int64_t>(a.R * pieces, (int64_t)cus * 16);
    if (len * (int64_t)sizeof(T) <= TOP_SMALL_BYTES)
        top_rows_kernel<T, TopSmall><<<grid, TopSmall::THREADS, 0, s>>>(a, pieces, len);
    else
        top_rows_kernel<T, TopLarge><<<grid, TopLarge::THREADS, 0, s>>>(a, pieces, len);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || pieces == 1)
        return e;
    top_join_kernel<T><<<(unsigned)std::min<int64_t>(a.R, (int64_t)cus * 16), TopJoin::THREADS, 0, s>>>(a, pieces);
    return hipGetLastError();
}

} // namespace

size_t top_rows_workspace_bytes(int dt, int64_t R, int64_t V, int64_t k, int cus)
{
    int pieces;
    int64_t len;
    split_top_rows(R, V, k, dt == FA_BF16 ? 2 : 4, cus, pieces, len);
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
    split_rows(R, V, dt == FA_BF16 ? 2 : 4, SPLIT_MAX, 1, cus, pieces, len);
    return pieces > 1 ? (size_t)(R * pieces) * sizeof(TopPiece) : 0;
}

hipError_t launch_distill(const DistillArgs &a, int dt, bool loss, int cus, hipStream_t s)
{
    if (a.R == 0)
        return hipSuccess;
    return dt == FA_BF16 ? distill_of<__bf16>(a, loss, cus, s) : distill_of<float>(a, loss, cus, s);
}

} // namespace fa
