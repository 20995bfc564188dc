// A client's top logits of each row (token), and the loss and gradient of a
// student distilled from several clients' top logits.
#include "learn_internal.h"

#include <algorithm>

namespace fa {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int WAVE = 64;
constexpr float NEG_INF = -__builtin_inff();

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

template <int THREADS> __device__ __forceinline__ int block_count(int v, int *lds)
{
#pragma unroll
    for (int o = WAVE / 2; o > 0; o >>= 1)
        v += __shfl_xor(v, o);
    if (threadIdx.x % WAVE == 0)
        lds[threadIdx.x / WAVE] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < THREADS / WAVE; w++)
        v += lds[w];
    __syncthreads();
    return v;
}

// Unsigned keys in the order of the values: NaN of either sign highest, then
// descending numbers, -0 and +0 equal.
__device__ __forceinline__ uint32_t key_of(float x)
{
    if (x != x)
        return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Max and sum of exp(x inv_tau - max) of a row, to every thread.
template <typename T, int THREADS>
__device__ __forceinline__ void row_stats(const T *x, int64_t V, float inv_tau, float *lds, float &mx, float &sum)
{
    float m = NEG_INF;
    for (int64_t i = threadIdx.x; i < V; i += THREADS)
        m = fmaxf(m, (float)x[i] * inv_tau);
    // fmaxf drops NaN: a NaN still enters the sum below
    mx = block_max<THREADS>(m, lds);
    float s = 0.f;
    for (int64_t i = threadIdx.x; i < V; i += THREADS) {
        const float y = (float)x[i] * inv_tau;
        s += y == NEG_INF ? 0.f : expf(y - mx);
    }
    sum = block_sum<THREADS>(s, lds);
}

// ------------------------------------------------------------ top logits
constexpr int TR_THREADS = 1024;

// One workgroup a row.  The k-th largest key is found bit by bit by counting;
// then one ordered pass writes the entries above it and, in index order, as
// many equal to it as are still wanted.
template <typename T> __global__ __launch_bounds__(TR_THREADS) void top_rows_kernel(TopRowsArgs p)
{
    __shared__ float fl[TR_THREADS / WAVE];
    __shared__ int il[TR_THREADS / WAVE];
    __shared__ int scan[TR_THREADS / WAVE][2];
    for (int64_t r = blockIdx.x; r < p.R; r += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + r * p.ldx;
        if (p.lse) {
            float mx, sum;
            row_stats<T, TR_THREADS>(x, p.V, p.inv_tau, fl, mx, sum);
            if (threadIdx.x == 0)
                p.lse[r] = mx == NEG_INF && sum == 0.f ? NEG_INF : mx + logf(sum);
        }
        uint32_t cut = 0; // largest key with at least k keys at or above it
        for (int bit = 31; bit >= 0; bit--) {
            const uint32_t t = cut | (1u << bit);
            int c = 0;
            for (int64_t i = threadIdx.x; i < p.V; i += TR_THREADS)
                c += key_of((float)x[i]) >= t;
            if (block_count<TR_THREADS>(c, il) >= p.k)
                cut = t;
        }
        int above = 0;
        for (int64_t i = threadIdx.x; i < p.V; i += TR_THREADS)
            above += key_of((float)x[i]) > cut;
        const int ties = p.k - block_count<TR_THREADS>(above, il);
        // ordered write: positions by counting entries before each one
        int done_gt = 0, done_eq = 0;
        const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
        for (int64_t i0 = 0; i0 < p.V; i0 += TR_THREADS) {
            const int64_t i = i0 + threadIdx.x;
            float v = 0.f;
            bool gt = false, eq = false;
            if (i < p.V) {
                v = (float)x[i];
                const uint32_t key = key_of(v);
                gt = key > cut;
                eq = key == cut;
            }
            const uint64_t bg = __ballot(gt), be = __ballot(eq);
            if (lane == 0) {
                scan[wave][0] = __popcll(bg);
                scan[wave][1] = __popcll(be);
            }
            __syncthreads();
            int g = done_gt, e = done_eq;
            for (int w = 0; w < TR_THREADS / WAVE; w++) {
                const int cg = scan[w][0], ce = scan[w][1];
                if (w < wave) {
                    g += cg;
                    e += ce;
                }
                done_gt += cg;
                done_eq += ce;
            }
            const uint64_t before = (1ull << lane) - 1;
            g += __popcll(bg & before);
            e += __popcll(be & before);
            if (gt || (eq && e < ties)) {
                const int at = g + (e < ties ? e : ties);
                p.idx[r * p.k + at] = (int32_t)i;
                p.val[r * p.k + at] = v;
            }
            __syncthreads();
        }
    }
}

// ------------------------------------------------------------ distillation
constexpr int DI_THREADS = 512;
constexpr int DI_MAX_ENTRIES = 4096; // of one row, over all clients

struct Lists {
    int32_t idx[DI_MAX_ENTRIES];
    float q[DI_MAX_ENTRIES];
    int len[FA_MAX_CLIENTS];   // entries in use; 0: the client did not send the row
    float share[FA_MAX_CLIENTS]; // n_c over the sum of n of the clients that did
    float kl[FA_MAX_CLIENTS];
    float mass[FA_MAX_CLIENTS];
};

// The row's lists into LDS: q_cj = exp(v/tau - L_c), each client's mass
// sum_j q_cj and, with LOSS, sum_j q_cj (log q_cj - log p_j).  One wavefront a
// client.  A list is used up to its first negative index; one that is not
// strictly increasing or passes V is left out whole and raises the flag.
template <typename T, bool LOSS>
__device__ __forceinline__ void load_lists(const DistillArgs &p, int64_t r, const T *z, float lse, Lists &l)
{
    const int lane = threadIdx.x % WAVE;
    for (int c = threadIdx.x / WAVE; c < p.clients; c += DI_THREADS / WAVE) {
        const int k = p.k[c], at = p.first[c];
        const int32_t *idx = p.idx[c] + r * k;
        const float *val = p.val[c] + r * k;
        int len = k;
        for (int j0 = 0; j0 < k; j0 += WAVE) {
            const uint64_t b = __ballot(j0 + lane < k && idx[j0 + lane] < 0);
            if (b) {
                len = j0 + __builtin_ctzll(b);
                break;
            }
        }
        bool bad = false;
        float m = NEG_INF, s = 0.f;
        for (int j = lane; j < len; j += WAVE) {
            const int i = idx[j];
            bad |= i >= p.V || (j > 0 && idx[j - 1] >= i);
            l.idx[at + j] = i;
            m = fmaxf(m, val[j] * p.inv_tau);
        }
        if (__ballot(bad)) {
            if (lane == 0 && p.err)
                *p.err = FA_ERR_INDEX;
            len = 0;
        }
        m = wave_max(m);
        for (int j = lane; j < len; j += WAVE) {
            const float y = val[j] * p.inv_tau;
            s += y == NEG_INF ? 0.f : expf(y - m);
        }
        s = wave_sum(s);
        if (m == NEG_INF && s == 0.f)
            len = 0; // nothing, or only -inf
        const float L = p.has_tlse ? p.tlse[c][r] : m + logf(s);
        float mass = 0.f, kl = 0.f;
        for (int j = lane; j < len; j += WAVE) {
            const float lq = val[j] * p.inv_tau - L;
            const float q = expf(lq);
            l.q[at + j] = q;
            mass += q;
            if (LOSS && q != 0.f)
                kl += q * (lq - ((float)z[l.idx[at + j]] * p.inv_tau - lse));
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
    float W = 0.f;
    for (int c = 0; c < p.clients; c++)
        W += l.len[c] ? p.n[c] : 0.f;
    for (int c = threadIdx.x; c < p.clients; c += DI_THREADS)
        l.share[c] = l.len[c] ? p.n[c] / W : 0.f;
    __syncthreads();
}

// Position of index i in client c's list, or -1.
__device__ __forceinline__ int find(const Lists &l, int at, int len, int i)
{
    int lo = 0, hi = len;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (l.idx[at + mid] < i)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo < len && l.idx[at + lo] == i ? lo : -1;
}

// One workgroup a row.
template <typename T, bool LOSS> __global__ __launch_bounds__(DI_THREADS) void distill_kernel(DistillArgs p)
{
    __shared__ Lists l;
    __shared__ float fl[DI_THREADS / WAVE];
    for (int64_t r = blockIdx.x; r < p.R; r += gridDim.x) {
        const T *z = static_cast<const T *>(p.z) + r * p.ldz;
        T *dz = p.dz ? static_cast<T *>(p.dz) + r * p.lddz : nullptr;
        const float g = p.row_weight ? p.row_weight[r] : 1.f;
        float lse = 0.f;
        bool empty = g == 0.f;
        if (LOSS && !empty) {
            float mx, sum;
            row_stats<T, DI_THREADS>(z, p.V, p.inv_tau, fl, mx, sum);
            lse = mx == NEG_INF && sum == 0.f ? NEG_INF : mx + logf(sum);
        } else if (!empty) {
            lse = p.lse[r];
        }
        if (LOSS && threadIdx.x == 0 && p.lse)
            p.lse[r] = lse;
        empty |= lse == NEG_INF;
        float M = 0.f;
        if (!empty) {
            load_lists<T, LOSS>(p, r, z, lse, l);
            float kl = 0.f;
            for (int c = 0; c < p.clients; c++) {
                if (l.len[c]) {
                    M = __builtin_fmaf(l.share[c], l.mass[c], M);
                    kl = __builtin_fmaf(l.share[c], l.kl[c], kl);
                }
            }
            if (LOSS && threadIdx.x == 0)
                p.loss[r] = g * (p.tau * p.tau) * kl;
        } else if (LOSS && threadIdx.x == 0) {
            p.loss[r] = 0.f;
        }
        if (!dz) {
            __syncthreads();
            continue;
        }
        bool sent = false;
        if (!empty)
            for (int c = 0; c < p.clients; c++)
                sent |= l.len[c] != 0;
        if (!sent) {
            for (int64_t i = threadIdx.x; i < p.V; i += DI_THREADS)
                dz[i] = (T)0.f;
            __syncthreads();
            continue;
        }
        // Listed indices: the first client that has an index adds the clients'
        // shares in client order.  Their values are taken from z before the
        // dense pass, as dz may be z, and written after it.
        const float gt = g * p.tau;
        float fix[DI_MAX_ENTRIES / DI_THREADS];
        const int total = p.first[p.clients];
#pragma unroll
        for (int e = 0; e < DI_MAX_ENTRIES / DI_THREADS; e++) {
            const int at = e * DI_THREADS + threadIdx.x;
            fix[e] = 0.f;
            if (at >= total)
                continue;
            int c = 0;
            while (p.first[c + 1] <= at)
                c++;
            if (at - p.first[c] >= l.len[c])
                continue;
            const int i = l.idx[at];
            float Q = l.share[c] * l.q[at];
            bool mine = true;
            for (int o = 0; o < p.clients; o++) {
                if (o == c)
                    continue;
                const int j = find(l, p.first[o], l.len[o], i);
                if (j < 0)
                    continue;
                if (o < c)
                    mine = false;
                else
                    Q = __builtin_fmaf(l.share[o], l.q[p.first[o] + j], Q);
            }
            if (!mine)
                continue;
            const float pr = expf((float)z[i] * p.inv_tau - lse);
            fix[e] = gt * (M * pr - Q);
        }
        __syncthreads();
        for (int64_t i = threadIdx.x; i < p.V; i += DI_THREADS)
            dz[i] = (T)(gt * (M * expf((float)z[i] * p.inv_tau - lse)));
        __syncthreads();
#pragma unroll
        for (int e = 0; e < DI_MAX_ENTRIES / DI_THREADS; e++) {
            const int at = e * DI_THREADS + threadIdx.x;
            if (at >= total)
                continue;
            int c = 0;
            while (p.first[c + 1] <= at)
                c++;
            if (at - p.first[c] >= l.len[c])
                continue;
            const int i = l.idx[at];
            bool mine = true;
            for (int o = 0; o < c; o++)
                mine &= find(l, p.first[o], l.len[o], i) < 0;
            if (mine)
                dz[i] = (T)fix[e];
        }
        __syncthreads();
    }
}

} // namespace

size_t top_rows_workspace_bytes(int, int64_t, int64_t, int64_t, int) { return 0; }

hipError_t launch_top_rows(const TopRowsArgs &a, int dt, int cus, hipStream_t s)
{
    if (a.R == 0)
        return hipSuccess;
    const unsigned grid = (unsigned)std::min<int64_t>(a.R, (int64_t)cus * 16);
    if (dt == FA_BF16)
        top_rows_kernel<__bf16><<<grid, TR_THREADS, 0, s>>>(a);
    else
        top_rows_kernel<float><<<grid, TR_THREADS, 0, s>>>(a);
    return hipGetLastError();
}

size_t distill_workspace_bytes(int, int64_t, int64_t, int) { return 0; }

hipError_t launch_distill(const DistillArgs &a, int dt, bool loss, int cus, hipStream_t s)
{
    if (a.R == 0)
        return hipSuccess;
    const unsigned grid = (unsigned)std::min<int64_t>(a.R, (int64_t)cus * 16);
    if (dt == FA_BF16) {
        if (loss)
            distill_kernel<__bf16, true><<<grid, DI_THREADS, 0, s>>>(a);
        else
            distill_kernel<__bf16, false><<<grid, DI_THREADS, 0, s>>>(a);
    } else {
        if (loss)
            distill_kernel<float, true><<<grid, DI_THREADS, 0, s>>>(a);
        else
            distill_kernel<float, false><<<grid, DI_THREADS, 0, s>>>(a);
    }
    return hipGetLastError();
}

} // namespace fa
