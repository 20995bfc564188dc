// Internal interface between the host library and the kernels of the linear
// layer (linear.hip), the per-row top logits and the distillation loss
// (logits.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fedavg.h"

namespace fa {

// ---------------------------------------------------------------- linear
// out = epilogue(sum_k A(m,k) B(n,k)).  A is stored [M][K] with row pitch lda,
// or [K][M] ("outer": the summed index is the slow one); B likewise with N.
struct GemmArgs {
    const void *a, *b;
    int64_t lda, ldb; // in elements
    int M, N, K;
    float alpha;
    const void *bias; // N values, nullable
    const void *res;  // [M][N], pitch ldr, nullable
    int64_t ldr;
    void *out; // [M][N], pitch ldo
    int64_t ldo;
    void *pre; // [M][N], pitch ldp, nullable: the value before the activation
    int64_t ldp;
    int act;
    bool a_padded; // A's rows are followed by zeros up to whole chunks
};

enum { GEMM_A_OUTER = 1, GEMM_B_OUTER = 2 };

// dz = dy * act'(preact) (dz null: not stored) and db = column sums of the
// unrounded dz (db null: not wanted; part: act_grad_partials(M, N) floats).
struct ActGradArgs {
    const void *dy, *pre;
    int64_t lddy, ldp;
    void *dz; // [M][N], pitch lddz, a multiple of 8, zeros up to it
    int64_t lddz;
    void *db;
    float *part;
    int64_t M, N;
    int act;
};
int64_t act_grad_partials(int64_t M, int64_t N, int cus);

// What a call's launches leave to launch_finish, which joins it all at once;
// zero-initialised.  The workspaces stay in use until then.
struct Finish {
    GemmArgs p[2]; // up to two products whose k was split
    const float *part[2];
    int splits[2];
    ActGradArgs g; // db
    int64_t parts;
    int64_t blocks[2], columns; // workgroups of each; 0: nothing to join
};

// Workspace bytes launch_gemm may use for this product (fp32 partial sums,
// aligned copies of operands).
size_t gemm_workspace_bytes(int dt, int64_t M, int64_t N, int64_t K, int layout, int cus);
hipError_t launch_gemm(const GemmArgs &a, int dt, int layout, void *ws, int cus, Finish &f, hipStream_t s);
hipError_t launch_act_grad(const ActGradArgs &a, int dt, int cus, Finish &f, hipStream_t s);
hipError_t launch_finish(const Finish &f, int dt, hipStream_t s);

// ---------------------------------------------------------------- logits
struct TopRowsArgs {
    const void *x;
    int64_t R, V, ldx;
    int k;
    float inv_tau;
    int32_t *idx;
    float *val, *lse;
    void *ws;
};
size_t top_rows_workspace_bytes(int dt, int64_t R, int64_t V, int64_t k, int cus);
hipError_t launch_top_rows(const TopRowsArgs &a, int dt, int cus, hipStream_t s);

struct DistillArgs {
    const int32_t *idx[FA_MAX_CLIENTS];
    const float *val[FA_MAX_CLIENTS];
    const float *tlse[FA_MAX_CLIENTS];
    float n[FA_MAX_CLIENTS];
    int k[FA_MAX_CLIENTS];
    int first[FA_MAX_CLIENTS + 1]; // first entry of each client in a row's joined list
    int clients; // contributing ones (n > 0, k > 0)
    int has_tlse;
    const void *z;
    int64_t R, V, ldz;
    float tau, inv_tau;
    const float *row_weight;
    float *loss;
    float *lse; // written by the loss, read by the gradient alone
    void *dz;   // nullable in the loss
    int64_t lddz;
    int *err;
    void *ws;
};
size_t distill_workspace_bytes(int dt, int64_t R, int64_t V, int cus);
hipError_t launch_distill(const DistillArgs &a, int dt, bool loss, int cus, hipStream_t s);

} // namespace fa
