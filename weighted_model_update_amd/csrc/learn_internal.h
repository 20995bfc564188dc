// Internal interface between the host library and the kernels of the linear
// layer (linear.hip), the layers on 8-bit weights (int8.hip), the per-row top
// logits and the distillation loss (logits.hip), and the orthogonalised update
// (orthogonal.hip).  Not part of the public ABI.
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
    bool a_padded, b_padded; // rows are followed by zeros up to whole chunks
    // 8-bit operands: M and N factors of the sums; null for the others
    const float *row_scale, *col_scale;
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
    // N factors of the stored dz, not of db; nullable.  With them there is a dz, and
    // fp32's is dz = a + 2^-8 b + 2^-16 c as three bf16 matrices, `plane` elements apart.
    const float *col_scale;
    int64_t plane;
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
int64_t finish_blocks(int64_t M, int64_t N); // Finish.blocks of a split product

// ---------------------------------------------------------------- 8-bit layers
struct QuantizeArgs {
    const void *x;
    int64_t R, C, ldx;
    int8_t *q;
    int64_t ldq, fill; // zeros follow the row up to column `fill` >= C
    float *scale;
};
hipError_t launch_quantize(const QuantizeArgs &a, int dt, hipStream_t s);

// As launch_gemm, for rows of 8-bit integers on both sides; dt is the type of
// bias, residual and results.
size_t gemm8_workspace_bytes(int64_t M, int64_t N, int64_t K, int cus);
hipError_t launch_gemm8(const GemmArgs &a, int dt, void *ws, int cus, hipStream_t s);

// Whether a product takes one launch that also brings x to 8 bits: few rows, which
// a workgroup holds, and weights whose rows are whole chunks.
bool few8_ok(int64_t M, int64_t K, const void *w, int64_t ldw);
// That launch, from rows a.a of dt (a.row_scale is not used).
hipError_t launch_few8(const GemmArgs &a, int dt, int cus, hipStream_t s);

// dx = alpha u w for u [M][N] (a.a, pitch a.lda, zeros behind the row) in bf16, one
// matrix (dt FA_BF16) or three of them, `plane` elements apart (FA_F32), and 8-bit w [N][K] (a.b).  As a product: a.M = M, a.N = K, a.K = N.
bool grad8_ok(int64_t N, int64_t K, const void *w, int64_t ldw);
size_t grad8_workspace_bytes(int dt, int64_t M, int64_t N, int64_t K, int cus);
hipError_t launch_grad8(const GemmArgs &a, int dt, int64_t plane, void *ws, int cus, Finish &f, hipStream_t s);

// out [rows][ldo] = w in bf16, or as it is, zeros from column `cols` on.
hipError_t launch_widen(const int8_t *w, int64_t ldw, int64_t rows, int64_t cols, void *out, int64_t ldo, hipStream_t s);
hipError_t launch_copy8(const int8_t *w, int64_t ldw, int64_t rows, int64_t cols, int8_t *out, int64_t ldo, hipStream_t s);

// ---------------------------------------------------------------- orthogonalised update
// out = rate O, or keep out + rate O (add), O the orthogonalised t [B][m][n].
struct OrthoArgs {
    const void *x; // the update, pitch ldx, stride_x from matrix to matrix
    int64_t ldx, stride_x;
    float *momentum; // nullable
    int64_t ldm, stride_m;
    float beta;
    int nesterov;
    int64_t B, m, n;
    int steps;
    double coef[FA_MAX_ORTHO_STEPS][3];
    bool unit; // x is divided by its norm already
    void *out;
    int64_t ldo, stride_o;
    int add;
    float keep, rate;
    void *ws;
};
// Whether the steps keep the singular values below 1e9 and, on long sides, their
// scales within fp32, by o.m, o.n, o.steps, o.coef and the result's type.
bool ortho_reach_ok(const OrthoArgs &o, int dt);
// For any steps, and for those of a call.
size_t ortho_workspace_bytes(int64_t B, int64_t m, int64_t n, int cus);
size_t ortho_workspace_needed(const OrthoArgs &o, int cus);
hipError_t launch_ortho(const OrthoArgs &o, int update_dt, int dt, int cus, hipStream_t s);

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
