// lq_layer.h -- internal launch interface of the recurrent layer's operators
// (lq_conv.cu, lq_norm.cu, lq_ssm.cu), used by the C ABI (lq_layer_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lq {

enum { kF32 = 0, kBF16 = 1, kF16 = 2 };   // lq_dtype

// Token rows of a batch of B sequences: packed (cu: B+1 row offsets on the
// device) or time-major (cu null, T = rows / B tokens each, row t*B + b).
struct Rows {
    const int *cu;
    int B;
    int rows;
};

struct ConvArgs {
    Rows r;
    int C, K, act;
    const void *x;
    int64_t ldx;
    const float *w, *bias;       // [C][K], [C] or null
    const void *state0;          // [B][K-1][C] or null (zeros)
    void *state_out;             // [B][K-1][C] (may be state0)
    void *y;
    int64_t ldy;
};

struct SsmArgs {
    Rows r;
    int H, G, dk, dv, softplus;
    const void *x, *dt, *Bm, *Cm;
    int64_t ldx, lddt, ldb, ldc;
    const float *A, *D, *dt_bias;   // [H]; D, dt_bias may be null
    const float *S0;                // [B][H][dk][dv] or null (zeros)
    float *S_out;                   // (may be S0)
    void *y;
    int64_t ldy;
    float *ws;                      // segment states and decays (ssm_ws_bytes)
    int64_t fail_row;               // self-test: a wait of the piece that starts or ends at this row counts as run out (-1: none)
};

struct NormArgs {
    int64_t rows;
    int G, D;
    float eps;
    const void *x;
    int64_t ldx;
    const float *w;          // [D], or [G][D] with w_groups
    int w_groups;
    const void *z;           // gate or null (norm_out)
    int64_t ldz;
    int act, gate_first;
    const void *res;         // or null
    int64_t ldres;
    float scale;
    const float *dscale;     // [G*D] or null
    void *h;                 // norm_in: the updated residual
    int64_t ldh;
    void *y;
    int64_t ldy;
};

cudaError_t launch_conv_prefill(const ConvArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_conv_step(const ConvArgs &a, int dtype, cudaStream_t s);

cudaError_t launch_ssm_prefill(const SsmArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_ssm_step(const SsmArgs &a, int dtype, cudaStream_t s);
size_t ssm_ws_bytes(int dtype, int B, int rows, int H, int G, int dk, int dv);

cudaError_t launch_norm_in(const NormArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_norm_out(const NormArgs &a, int dtype, int x_dtype, cudaStream_t s);

}  // namespace lq
