// lq_ssm.h -- what the scan's prompt kernels share: the pieces a batch is cut
// into and the workspace that carries states from piece to piece.
#pragma once

#include "lq_act.cuh"

namespace lq {

// Workspace of a batch cut into pieces: [pieces][H][dk][dv] states -- a piece's
// own state (from zero) after the first pass, the state it starts from after
// the join -- then [pieces][H] decays.  Pieces are numbered by find_piece;
// piece_count(r, seg) of them.
__host__ __device__ inline float *ssm_decays(const SsmArgs &a, int seg) {
    return a.ws + piece_count(a.r, seg) * a.H * a.dk * a.dv;
}

// Log2 decays and their running sums as fixed point with 32 fraction bits: the
// sum of a chunk (at most 128 x 150) and every difference are exact to 2^-33 per
// token, and cost integer adds (FP64 sums took 4000 cycles a chunk here).
__device__ __forceinline__ long long decay_fix(float l) { return __float2ll_rn(l * 4294967296.0f); }
__device__ __forceinline__ float decay_f(long long v) {
    return fmaf((float)(unsigned)v, 0x1p-32f, (float)(int)(v >> 32));
}
// The same as an integer part and a fraction (to 2^-25), both floats.
__device__ __forceinline__ void decay_parts(long long v, float &whole, float &fraction) {
    whole = (float)(int)(v >> 32);
    fraction = (float)(unsigned)v * 0x1p-32f;
}

// A token's step d and log2 decay d A: within +-150 (2^-150 is flushed to 0 in
// FP32, 2^150 is its infinity), so that no difference of sums is inf - inf.  A
// decay that is not a number makes the step one, which shows in all it touches.
__device__ __forceinline__ long long decay_of(float &d, float A2) {
    float l = d * A2;
    if (l != l) d = l;
    l = fminf(fmaxf(l, -150.0f), 150.0f);
    return decay_fix(l);
}

__device__ __forceinline__ long long warp_scan(long long v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, v, m);
        if (lane >= m) v += o;
    }
    return v;
}

// The join and the scan after it are launched while the kernel before still runs
// (programmatic dependent launch) and wait until it is done and its results are
// there: the launches and what comes ahead of the wait are hidden (600 bf16 tokens
// of two sequences: 24 us against 26).  Nothing that a kernel before writes is read,
// and nothing that it reads is written, ahead of the wait.
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// Chain the pieces of every sequence cut in more than one:  S = S0; for each
// piece, slot <- S and S <- decay S + own.
// early: the scan's CTAs may take their places meanwhile (one per SM; several per SM
// would pile up on the SMs that are free first, 43 us against 34 for 2048 f32 tokens
// of 4 heads of 128 x 64).
cudaError_t launch_ssm_join(const SsmArgs &a, int seg, bool early, cudaStream_t s);

// The chunked scans, with pieces of seg tokens (whole chunks); split: at least
// one sequence may be cut.
cudaError_t launch_ssm_umma(const SsmArgs &a, int seg, bool split, cudaStream_t s);            // bf16
cudaError_t launch_ssm_tc(const SsmArgs &a, int dtype, int seg, bool split, cudaStream_t s);   // f32, f16

}  // namespace lq
