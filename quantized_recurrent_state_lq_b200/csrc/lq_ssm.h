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

// Chain the pieces of every sequence cut in more than one:  S = S0; for each
// piece, slot <- S and S <- decay S + own.
cudaError_t launch_ssm_join(const SsmArgs &a, int seg, cudaStream_t s);

// The chunked scans, with pieces of seg tokens (a multiple of 128); split: at
// least one sequence may be cut.
cudaError_t launch_ssm_umma(const SsmArgs &a, int seg, bool split, cudaStream_t s);            // bf16
cudaError_t launch_ssm_tc(const SsmArgs &a, int dtype, int seg, bool split, cudaStream_t s);   // f32, f16

}  // namespace lq
