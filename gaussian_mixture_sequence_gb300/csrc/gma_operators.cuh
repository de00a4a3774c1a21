// Launchers of the operators around the mixer, and what they take of the shared sources.  (Apart from
// gma_internal.cuh, whose contents key the DRAM counters of the mixer's kernels.)
#pragma once
#include "gma_internal.cuh"

namespace gma {

// [d2][d1][d0] without a swizzle, boxes of box0 x box1 x 1 (box0 elements a multiple of 16 bytes).
bool make_tma_rows(CUtensorMap *m, const void *base, bool bf16, unsigned long long d0, unsigned long long d1,
                   unsigned long long d2, unsigned box0, unsigned box1);

// Shapes that the tensor-core routing of every component fits: those of resp_gtc_applies and K = 128, where
// the balance loss takes it, as it needs the posteriors that the bounded routing drops.
bool resp_gtc_fits(const Dims &dm);

// Gated linear recurrence (gma_scan.cu).  S slices of [N][D]; lengths indexed by slice / H.
struct ScanDims {
    int S, H, N, D;
    bool mean, bf16;
};
cudaError_t launch_scan_fwd(const ScanDims &sd, const void *x, const void *gate, const int *lengths,
                            const float *state_in, float *state_out, void *out, cudaStream_t st);
cudaError_t launch_scan_bwd(const ScanDims &sd, const void *x, const void *gate, const void *out, const void *dout,
                            const int *lengths, const float *state_in, const float *dstate_out, void *dx, void *dgate,
                            float *dstate_in, cudaStream_t st);
cudaError_t launch_scan_step(const ScanDims &sd, const void *x, const void *gate, float *state, void *out,
                             cudaStream_t st);

// Beam selection and state reordering (gma_beam.cu).
struct BeamDims {
    int B, W, V, ld, eos, pad;
    bool bf16;
};
constexpr int kMaxBeams = 32;
size_t beam_ws_bytes(const BeamDims &bd);
cudaError_t launch_beam_select(const BeamDims &bd, const void *logits, const float *score_in,
                               const unsigned char *finished_in, float *score_out, int *parent, int *token,
                               unsigned char *finished_out, void *ws, cudaStream_t st);
cudaError_t launch_beam_reorder(int B, int W, size_t row_bytes, const int *parent, void *state, cudaStream_t st);

// Balance loss and its gradients (gma_balance.cu).  Scratch of the refinement: prec[H][K][D]
// (1/sigma^2 as two fp32 values), cst2[H][K] (the component's constant, two fp32 values),
// second[H] (the scale of the posteriors that are refined),
// psum / pcnt [H][blocks][K] (partial sums over a part of the rows).  Scratch of the gradients:
// inv[H][K][D] (1/sigma^2 and mu, by pairs of features), terms[rows][K] and n_terms[rows] (the terms of each row that
// count), hist[H][K] (the terms of each component) and part[H][parts][K (2 D + 1)].
int balance_blocks(const Dims &dm);
int balance_parts(const Dims &dm);
cudaError_t launch_balance_prep(const Dims &dm, const gma_params &p, float2 *prec, float2 *cst2, float *second,
                                cudaStream_t st);
cudaError_t launch_balance_loss(const Dims &dm, const gma_params &p, const void *x, const int *lengths,
                                const float2 *prec, const float2 *cst2, float *second, float *gamma, float *psum,
                                int *pcnt, float *loss, long long *counts, float *prob, cudaStream_t st);
cudaError_t launch_balance_grad(const Dims &dm, const gma_params &p, const void *x, const int *lengths,
                                const float *gamma, const long long *counts, const float *dloss, float *inv,
                                float2 *terms, int *n_terms, int *hist, float *part, float *dx, float *dmu, float *dvar,
                                float *dlogit, bool accumulate, cudaStream_t st);

} // namespace gma
