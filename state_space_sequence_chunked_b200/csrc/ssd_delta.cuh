// Internal declarations of the gated delta rule's kernels (not part of the ABI).
#pragma once

#include "ssd_internal.cuh"

namespace ssd {

// One problem, validated by the API layer.
struct DeltaProblem {
    int64_t B, L, H, P, G, N;
    ssd_dtype_t dtype;
    const void *x, *g, *beta, *Bm, *Cm;
    const float *h0;
    void *y;
    float *h_final;
};

// Cotangents in and gradients out (dh_final and dh0 may be NULL).
struct DeltaGrads {
    const void *dy;
    const float *dh_final;
    void *dx, *dg, *dbeta, *dBm, *dCm;
    float *dh0;
};

constexpr int kSeg = 32;  // tokens per segment of the general backward
// What the gradients that sum over state rows need of sequences of at most kSeg tokens, err and z each in two bf16
// parts [B, L, H, P] (their states are the initial one and the final one's cotangent).
struct DeltaParts {
    const void *err, *err_lo, *z, *z_lo;
};

// A log decay as it enters a cumulated sum: exp of anything below is 0 in fp32 all the same, and a
// decay of minus infinity (a reset of the state) must not turn differences of sums into NaN.
__device__ __forceinline__ double clamp_log_decay(float g) { return g < -1e4f ? -1e4 : (double)g; }

// ---- general path: fp32 arithmetic, token by token ----
cudaError_t delta_seq_fwd(const DeltaProblem &p, cudaStream_t s);
size_t delta_seq_bwd_workspace_bytes(const DeltaProblem &p);
cudaError_t delta_seq_bwd(const DeltaProblem &p, const DeltaGrads &g, void *ws, cudaStream_t s);
// dx, dg, dbeta and the per-head fp32 parts of dB, dC [B, L, H, N] of bf16 sequences of at most kSeg tokens
cudaError_t delta_short_grads(const DeltaProblem &p, const DeltaGrads &g, const DeltaParts &parts, float *dB, float *dC, cudaStream_t s);
// dBm, dCm [B, L, G, N] from per-head fp32 parts [B, L, H, N], added in head order
cudaError_t delta_group_sum_launch(const DeltaProblem &p, const float *dB_part, const float *dC_part, void *dBm, void *dCm,
                                   cudaStream_t s);
// ---- chunked tensor-core path (bf16, dstate <= 128) ----
constexpr int kDeltaChunk = 64;
bool delta_mma_supported(const DeltaProblem &p, bool backward);
size_t delta_mma_fwd_workspace_bytes(const DeltaProblem &p);
int delta_mma_fwd_kernels(const DeltaProblem &p);
cudaError_t delta_mma_fwd(const DeltaProblem &p, void *ws, cudaStream_t s);
size_t delta_mma_bwd_workspace_bytes(const DeltaProblem &p);
int delta_mma_bwd_kernels(const DeltaProblem &p);
cudaError_t delta_mma_bwd(const DeltaProblem &p, const DeltaGrads &g, void *ws, cudaStream_t s);

// The chains over the chunks on tcgen05 (ssd_delta_tc.cu), after k_delta_prep: the forward's, or the
// backward pass's recomputation and reverse chain together. states and cots [B, H, chunks, P, N], err, u
// and z [B, L, H, P], bf16, are the latter's; with z_lo there, no states and cotangents leave the chains, nor dx, but
// err and z in two parts each, err's second in the place of u.
struct DeltaChain {
    const char *prep;
    int64_t prep_bytes;    // per chunk and head
    int scal_at, rows_at;  // the backward pass: the scalars; W and P by rows of blocks
    int *status, *flags;   // cleared before: the status word, a counter per CTA
    float *hand;           // delta_tc_hand_bytes
    void *states, *err, *u, *cots, *z, *z_lo;
};
int delta_tc_grid(const DeltaProblem &p, bool backward);
size_t delta_tc_hand_bytes(const DeltaProblem &p, bool backward);
cudaError_t delta_tc_fwd(const DeltaProblem &p, const DeltaChain &ch, cudaStream_t s);
cudaError_t delta_tc_bwd(const DeltaProblem &p, const DeltaGrads &g, const DeltaChain &ch, cudaStream_t s);
// After both chains (ssd_delta_grads.cu): dBm, dCm, dg, dbeta. With more than one slice of a group's heads
// the keys' and queries' gradients are fp32 parts [B, L, G * slices, N], to be summed.
int delta_grads_slices(const DeltaProblem &p);
cudaError_t delta_grads(const DeltaProblem &p, const DeltaGrads &g, const DeltaChain &ch, float *dB_part, float *dC_part,
                        cudaStream_t s);

// one token (p.L, p.h0, p.h_final unused); state_out may be state_in
cudaError_t delta_step(const DeltaProblem &p, const float *state_in, float *state_out, cudaStream_t s);

// packed pairs of fp32: a b, and c + a b
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\tmul.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
        "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

}  // namespace ssd
