// Internal declarations of the residual and gated norms (not part of the ABI).
#pragma once

#include <initializer_list>

#include "ssd_internal.cuh"

namespace ssd {

// residual: of the forward, or (backward) the sum the forward left. Optional pointers: residual
// (forward), scale, res_out, x (backward).
struct AddNormArgs {
    int64_t rows, dim;
    ssd_dtype_t dtype, res_dtype;
    const void *x, *residual;
    const float *scale, *weight;
    float eps;
    void *res_out, *out;
};
struct AddNormGrads {
    const void *dout, *dres_in;
    void *dres, *dx;
    float *dw, *dscale;
};
struct GateNormArgs {
    int64_t rows, dim, ngroups;
    ssd_dtype_t dtype;
    const void *y, *z;
    int64_t z_stride;
    const float *weight;
    float eps;
    void *out;
};
struct GateNormGrads {
    const void *dout;
    void *dy, *dz;
    int64_t dz_stride;
    float *dw;
};

int norm_max_group();  // channels of one normalised group
size_t norm_bwd_workspace_bytes(int64_t rows, int64_t dim);
cudaError_t add_rmsnorm_launch(const AddNormArgs &a, cudaStream_t s);
cudaError_t add_rmsnorm_bwd_launch(const AddNormArgs &a, const AddNormGrads &g, float *ws, cudaStream_t s);
cudaError_t norm_gate_launch(const GateNormArgs &a, cudaStream_t s);
// gate_first: of ssd_gated_rmsnorm; else of ssd_norm_gate
cudaError_t gate_norm_bwd_launch(const GateNormArgs &a, const GateNormGrads &g, bool gate_first, float *ws, cudaStream_t s);

}  // namespace ssd
