// backward.cuh -- what the two paths of the prefill's backward pass share: the operands of a
// call and the kernels behind the gradients' sums.
#pragma once

#include "common.cuh"

namespace ssd {

// One call of the backward pass.  Layouts as in include/ssd.h.
struct BwdArgs {
    int b, T, H, N, G, io;
    const void *dy, *x;
    const float* dt;
    DtMap dtm;
    const float* A;
    const void *B, *C;
    const float *D, *h0, *dhf;  // h0, dhf may be nullptr (zero)
    void* dx;
    float *ddt, *dA;
    void *dB, *dC;
    float *dD, *dh0, *dbias;  // dh0, dbias may be nullptr (not wanted)
};

// softplus'(z) behind the clamp: sigmoid(z) where the clamp lets softplus(z) through, else 0.
__device__ __forceinline__ float dt_slope(float z, const DtMap& m) {
    const float sp = z > 20.f ? z : log1pf(expf(z));
    return sp >= m.lo && sp <= m.hi ? 1.f / (1.f + expf(-z)) : 0.f;
}

// Sums over the chunks: dA, dD and (if wanted) the bias gradient from per-(chunk, head) parts
// [n][H] each, in chunk order per thread and in fp64, so the result depends on the shape alone.
int launch_bwd_head_sums(const float* part_dA, const float* part_dD, const float* part_db, int n, int H, float* dA,
                         float* dD, float* db, cudaStream_t s);

}  // namespace ssd
