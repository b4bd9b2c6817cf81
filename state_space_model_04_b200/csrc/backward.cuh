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

// Sums over the chunks: dA, dD and (pb not nullptr) the bias gradient from per-(chunk, head) parts
// [n][H] each, in a fixed order and in fp64, so the result depends on the shape alone.  One block
// a sum, behind the blocks that add up dB and dC: in a launch of their own they cost small calls
// 3 us more.
struct HeadSums {
    const float *pA, *pD, *pb;
    int n, H;
    float *dA, *dD, *db;
    __host__ int blocks() const { return H * (pb ? 3 : 2); }
};
template <int kThr>
__device__ __forceinline__ void head_sum(const HeadSums& p, int block) {
    __shared__ double s[kThr / 32];
    const int h = block % p.H, which = block / p.H;
    const float* src = which == 0 ? p.pA : which == 1 ? p.pD : p.pb;
    double a = 0.0;
#pragma unroll 4
    for (int i = threadIdx.x; i < p.n; i += kThr) a += src[(size_t)i * p.H + h];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kThr / 32; ++i) a += s[i];
        (which == 0 ? p.dA : which == 1 ? p.dD : p.db)[h] = (float)a;
    }
}

}  // namespace ssd
