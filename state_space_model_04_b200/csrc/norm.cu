// norm.cu -- the two RMS norms of a block, forward and backward: the residual norm ahead of
// it and the gated norm behind its SSD.
//
// Residual norm, per row of D elements:
//   r = residual + s x,  k = (mean(r^2) + eps)^(-1/2),  out = r k w
//   backward, g = dout w:  dr = k (g - r k^2 mean(g r)) + dr_out,  dx = s dr,
//                          dresidual = dr,  dw = sum over rows of dout r k
// Gated norm, per group of D / groups elements of a row (silu(z) = z sigmoid(z)):
//   gate first:  v = y silu(z),  out = v k(v) w
//                g = dout w:  dv = k (g - v k^2 mean(g v)),  dy = dv silu(z),
//                dz = dv y silu'(z),  dw = sum of dout v k
//   norm first:  out = y k(y) w silu(z)
//                t = dout silu(z), g = t w:  dy = k (g - y k^2 mean(g y)),
//                dz = dout y k w silu'(z),  dw = sum of t y k
// Everything is computed in fp32 from the stored operands and rounded once, on the store.
//
// Bound: device memory.  Each operand is read once and each result written once; a segment
// (a row, or one group of a row) stays in registers between its reductions and its results.
// A segment belongs to `tps` threads of a block (blockDim.x), blockDim.y segments side by
// side; the block then walks rows by a grid stride with its weights held in registers.  In the
// backward pass the thread owns the same columns of every row it sees, so dw is summed in
// registers over the rows, stored once per block to the workspace, and a second kernel adds
// the blocks' sums in a fixed order (no atomics: the same call gives the same bits).
#include <algorithm>
#include <cmath>
#include "common.cuh"

namespace ssd {
namespace {

constexpr int kMaxThreads = 512;
// rows a block walks in the backward pass are spread over at most this many blocks an SM
constexpr int kBwdBlocksPerSM = 6;
constexpr int kSumRows = 32;  // threads along the parts in the dw sum kernel

int norm_sm_count() {
    static const int n = [] {
        int v = 0;
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, 0) != cudaSuccess || v < 1) v = 148;
        return v;
    }();
    return n;
}

// ---- V consecutive elements as fp32 (V = 8: 16-byte accesses; V = 1: one element)
template <int V>
__device__ __forceinline__ void loadv(const float* p, float (&o)[V]) {
    if constexpr (V == 8) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
    } else {
        o[0] = *p;
    }
}
template <int V>
__device__ __forceinline__ void loadv(const __nv_bfloat16* p, float (&o)[V]) {
    if constexpr (V == 8) {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = __uint_as_float(u[i] << 16);
            o[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
        o[0] = __bfloat162float(*p);
    }
}
template <int V>
__device__ __forceinline__ void storev(float* p, const float (&v)[V]) {
    if constexpr (V == 8) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *p = v[0];
    }
}
template <int V>
__device__ __forceinline__ void storev(__nv_bfloat16* p, const float (&v)[V]) {
    if constexpr (V == 8) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&t);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        *p = __float2bfloat16_rn(v[0]);
    }
}

// Sum of a (and b) over the threads of one segment.  A segment of at most 32 threads is one
// warp; longer ones meet in shared memory.  `red` holds 2 x [blockDim.y][warps] pairs used in
// turn (`flip`), so one barrier a row is enough: a block can be at most one row ahead of its
// slowest warp.  Every thread of the block calls this the same number of times.
__device__ __forceinline__ float2 segment_sum(float a, float b, float2* red, int flip) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (blockDim.x == 32) return make_float2(a, b);
    const int nw = blockDim.x >> 5, w = threadIdx.x >> 5;
    float2* mine = red + (flip * blockDim.y + threadIdx.y) * nw;
    if ((threadIdx.x & 31) == 0) mine[w] = make_float2(a, b);
    __syncthreads();
    float2 t = make_float2(0.f, 0.f);
    for (int i = 0; i < nw; ++i) {
        const float2 m = mine[i];
        t.x += m.x;
        t.y += m.y;
    }
    return t;
}

__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

struct ResFwd {
    const void* x;
    const void* res;  // or nullptr
    const float* w;
    void* out;
    void* r;  // or nullptr
    long long rows, ld_x, ld_res, ld_out, ld_r;
    int D;
    float scale, eps;
};
struct ResBwd {
    const void* dout;
    const void* r;
    const float* w;
    const void* dr_out;  // or nullptr
    void* dx;            // or nullptr
    void* dres;          // or nullptr
    float* part;         // [gridDim.x * blockDim.y][D] sums of dw, or nullptr
    long long rows, ld_dout, ld_r, ld_dro, ld_dx, ld_dres;
    int D;
    float scale, eps;
};
struct GateFwd {
    const void* y;
    const void* z;
    const float* w;
    void* out;
    long long rows, ld_y, ld_z, ld_out;
    int D, L;  // L = D / groups; blockIdx.y is the group
    float eps;
};
struct GateBwd {
    const void* dout;
    const void* y;
    const void* z;
    const float* w;
    void* dy;
    void* dz;
    float* part;  // or nullptr
    long long rows, ld_dout, ld_y, ld_z, ld_dy, ld_dz;
    int D, L;
    float eps;
};

#define SSD_NORM_PROLOGUE(LEN)                                                                   \
    extern __shared__ float2 red[];                                                              \
    const int tps = blockDim.x;                                                                  \
    const long long row_step = (long long)gridDim.x * blockDim.y;                                \
    const long long row_end = (p.rows + row_step - 1) / row_step * row_step;                     \
    const float inv_len = 1.f / (float)(LEN);                                                    \
    int col[VPT];                                                                                \
    bool has[VPT];                                                                               \
    _Pragma("unroll") for (int i = 0; i < VPT; ++i) {                                            \
        col[i] = (i * tps + (int)threadIdx.x) * V;                                               \
        has[i] = col[i] < (LEN);                                                                 \
    }                                                                                            \
    int flip = 0;

template <typename TIO, typename TRES, int V, int VPT>
__global__ void __launch_bounds__(kMaxThreads) ssd_residual_norm_kernel(const ResFwd p) {
    SSD_NORM_PROLOGUE(p.D)
    float w[VPT][V];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (has[i]) loadv<V>(p.w + col[i], w[i]);
    for (long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y; row < row_end; row += row_step) {
        const bool in = row < p.rows;
        float r[VPT][V], ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int v = 0; v < V; ++v) r[i][v] = 0.f;
            if (in && has[i]) {
                float xv[V];
                if (p.res) loadv<V>(static_cast<const TRES*>(p.res) + row * p.ld_res + col[i], r[i]);
                loadv<V>(static_cast<const TIO*>(p.x) + row * p.ld_x + col[i], xv);
#pragma unroll
                for (int v = 0; v < V; ++v) r[i][v] = fmaf(p.scale, xv[v], r[i][v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) ss = fmaf(r[i][v], r[i][v], ss);
        }
        const float k = rsqrtf(segment_sum(ss, 0.f, red, flip).x * inv_len + p.eps);
        flip ^= 1;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (in && has[i]) {
                if (p.r) storev<V>(static_cast<TRES*>(p.r) + row * p.ld_r + col[i], r[i]);
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = r[i][v] * k * w[i][v];
                storev<V>(static_cast<TIO*>(p.out) + row * p.ld_out + col[i], o);
            }
        }
    }
}

template <typename TIO, typename TRES, int V, int VPT>
__global__ void __launch_bounds__(kMaxThreads) ssd_residual_norm_backward_kernel(const ResBwd p) {
    SSD_NORM_PROLOGUE(p.D)
    float w[VPT][V], dw[VPT][V];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (has[i]) loadv<V>(p.w + col[i], w[i]);
#pragma unroll
        for (int v = 0; v < V; ++v) dw[i][v] = 0.f;
    }
    for (long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y; row < row_end; row += row_step) {
        const bool in = row < p.rows;
        float r[VPT][V], g[VPT][V], d[VPT][V], ss = 0.f, gr = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int v = 0; v < V; ++v) r[i][v] = g[i][v] = d[i][v] = 0.f;
            if (in && has[i]) {
                loadv<V>(static_cast<const TRES*>(p.r) + row * p.ld_r + col[i], r[i]);
                loadv<V>(static_cast<const TIO*>(p.dout) + row * p.ld_dout + col[i], g[i]);
                if (p.dr_out) loadv<V>(static_cast<const TRES*>(p.dr_out) + row * p.ld_dro + col[i], d[i]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    ss = fmaf(r[i][v], r[i][v], ss);
                    gr = fmaf(g[i][v] * w[i][v], r[i][v], gr);
                }
            }
        }
        const float2 sum = segment_sum(ss, gr, red, flip);
        flip ^= 1;
        const float k = rsqrtf(sum.x * inv_len + p.eps);
        const float m = sum.y * inv_len * k * k;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (in && has[i]) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    dw[i][v] = fmaf(g[i][v], r[i][v] * k, dw[i][v]);
                    d[i][v] = fmaf(k, g[i][v] * w[i][v] - r[i][v] * m, d[i][v]);
                }
                if (p.dres) storev<V>(static_cast<TRES*>(p.dres) + row * p.ld_dres + col[i], d[i]);
                if (p.dx) {
#pragma unroll
                    for (int v = 0; v < V; ++v) d[i][v] *= p.scale;
                    storev<V>(static_cast<TIO*>(p.dx) + row * p.ld_dx + col[i], d[i]);
                }
            }
        }
    }
    if (p.part) {
        float* part = p.part + (size_t)(blockIdx.x * blockDim.y + threadIdx.y) * p.D;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (has[i]) storev<V>(part + col[i], dw[i]);
    }
}

template <typename TIO, bool kNormFirst, int V, int VPT>
__global__ void __launch_bounds__(kMaxThreads) ssd_gated_norm_kernel(const GateFwd p) {
    SSD_NORM_PROLOGUE(p.L)
    const int base = blockIdx.y * p.L;
    float w[VPT][V];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (has[i]) loadv<V>(p.w + base + col[i], w[i]);
    for (long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y; row < row_end; row += row_step) {
        const bool in = row < p.rows;
        float a[VPT][V], gt[VPT][V], ss = 0.f;  // a: what is normalised; gt: silu(z) where it follows the norm
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int v = 0; v < V; ++v) a[i][v] = gt[i][v] = 0.f;
            if (in && has[i]) {
                loadv<V>(static_cast<const TIO*>(p.y) + row * p.ld_y + base + col[i], a[i]);
                loadv<V>(static_cast<const TIO*>(p.z) + row * p.ld_z + base + col[i], gt[i]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    gt[i][v] *= sigmoid_f(gt[i][v]);
                    if (!kNormFirst) a[i][v] *= gt[i][v];
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) ss = fmaf(a[i][v], a[i][v], ss);
        }
        const float k = rsqrtf(segment_sum(ss, 0.f, red, flip).x * inv_len + p.eps);
        flip ^= 1;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (in && has[i]) {
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    o[v] = a[i][v] * k * w[i][v];
                    if (kNormFirst) o[v] *= gt[i][v];
                }
                storev<V>(static_cast<TIO*>(p.out) + row * p.ld_out + base + col[i], o);
            }
        }
    }
}

template <typename TIO, bool kNormFirst, int V, int VPT>
__global__ void __launch_bounds__(kMaxThreads) ssd_gated_norm_backward_kernel(const GateBwd p) {
    SSD_NORM_PROLOGUE(p.L)
    const int base = blockIdx.y * p.L;
    float w[VPT][V], dw[VPT][V];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (has[i]) loadv<V>(p.w + base + col[i], w[i]);
#pragma unroll
        for (int v = 0; v < V; ++v) dw[i][v] = 0.f;
    }
    for (long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y; row < row_end; row += row_step) {
        const bool in = row < p.rows;
        float y[VPT][V], z[VPT][V], g[VPT][V], ss = 0.f, gv = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int v = 0; v < V; ++v) y[i][v] = z[i][v] = g[i][v] = 0.f;
            if (in && has[i]) {
                loadv<V>(static_cast<const TIO*>(p.y) + row * p.ld_y + base + col[i], y[i]);
                loadv<V>(static_cast<const TIO*>(p.z) + row * p.ld_z + base + col[i], z[i]);
                loadv<V>(static_cast<const TIO*>(p.dout) + row * p.ld_dout + base + col[i], g[i]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float gate = z[i][v] * sigmoid_f(z[i][v]);
                    const float n = kNormFirst ? y[i][v] : y[i][v] * gate;  // what is normalised
                    const float t = kNormFirst ? g[i][v] * gate : g[i][v];  // gradient behind the weight
                    ss = fmaf(n, n, ss);
                    gv = fmaf(t * w[i][v], n, gv);
                }
            }
        }
        const float2 sum = segment_sum(ss, gv, red, flip);
        flip ^= 1;
        const float k = rsqrtf(sum.x * inv_len + p.eps);
        const float m = sum.y * inv_len * k * k;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (in && has[i]) {
                float dy[V], dz[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float sg = sigmoid_f(z[i][v]), gate = z[i][v] * sg;
                    const float dgate = fmaf(gate, 1.f - sg, sg);  // silu'(z)
                    if (kNormFirst) {
                        const float n = y[i][v] * k, t = g[i][v] * gate;
                        dw[i][v] = fmaf(t, n, dw[i][v]);
                        dy[v] = k * (t * w[i][v] - y[i][v] * m);
                        dz[v] = g[i][v] * n * w[i][v] * dgate;
                    } else {
                        const float n = y[i][v] * gate;
                        dw[i][v] = fmaf(g[i][v], n * k, dw[i][v]);
                        const float dn = k * (g[i][v] * w[i][v] - n * m);
                        dy[v] = dn * gate;
                        dz[v] = dn * y[i][v] * dgate;
                    }
                }
                storev<V>(static_cast<TIO*>(p.dy) + row * p.ld_dy + base + col[i], dy);
                storev<V>(static_cast<TIO*>(p.dz) + row * p.ld_dz + base + col[i], dz);
            }
        }
    }
    if (p.part) {
        float* part = p.part + (size_t)(blockIdx.x * blockDim.y + threadIdx.y) * p.D + base;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (has[i]) storev<V>(part + col[i], dw[i]);
    }
}

// dw[c] = sum over the parts, in part order per thread row and then over the thread rows.
__global__ void __launch_bounds__(32 * kSumRows) ssd_norm_dweight_kernel(const float* part, float* dw, int parts, int D) {
    __shared__ float s[kSumRows][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float a = 0.f;
    if (c < D)
        for (int i = threadIdx.y; i < parts; i += kSumRows) a += part[(size_t)i * D + c];
    s[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    float t = s[threadIdx.x][threadIdx.y];  // transposed: a warp now holds one column's rows
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int cc = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && cc < D) dw[cc] = t;
}

// Launch shape of one call: V elements an access, VPT accesses a thread and operand, tps
// threads a segment, seg segments a block, and blocks along the rows.
struct Shape {
    int V, vpt, tps, seg, blocks;
    size_t smem;
};

// Vector accesses need every operand's row starts on 16 bytes and segments of whole vectors
// (`vec`); otherwise elements are read one by one.  A thread takes one access of a segment
// while that leaves at most 384 threads a segment, two up to 768 and four beyond: few accesses
// keep the registers low and several blocks on an SM.
Shape norm_shape(long long rows, int groups, int L, bool vec, bool backward) {
    Shape s;
    s.V = vec ? 8 : 1;
    const int n = (L + s.V - 1) / s.V;
    if (vec) s.vpt = n <= 384 ? 1 : n <= 768 ? 2 : 4;
    else s.vpt = n <= 4 * kMaxThreads ? 4 : 32;
    s.tps = ((n + s.vpt - 1) / s.vpt + 31) / 32 * 32;
    s.seg = s.tps >= 256 ? 1 : std::max(1, 256 / s.tps);
    s.smem = 2 * sizeof(float2) * s.seg * (s.tps / 32);
    const long long want = (rows + s.seg - 1) / s.seg;
    // forward: a few waves of blocks; backward: one wave, since each block stores a part of dw
    const int per_sm = backward ? kBwdBlocksPerSM : 4 * std::max(1, 2048 / (s.tps * s.seg));
    const long long cap = std::max<long long>(1, (long long)norm_sm_count() * per_sm / groups);
    s.blocks = (int)std::min(want, cap);
    return s;
}

template <typename K, typename Prm>
int launch_norm(const char* name, K k, const Shape& sh, int groups, const Prm& p, cudaStream_t s) {
    LaunchScope ls(name, s);
    k<<<dim3(sh.blocks, groups), dim3(sh.tps, sh.seg), sh.smem, s>>>(p);
    SSD_CUDA_TRY(cudaGetLastError());
    return SSD_OK;
}

int launch_dweight(const float* part, float* dw, int parts, int D, cudaStream_t s) {
    LaunchScope ls("ssd_norm_dweight", s);
    ssd_norm_dweight_kernel<<<(D + 31) / 32, dim3(32, kSumRows), 0, s>>>(part, dw, parts, D);
    SSD_CUDA_TRY(cudaGetLastError());
    return SSD_OK;
}

// the kernel of a shape among the five (V, VPT) instances
#define SSD_NORM_PICK(kernel, A, B)                                                         \
    (sh.V == 8 ? (sh.vpt == 1 ? kernel<A, B, 8, 1> : sh.vpt == 2 ? kernel<A, B, 8, 2> : kernel<A, B, 8, 4>) \
               : (sh.vpt == 4 ? kernel<A, B, 1, 4> : kernel<A, B, 1, 32>))

bool vec_ok(const void* p, long long ld, int elem) {
    return !p || (aligned16(p) && (ld * elem) % 16 == 0);
}

}  // namespace

// Bytes of the backward passes' workspace: the blocks' sums of dw, for the vector and the
// element shapes alike.
size_t norm_workspace_bytes(long long rows, int D, int groups) {
    const int L = D / groups;
    size_t parts = 0;
    for (int v = 0; v < 2; ++v) {
        if (v && L % 8) continue;
        const Shape s = norm_shape(rows, groups, L, v != 0, true);
        parts = std::max(parts, (size_t)s.blocks * s.seg);
    }
    return round_up(parts * D * sizeof(float), 256);
}

int launch_residual_norm(long long rows, int D, int io, int res_dtype, const void* x, long long ld_x,
                         const void* res, long long ld_res, float scale, const float* w, float eps, void* out,
                         long long ld_out, void* r, long long ld_r, cudaStream_t s) {
    const int eb = io == SSD_BF16 ? 2 : 4, rb = res_dtype == SSD_BF16 ? 2 : 4;
    const bool vec = D % 8 == 0 && vec_ok(x, ld_x, eb) && vec_ok(res, ld_res, rb) && vec_ok(out, ld_out, eb) &&
                     vec_ok(r, ld_r, rb) && aligned16(w);
    const Shape sh = norm_shape(rows, 1, D, vec, false);
    const ResFwd p{x, res, w, out, r, rows, ld_x, ld_res, ld_out, ld_r, D, scale, eps};
    const char* name = "ssd_residual_norm";
    if (io == SSD_F32) return launch_norm(name, SSD_NORM_PICK(ssd_residual_norm_kernel, float, float), sh, 1, p, s);
    if (res_dtype == SSD_F32)
        return launch_norm(name, SSD_NORM_PICK(ssd_residual_norm_kernel, __nv_bfloat16, float), sh, 1, p, s);
    return launch_norm(name, SSD_NORM_PICK(ssd_residual_norm_kernel, __nv_bfloat16, __nv_bfloat16), sh, 1, p, s);
}

int launch_residual_norm_backward(long long rows, int D, int io, int res_dtype, const void* dout, long long ld_dout,
                                  const void* r, long long ld_r, const float* w, const void* dro, long long ld_dro,
                                  float scale, float eps, void* dx, long long ld_dx, void* dres, long long ld_dres,
                                  float* dw, void* ws, cudaStream_t s) {
    const int eb = io == SSD_BF16 ? 2 : 4, rb = res_dtype == SSD_BF16 ? 2 : 4;
    const bool vec = D % 8 == 0 && vec_ok(dout, ld_dout, eb) && vec_ok(r, ld_r, rb) && vec_ok(dro, ld_dro, rb) &&
                     vec_ok(dx, ld_dx, eb) && vec_ok(dres, ld_dres, rb) && aligned16(w);
    const Shape sh = norm_shape(rows, 1, D, vec, true);
    const ResBwd p{dout, r, w, dro, dx, dres, dw ? static_cast<float*>(ws) : nullptr, rows, ld_dout, ld_r, ld_dro,
                   ld_dx, ld_dres, D, scale, eps};
    const char* name = "ssd_residual_norm_backward";
    int st;
    if (io == SSD_F32)
        st = launch_norm(name, SSD_NORM_PICK(ssd_residual_norm_backward_kernel, float, float), sh, 1, p, s);
    else if (res_dtype == SSD_F32)
        st = launch_norm(name, SSD_NORM_PICK(ssd_residual_norm_backward_kernel, __nv_bfloat16, float), sh, 1, p, s);
    else
        st = launch_norm(name, SSD_NORM_PICK(ssd_residual_norm_backward_kernel, __nv_bfloat16, __nv_bfloat16), sh, 1,
                         p, s);
    if (st != SSD_OK || !dw) return st;
    return launch_dweight(static_cast<float*>(ws), dw, sh.blocks * sh.seg, D, s);
}

int launch_gated_norm(long long rows, int D, int groups, int io, int norm_first, const void* y, long long ld_y,
                      const void* z, long long ld_z, const float* w, float eps, void* out, long long ld_out,
                      cudaStream_t s) {
    const int eb = io == SSD_BF16 ? 2 : 4, L = D / groups;
    const bool vec = L % 8 == 0 && vec_ok(y, ld_y, eb) && vec_ok(z, ld_z, eb) && vec_ok(out, ld_out, eb) && aligned16(w);
    const Shape sh = norm_shape(rows, groups, L, vec, false);
    const GateFwd p{y, z, w, out, rows, ld_y, ld_z, ld_out, D, L, eps};
    const char* name = "ssd_gated_norm";
    if (io == SSD_F32)
        return norm_first ? launch_norm(name, SSD_NORM_PICK(ssd_gated_norm_kernel, float, true), sh, groups, p, s)
                          : launch_norm(name, SSD_NORM_PICK(ssd_gated_norm_kernel, float, false), sh, groups, p, s);
    return norm_first ? launch_norm(name, SSD_NORM_PICK(ssd_gated_norm_kernel, __nv_bfloat16, true), sh, groups, p, s)
                      : launch_norm(name, SSD_NORM_PICK(ssd_gated_norm_kernel, __nv_bfloat16, false), sh, groups, p, s);
}

int launch_gated_norm_backward(long long rows, int D, int groups, int io, int norm_first, const void* dout,
                               long long ld_dout, const void* y, long long ld_y, const void* z, long long ld_z,
                               const float* w, float eps, void* dy, long long ld_dy, void* dz, long long ld_dz,
                               float* dw, void* ws, cudaStream_t s) {
    const int eb = io == SSD_BF16 ? 2 : 4, L = D / groups;
    const bool vec = L % 8 == 0 && vec_ok(dout, ld_dout, eb) && vec_ok(y, ld_y, eb) && vec_ok(z, ld_z, eb) &&
                     vec_ok(dy, ld_dy, eb) && vec_ok(dz, ld_dz, eb) && aligned16(w);
    const Shape sh = norm_shape(rows, groups, L, vec, true);
    const GateBwd p{dout, y, z, w, dy, dz, dw ? static_cast<float*>(ws) : nullptr, rows, ld_dout, ld_y, ld_z, ld_dy,
                    ld_dz, D, L, eps};
    const char* name = "ssd_gated_norm_backward";
    int st;
    if (io == SSD_F32)
        st = norm_first ? launch_norm(name, SSD_NORM_PICK(ssd_gated_norm_backward_kernel, float, true), sh, groups, p, s)
                        : launch_norm(name, SSD_NORM_PICK(ssd_gated_norm_backward_kernel, float, false), sh, groups, p, s);
    else
        st = norm_first
                 ? launch_norm(name, SSD_NORM_PICK(ssd_gated_norm_backward_kernel, __nv_bfloat16, true), sh, groups, p, s)
                 : launch_norm(name, SSD_NORM_PICK(ssd_gated_norm_backward_kernel, __nv_bfloat16, false), sh, groups, p, s);
    if (st != SSD_OK || !dw) return st;
    return launch_dweight(static_cast<float*>(ws), dw, sh.blocks * sh.seg, D, s);
}

}  // namespace ssd
