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
// Bound: device memory, with the issue of instructions close behind in the gated backward pass.
// Each operand is read once and each result written once; a segment (a row, or one group of a row)
// stays in registers, as stored, between its reductions and its results.  A segment belongs to
// `tps` threads of a block (blockDim.x), 8 elements a thread up to 1024 threads, blockDim.y
// segments side by side; the block walks rows by a grid stride with its weights in registers.
// Measured in a graph of calls, against a copy's 6.55 TB/s: residual forward 154 us, 100 %, and backward
// 201 us, 102 % (32768 x 2560, bf16, fp32 residual; bf16 residual 114 and 143 us, 90 %), gated forward
// 94 us, 82 % (16384 x 5120 in 8 groups), and backward 163 us, 78 % (one group), in either order.  Copies
// to shared memory some rows ahead (cp.async) were slower than loads by more threads.  In the backward
// pass the thread owns the same columns of every row it sees, so dw is summed in registers over the rows, stored
// once per block to the workspace, and a second kernel adds the blocks' sums in a fixed order (no
// atomics: the same call gives the same bits).
#include <algorithm>
#include <cmath>
#include <type_traits>
#include "tc.cuh"

namespace ssd {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kWarpThreads = 256;   // blocks of a warp a segment
constexpr int kPairThreads = 640;   // blocks up to here are built with more registers a thread
constexpr int kMaxBlocksPerSM = 8;
constexpr int kSumRows = 32;        // threads along the parts in the dw sum kernel

// Two fp32 values, operation by operation.  (The packed fp32 instructions of sm_100 hold such a pair in an
// aligned register pair: they save issue slots here and cost registers and moves, level at best.)
struct f2 { float x, y; };
__device__ __forceinline__ f2 both(float a) { return {a, a}; }
__device__ __forceinline__ f2 mul(f2 a, f2 b) { return {a.x * b.x, a.y * b.y}; }
__device__ __forceinline__ f2 fma(f2 a, f2 b, f2 c) { return {fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)}; }

// ---- a thread's V elements of an operand as stored (V = 8: 16-byte accesses; V = 2: two elements,
// one by one), and as pairs of fp32
template <typename T, int V> struct Raw;
template <> struct Raw<float, 8> { float4 a, b; };
template <> struct Raw<__nv_bfloat16, 8> { uint4 a; };
template <typename T> struct Raw<T, 2> { T a, b; };

__device__ __forceinline__ void load(Raw<float, 8>& r, const float* p, int) {
    r.a = *reinterpret_cast<const float4*>(p), r.b = *reinterpret_cast<const float4*>(p + 4);
}
__device__ __forceinline__ void load(Raw<__nv_bfloat16, 8>& r, const __nv_bfloat16* p, int) {
    r.a = *reinterpret_cast<const uint4*>(p);
}
template <typename T> __device__ __forceinline__ void load(Raw<T, 2>& r, const T* p, int n) {  // n: elements there are
    r.a = p[0];
    r.b = n > 1 ? p[1] : T(0.f);
}
__device__ __forceinline__ float f32(float v) { return v; }
__device__ __forceinline__ float f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ f2 pair(const Raw<float, 8>& r, int j) {
    return j == 0 ? f2{r.a.x, r.a.y} : j == 1 ? f2{r.a.z, r.a.w} : j == 2 ? f2{r.b.x, r.b.y} : f2{r.b.z, r.b.w};
}
__device__ __forceinline__ f2 pair(const Raw<__nv_bfloat16, 8>& r, int j) {
    const uint32_t u = j == 0 ? r.a.x : j == 1 ? r.a.y : j == 2 ? r.a.z : r.a.w;
    return f2{__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)};
}
template <typename T> __device__ __forceinline__ f2 pair(const Raw<T, 2>& r, int) { return f2{f32(r.a), f32(r.b)}; }

// Keeps the compiler from carrying the unpacked values of a bf16 operand across a reduction beside
// the stored ones: they are unpacked again behind it, for half the registers.
__device__ __forceinline__ void repack(Raw<__nv_bfloat16, 8>& r) {
    asm volatile("" : "+r"(r.a.x), "+r"(r.a.y), "+r"(r.a.z), "+r"(r.a.w));
}
template <typename R> __device__ __forceinline__ void repack(R&) {}

__device__ __forceinline__ void store(float* p, const f2 (&v)[4], int) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const f2 (&v)[4], int) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[i].x, v[i].y);
        u[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
template <typename T> __device__ __forceinline__ void store(T* p, const f2 (&v)[1], int n) {
    put(p, v[0].x);
    if (n > 1) put(p + 1, v[0].y);
}

// Sum of a (and b) over the threads of one segment.  A segment of at most 32 threads is one
// warp; longer ones meet in shared memory.  `red` holds 2 x [blockDim.y][32] pairs used in
// turn (`flip`), so one barrier a row is enough: a block can be at most one row ahead of its
// slowest warp.  Every thread of the block calls this the same number of times.
template <bool kTwo>
__device__ __forceinline__ float2 segment_sum(float a, float b, float2* red, int flip) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        if (kTwo) b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (blockDim.x == 32) return make_float2(a, b);
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    float2* mine = red + (flip * blockDim.y + threadIdx.y) * 32;
    if (lane == 0) mine[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 t = lane < nw ? mine[lane] : make_float2(0.f, 0.f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
        if (kTwo) t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
    }
    return t;
}

// The same for two sums in half the shuffles: after one exchange lanes 0-15 hold the warp's half sums
// of a and lanes 16-31 those of b, and the steps that follow add both.  For the gated backward pass,
// which is bound by its instructions (8192 x 8192: 203 -> 193 us); the residual one waits for memory
// and loses by the longer chain (231 -> 237 us).
__device__ __forceinline__ float2 segment_sum_packed(float a, float b, float2* red, int flip) {
    const int lane = threadIdx.x & 31;
    const bool up = lane & 16;
    float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (blockDim.x > 32) {
        const int nw = blockDim.x >> 5, i = lane & 15;
        float* mine = reinterpret_cast<float*>(red + (flip * blockDim.y + threadIdx.y) * 32) + (up ? 32 : 0);
        if (i == 0) mine[threadIdx.x >> 5] = v;
        __syncthreads();
        v = i < nw ? mine[i] : 0.f;
        if (i + 16 < nw) v += mine[i + 16];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
}

// The gate's sigmoid.  For bf16 operands 1 / (1 + 2^(-z log2 e)) by the two approximate instructions
// (2 ulp each): the product's rounding makes it |z| 2^-24 off for negative z, at most 2^-17 down to
// z = -87.3, below which it is zero (silu(z) above -1.1e-36); the results round by 2^-8.  For fp32 operands
// e^z / (1 + e^z) or 1 / (1 + e^-z), whichever has the exponential below one: no larger error for closed
// gates, and none lost before the exponential itself is.
__device__ __forceinline__ float sigmoid1(__nv_bfloat16, float z) {
    float a = z * -1.4426950408889634f;
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    a += 1.f;
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    return a;
}
__device__ __forceinline__ float sigmoid1(float, float z) {
    const float e = expf(-fabsf(z));
    float r = 1.f + e;
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(r));
    return z < 0.f ? e * r : r;
}
template <typename T> __device__ __forceinline__ f2 sigmoid2(f2 z) { return {sigmoid1(T(), z.x), sigmoid1(T(), z.y)}; }

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

// Common to the kernels below.  V elements an access; a thread's accesses of a segment lie V tps
// elements apart.  col: element of an access, left: elements the segment has there (<= 0: none).
// An element's address is the operand's place at the block's row, the same for all threads and so
// held in uniform registers, and a 32-bit byte offset of the thread.
#define SSD_NORM_PROLOGUE(LEN)                                                                            \
    extern __shared__ float2 red[];                                                                       \
    constexpr int kPairs = V / 2;                                                                         \
    const int tps = blockDim.x;                                                                           \
    const float inv_len = 1.f / (float)(LEN);                                                             \
    int col[VPT], left[VPT];                                                                              \
    _Pragma("unroll") for (int i = 0; i < VPT; ++i) {                                                     \
        col[i] = (i * tps + (int)threadIdx.x) * V;                                                        \
        left[i] = (LEN) - col[i];                                                                         \
    }                                                                                                     \
    int flip = 0;
#define SSD_NORM_ROWS                                                                                     \
    for (long long row = (long long)blockIdx.x * blockDim.y; row < p.rows; row += (long long)gridDim.x * blockDim.y)
// an operand: its first element, row stride, and the thread's offset
template <typename T> struct At {
    T* p;
    long long ld;
    uint32_t off;
    __device__ __forceinline__ At(T* p_, long long ld_) : p(p_), ld(ld_), off((uint32_t)(threadIdx.y * ld_ * sizeof(T))) {}
    __device__ __forceinline__ T* operator()(long long row, int col) const {
        using C = typename std::conditional<std::is_const<T>::value, const char, char>::type;
        return reinterpret_cast<T*>(reinterpret_cast<C*>(p + row * ld) + (off + (uint32_t)col * (uint32_t)sizeof(T)));
    }
};
// The operands of a row: loaded DEPTH rows ahead where the registers allow, so that memory is busy
// through a row's reduction and stores.
#define SSD_NORM_FIRST(DEPTH)                                                                             \
    constexpr int kAhead = VPT == 1 && kThr == kPairThreads ? (DEPTH) : 0;                                \
    const long long step = (long long)gridDim.x * blockDim.y;                                             \
    Row cur = {}, next[kAhead > 0 ? kAhead : 1] = {};                                                     \
    _Pragma("unroll") for (int d = 0; d < kAhead; ++d) fetch(next[d], (long long)blockIdx.x * blockDim.y + d * step);
#define SSD_NORM_NEXT                                                                                     \
    if constexpr (kAhead > 0) {                                                                           \
        cur = next[0];                                                                                    \
        _Pragma("unroll") for (int d = 0; d + 1 < kAhead; ++d) next[d] = next[d + 1];                     \
        fetch(next[kAhead - 1], row + kAhead * step);                                                     \
    } else {                                                                                              \
        fetch(cur, row);                                                                                  \
    }
// The weights: in registers, or where a thread has none to spare (kLean: blocks above kPairThreads,
// and several accesses a thread) read again for every row, from the L1 cache.
#define SSD_NORM_WEIGHT(SRC)                                                                              \
    constexpr bool kLean = kThr > kPairThreads;                                                           \
    const float* const wsrc = (SRC);                                                                      \
    f2 wreg[kLean ? 1 : VPT][kLean ? 1 : kPairs];                                                         \
    if constexpr (!kLean) {                                                                               \
        _Pragma("unroll") for (int i = 0; i < VPT; ++i) {                                                 \
            Raw<float, V> raw = {};                                                                       \
            if (left[i] > 0) load(raw, wsrc + col[i], left[i]);                                           \
            _Pragma("unroll") for (int j = 0; j < kPairs; ++j) wreg[i][j] = pair(raw, j);                 \
        }                                                                                                 \
    }                                                                                                     \
    /* weights of pair j of access i, which the segment has */                                            \
    auto w = [&](int i, int j) -> f2 {                                                                    \
        if constexpr (!kLean) return wreg[i][j];                                                          \
        else if constexpr (V == 8) {                                                                      \
            const float2 v = __ldg(reinterpret_cast<const float2*>(wsrc + col[i]) + j);                   \
            return {v.x, v.y};                                                                            \
        } else return {__ldg(wsrc + col[i]), left[i] > 1 ? __ldg(wsrc + col[i] + 1) : 0.f};               \
    };
#define SSD_NORM_DW                                                                                       \
    f2 dw[VPT][kPairs];                                                                                   \
    _Pragma("unroll") for (int i = 0; i < VPT; ++i)                                                       \
        _Pragma("unroll") for (int j = 0; j < kPairs; ++j) dw[i][j] = {};
#define SSD_NORM_DW_STORE(BASE)                                                                           \
    if (p.part) {                                                                                         \
        float* part = p.part + (size_t)(blockIdx.x * blockDim.y + threadIdx.y) * p.D + (BASE);            \
        _Pragma("unroll") for (int i = 0; i < VPT; ++i)                                                   \
            if (left[i] > 0) store(part + col[i], dw[i], left[i]);                                        \
    }
__device__ __forceinline__ float hsum(f2 v) { return v.x + v.y; }

template <typename TIO, typename TRES, int V, int VPT, int kThr>
__global__ void __launch_bounds__(kThr, kThr == kPairThreads ? 2 : 1) ssd_residual_norm_kernel(const ResFwd p) {
    SSD_NORM_PROLOGUE(p.D)
    SSD_NORM_WEIGHT(p.w)
    const f2 scale2 = both(p.scale);
    const At<const TIO> px(static_cast<const TIO*>(p.x), p.ld_x);
    const At<const TRES> pres(static_cast<const TRES*>(p.res), p.ld_res);
    const At<TIO> pout(static_cast<TIO*>(p.out), p.ld_out);
    const At<TRES> pr(static_cast<TRES*>(p.r), p.ld_r);
    SSD_NORM_ROWS {
        const bool in = row + threadIdx.y < p.rows;
        f2 r[VPT][kPairs], ss = {};
        Raw<TIO, V> x[VPT] = {};
        Raw<TRES, V> res[VPT] = {};
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && left[i] > 0) {
                load(x[i], px(row, col[i]), left[i]);
                if (p.res) load(res[i], pres(row, col[i]), left[i]);
            }
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                r[i][j] = fma(scale2, pair(x[i], j), pair(res[i], j));
                ss = fma(r[i][j], r[i][j], ss);
            }
        const float k = rsqrtf(segment_sum<false>(hsum(ss), 0.f, red, flip).x * inv_len + p.eps);
        flip ^= 1;
        const f2 k2 = both(k);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && left[i] > 0) {
                if (p.r) store(pr(row, col[i]), r[i], left[i]);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) r[i][j] = mul(mul(r[i][j], k2), w(i, j));
                store(pout(row, col[i]), r[i], left[i]);
            }
    }
}

template <typename TIO, typename TRES, int V, int VPT, int kThr>
__global__ void __launch_bounds__(kThr) ssd_residual_norm_backward_kernel(const ResBwd p) {
    SSD_NORM_PROLOGUE(p.D)
    SSD_NORM_WEIGHT(p.w)
    SSD_NORM_DW
    if (p.part) griddep_launch();  // the weight gradient follows, and waits
    const f2 scale2 = both(p.scale);
    const At<const TIO> pg(static_cast<const TIO*>(p.dout), p.ld_dout);
    const At<const TRES> pr(static_cast<const TRES*>(p.r), p.ld_r), pd(static_cast<const TRES*>(p.dr_out), p.ld_dro);
    const At<TIO> pdx(static_cast<TIO*>(p.dx), p.ld_dx);
    const At<TRES> pdres(static_cast<TRES*>(p.dres), p.ld_dres);
    struct Row {
        Raw<TRES, V> r[VPT], d[VPT];
        Raw<TIO, V> g[VPT];
    };
    auto fetch = [&](Row& o, long long row) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (row + threadIdx.y < p.rows && left[i] > 0) {
                load(o.r[i], pr(row, col[i]), left[i]);
                load(o.g[i], pg(row, col[i]), left[i]);
                if (p.dr_out) load(o.d[i], pd(row, col[i]), left[i]);
            }
    };
    SSD_NORM_FIRST(1)
    SSD_NORM_ROWS {
        const bool in = row + threadIdx.y < p.rows;
        f2 ss = {}, gr = {};
        SSD_NORM_NEXT
        auto &r = cur.r, &d = cur.d;
        auto& g = cur.g;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && left[i] > 0) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const f2 rv = pair(r[i], j);
                    ss = fma(rv, rv, ss);
                    gr = fma(mul(pair(g[i], j), w(i, j)), rv, gr);
                }
            }
        const float2 sum = segment_sum<true>(hsum(ss), hsum(gr), red, flip);
        flip ^= 1;
        const float k = rsqrtf(sum.x * inv_len + p.eps);
        const f2 k2 = both(k), m2 = both(-sum.y * inv_len * k * k);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && left[i] > 0) {
                f2 o[kPairs];
                repack(r[i]), repack(g[i]), repack(d[i]);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const f2 rv = pair(r[i], j), gv = pair(g[i], j);
                    dw[i][j] = fma(gv, mul(rv, k2), dw[i][j]);
                    o[j] = fma(k2, fma(rv, m2, mul(gv, w(i, j))), pair(d[i], j));
                }
                if (p.dres) store(pdres(row, col[i]), o, left[i]);
                if (p.dx) {
#pragma unroll
                    for (int j = 0; j < kPairs; ++j) o[j] = mul(o[j], scale2);
                    store(pdx(row, col[i]), o, left[i]);
                }
            }
    }
    SSD_NORM_DW_STORE(0)
}

// Vectors a thread up to which the forward pass runs three blocks of warp segments an SM (two beyond).
__host__ __device__ constexpr int three_blocks(bool bf16, bool norm_first) { return !bf16 ? 0 : norm_first ? 2 : 3; }

template <typename TIO, bool kNormFirst, int V, int VPT, int kThr>
__global__ void __launch_bounds__(kThr, kThr != kWarpThreads ? 0 : VPT <= three_blocks(sizeof(TIO) == 2, kNormFirst) ? 3 : 2)
ssd_gated_norm_kernel(const GateFwd p) {
    SSD_NORM_PROLOGUE(p.L)
    const int base = blockIdx.y * p.L;
    SSD_NORM_WEIGHT(p.w + base)
    const At<const TIO> py(static_cast<const TIO*>(p.y) + base, p.ld_y), pz(static_cast<const TIO*>(p.z) + base, p.ld_z);
    const At<TIO> pout(static_cast<TIO*>(p.out) + base, p.ld_out);
    struct Row {
        Raw<TIO, V> y[VPT], z[VPT];
    };
    auto fetch = [&](Row& o, long long row) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (row + threadIdx.y < p.rows && left[i] > 0) {
                load(o.y[i], py(row, col[i]), left[i]);
                load(o.z[i], pz(row, col[i]), left[i]);
            }
    };
    SSD_NORM_FIRST(1)
    SSD_NORM_ROWS {
        const bool in = row + threadIdx.y < p.rows;
        f2 a[VPT][kPairs], gt[VPT][kPairs], ss = {};  // a: what is normalised; gt: silu(z)
        SSD_NORM_NEXT
        auto &y = cur.y, &z = cur.z;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const f2 zv = pair(z[i], j);
                gt[i][j] = mul(zv, sigmoid2<TIO>(zv));
                a[i][j] = kNormFirst ? pair(y[i], j) : mul(pair(y[i], j), gt[i][j]);
                ss = fma(a[i][j], a[i][j], ss);
            }
        const float k = rsqrtf(segment_sum<false>(hsum(ss), 0.f, red, flip).x * inv_len + p.eps);
        flip ^= 1;
        const f2 k2 = both(k);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && left[i] > 0) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    a[i][j] = mul(mul(a[i][j], k2), w(i, j));
                    if (kNormFirst) a[i][j] = mul(a[i][j], gt[i][j]);
                }
                store(pout(row, col[i]), a[i], left[i]);
            }
    }
}

// (One block an SM asked for by name gives the compiler 96 registers up to 640 threads; left open it
// takes fewer and is slower, 165 against 120 us for 30000 x 1025.  At 1024 threads it is the other way
// round, 207 against 193 us for 8192 x 8192.)
template <typename TIO, bool kNormFirst, int V, int VPT, int kThr>
__global__ void __launch_bounds__(kThr, kThr == kWarpThreads ? 2 : kThr == kPairThreads ? 1 : 0)
ssd_gated_norm_backward_kernel(const GateBwd p) {
    SSD_NORM_PROLOGUE(p.L)
    const int base = blockIdx.y * p.L;
    SSD_NORM_WEIGHT(p.w + base)
    SSD_NORM_DW
    if (p.part) griddep_launch();  // the weight gradient follows, and waits
    const At<const TIO> pg(static_cast<const TIO*>(p.dout) + base, p.ld_dout), py(static_cast<const TIO*>(p.y) + base, p.ld_y),
        pz(static_cast<const TIO*>(p.z) + base, p.ld_z);
    const At<TIO> pdy(static_cast<TIO*>(p.dy) + base, p.ld_dy), pdz(static_cast<TIO*>(p.dz) + base, p.ld_dz);
    struct Row {
        Raw<TIO, V> y[VPT], z[VPT], g[VPT];
    };
    auto fetch = [&](Row& o, long long row) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (row + threadIdx.y < p.rows && left[i] > 0) {
                load(o.z[i], pz(row, col[i]), left[i]);
                load(o.y[i], py(row, col[i]), left[i]);
                load(o.g[i], pg(row, col[i]), left[i]);
            }
    };
    SSD_NORM_FIRST(1)
    SSD_NORM_ROWS {
        const bool in = row + threadIdx.y < p.rows;
        f2 ss = {}, gv = {}, sg[kLean ? 1 : VPT][kLean ? 1 : kPairs];
        SSD_NORM_NEXT
        auto &y = cur.y, &z = cur.z, &g = cur.g;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && left[i] > 0) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const f2 zv = pair(z[i], j), s1 = sigmoid2<TIO>(zv), gate = mul(zv, s1);
                    if constexpr (!kLean) sg[i][j] = s1;
                    const f2 n = kNormFirst ? pair(y[i], j) : mul(pair(y[i], j), gate);              // what is normalised
                    const f2 t = mul(kNormFirst ? mul(pair(g[i], j), gate) : pair(g[i], j), w(i, j));  // its gradient over k
                    ss = fma(n, n, ss);
                    gv = fma(t, n, gv);
                }
            }
        const float2 sum = segment_sum_packed(hsum(ss), hsum(gv), red, flip);
        flip ^= 1;
        const float k = rsqrtf(sum.x * inv_len + p.eps);
        const f2 k2 = both(k), m2 = both(-sum.y * inv_len * k * k);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in && left[i] > 0) {
                f2 dy[kPairs], dz[kPairs];
                repack(y[i]), repack(z[i]), repack(g[i]);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const f2 zv = pair(z[i], j), yv = pair(y[i], j), go = pair(g[i], j);
                    f2 s1;
                    if constexpr (kLean) s1 = sigmoid2<TIO>(zv);
                    else s1 = sg[i][j];
                    const f2 gate = mul(zv, s1);
                    const f2 dgate = fma(gate, fma(s1, both(-1.f), both(1.f)), s1);  // silu'(z)
                    if (kNormFirst) {
                        const f2 n = mul(yv, k2), t = mul(go, gate);
                        dw[i][j] = fma(t, n, dw[i][j]);
                        dy[j] = mul(k2, fma(yv, m2, mul(t, w(i, j))));
                        dz[j] = mul(mul(go, n), mul(w(i, j), dgate));
                    } else {
                        const f2 n = mul(yv, gate);
                        dw[i][j] = fma(go, mul(n, k2), dw[i][j]);
                        const f2 dn = mul(k2, fma(n, m2, mul(go, w(i, j))));
                        dy[j] = mul(dn, gate);
                        dz[j] = mul(mul(dn, yv), dgate);
                    }
                }
                store(pdy(row, col[i]), dy, left[i]);
                store(pdz(row, col[i]), dz, left[i]);
            }
    }
    SSD_NORM_DW_STORE(base)
}

// dw[c] = sum over the parts, in part order per thread row and then over the thread rows.
__global__ void __launch_bounds__(32 * kSumRows) ssd_norm_dweight_kernel(const float* part, float* dw, int parts, int D) {
    __shared__ float s[kSumRows][33];
    griddep_wait();  // started while the backward pass ends
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
    bool warps;  // a warp a segment
    size_t smem;
};

// Threads an SM holds of the one-vector kernels: their registers are up to 48 in the residual forward
// pass, 56 in the gated one on bf16, 96 in the backward passes (which hold dw and a row ahead).
constexpr int kFwdThreads = 1280, kGatedThreads = 1152, kBwdThreads = 672;

// Vector accesses need every operand's row starts on 16 bytes and segments of whole vectors
// (`vec`); otherwise elements are read one by one, in pairs.  A thread takes one vector of a segment
// up to 1024 threads and two beyond: more threads with one vector each measured faster than fewer
// with more (gated backward, 5120 bf16 elements: two vectors a thread took 371 us).
// The gated norm's short segments, from 257 elements, go to a warp each instead, whose sums need no
// barrier, up to as many vectors a thread (`warp_vectors`, 0: never) as its registers hold, and three
// blocks of them an SM up to `three` vectors, where they still fit.  Warps against blocks in us, 84 M
// elements in groups of 384, 640 and 1024 (2 to 4 vectors), the two orders alike but where told:
//   forward bf16   100 117   94 104   84 95            three blocks an SM against two 100 117, 94 97, and
//                                                      norm first, where three spill at 640, 133 98
//   forward fp32   165 167   167 197  174 154 (norm first 192 197)
//   backward bf16  187 210   179 196  227 169
//   backward fp32  279 330   383 307  465 304
// The residual norm, bound by memory, is slower that way (102 against 93 us).
// `ld`: the longest row stride in bytes.  The rows of a block's segments start within 2^32 bytes of
// its first one's (a thread's offset has 32 bits), or the block takes one segment at a time.
Shape norm_shape(long long rows, int groups, int L, bool vec, int warp_vectors, int three, int resident, long long ld) {
    Shape s;
    s.V = vec ? 8 : 2;
    const int n = (L + s.V - 1) / s.V;
    s.warps = vec && n > 32 && n <= 32 * warp_vectors;
    s.vpt = s.warps ? (n + 31) / 32 : n <= kMaxThreads ? 1 : vec ? 2 : n <= 4 * kMaxThreads ? 4 : 8;
    s.tps = ((n + s.vpt - 1) / s.vpt + 31) / 32 * 32;
    s.seg = s.tps >= 256 ? 1 : std::max(1, 256 / s.tps);
    const int thr = s.tps * s.seg;
    s.smem = 2 * sizeof(float2) * s.seg * 32;
    // one wave of blocks: each holds its weights, and in the backward pass stores a part of dw
    if (s.warps) resident = (s.vpt <= three ? 3 : 2) * kWarpThreads;
    else if (s.vpt > 1 || thr > kPairThreads) resident = kMaxThreads;
    else if (!vec) resident = kFwdThreads;
    const int per_sm = std::max(1, std::min(kMaxBlocksPerSM, resident / thr));
    if (s.seg > 1 && ld > ((1LL << 32) - 4LL * L) / (s.seg - 1)) {
        s.seg = 1;
        s.smem = 2 * sizeof(float2) * 32;
    }
    const long long want = (rows + s.seg - 1) / s.seg;
    s.blocks = (int)std::min(want, std::max<long long>(1, (long long)device_sms() * per_sm / groups));
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
    SSD_CUDA_TRY(launch_pdl(ssd_norm_dweight_kernel, dim3((D + 31) / 32), dim3(32, kSumRows), 0, s, part, dw, parts, D));
    return SSD_OK;
}

// the kernel of a shape among its instances
#define SSD_NORM_PICK(kernel, A, B)                                                                                    \
    (sh.vpt == 1 ? (sh.tps * sh.seg <= kPairThreads ? (sh.V == 8 ? kernel<A, B, 8, 1, kPairThreads>                    \
                                                                 : kernel<A, B, 2, 1, kPairThreads>)                   \
                                                    : (sh.V == 8 ? kernel<A, B, 8, 1, kMaxThreads>                     \
                                                                 : kernel<A, B, 2, 1, kMaxThreads>))                   \
     : sh.V == 8 ? kernel<A, B, 8, 2, kMaxThreads>                                                                     \
     : sh.vpt == 4 ? kernel<A, B, 2, 4, kMaxThreads> : kernel<A, B, 2, 8, kMaxThreads>)
#define SSD_NORM_WARP2(kernel, A, B) kernel<A, B, 8, 2, kWarpThreads>
#define SSD_NORM_WARP3(kernel, A, B) (sh.vpt == 2 ? SSD_NORM_WARP2(kernel, A, B) : kernel<A, B, 8, 3, kWarpThreads>)
#define SSD_NORM_WARP4(kernel, A, B) (sh.vpt < 4 ? SSD_NORM_WARP3(kernel, A, B) : kernel<A, B, 8, 4, kWarpThreads>)
// WARP: the instances of a warp a segment, up to the type's and direction's vectors below
#define SSD_NORM_PICK_GATED(kernel, A, B, WARP) (sh.warps ? WARP(kernel, A, B) : SSD_NORM_PICK(kernel, A, B))
constexpr int kFwdWarpBf16 = 4, kFwdWarpF32 = 3, kBwdWarpBf16 = 3, kBwdWarpF32 = 2;

bool vec_ok(const void* p, long long ld, int elem) {
    return !p || (aligned16(p) && (ld * elem) % 16 == 0);
}

}  // namespace

// Bytes of the backward passes' workspace: the blocks' sums of dw, for the vector and the
// element shapes alike.
size_t norm_workspace_bytes(long long rows, int D, int groups) {
    const int L = D / groups;
    size_t parts = 0;
    for (int v = 0; v < 3; ++v) {
        if (v && L % 8) continue;
        const Shape s = norm_shape(rows, groups, L, v != 0, v == 2 ? std::max(kBwdWarpBf16, kBwdWarpF32) : 0, 0, kBwdThreads, 0);
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
    const long long ld = std::max({ld_x * eb, ld_out * eb, res ? ld_res * rb : 0, r ? ld_r * rb : 0});
    const Shape sh = norm_shape(rows, 1, D, vec, 0, 0, kFwdThreads, ld);
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
    const long long ld =
        std::max({ld_dout * eb, ld_r * rb, dro ? ld_dro * rb : 0, dx ? ld_dx * eb : 0, dres ? ld_dres * rb : 0});
    const Shape sh = norm_shape(rows, 1, D, vec, 0, 0, kBwdThreads, ld);
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
    const Shape sh = norm_shape(rows, groups, L, vec, io == SSD_BF16 ? kFwdWarpBf16 : kFwdWarpF32,
                                three_blocks(io == SSD_BF16, norm_first != 0), kGatedThreads, std::max({ld_y, ld_z, ld_out}) * eb);
    const GateFwd p{y, z, w, out, rows, ld_y, ld_z, ld_out, D, L, eps};
    const char* name = "ssd_gated_norm";
    if (io == SSD_F32)
        return launch_norm(name,
                           norm_first ? SSD_NORM_PICK_GATED(ssd_gated_norm_kernel, float, true, SSD_NORM_WARP3)
                                      : SSD_NORM_PICK_GATED(ssd_gated_norm_kernel, float, false, SSD_NORM_WARP3),
                           sh, groups, p, s);
    return launch_norm(name,
                       norm_first ? SSD_NORM_PICK_GATED(ssd_gated_norm_kernel, __nv_bfloat16, true, SSD_NORM_WARP4)
                                  : SSD_NORM_PICK_GATED(ssd_gated_norm_kernel, __nv_bfloat16, false, SSD_NORM_WARP4),
                       sh, groups, p, s);
}

int launch_gated_norm_backward(long long rows, int D, int groups, int io, int norm_first, const void* dout,
                               long long ld_dout, const void* y, long long ld_y, const void* z, long long ld_z,
                               const float* w, float eps, void* dy, long long ld_dy, void* dz, long long ld_dz,
                               float* dw, void* ws, cudaStream_t s) {
    const int eb = io == SSD_BF16 ? 2 : 4, L = D / groups;
    const bool vec = L % 8 == 0 && vec_ok(dout, ld_dout, eb) && vec_ok(y, ld_y, eb) && vec_ok(z, ld_z, eb) &&
                     vec_ok(dy, ld_dy, eb) && vec_ok(dz, ld_dz, eb) && aligned16(w);
    const Shape sh = norm_shape(rows, groups, L, vec, io == SSD_BF16 ? kBwdWarpBf16 : kBwdWarpF32, 0, kBwdThreads,
                                std::max({ld_dout, ld_y, ld_z, ld_dy, ld_dz}) * eb);
    const GateBwd p{dout, y, z, w, dy, dz, dw ? static_cast<float*>(ws) : nullptr, rows, ld_dout, ld_y, ld_z, ld_dy,
                    ld_dz, D, L, eps};
    const char* name = "ssd_gated_norm_backward";
    int st;
    if (io == SSD_F32)
        st = launch_norm(name,
                         norm_first ? SSD_NORM_PICK_GATED(ssd_gated_norm_backward_kernel, float, true, SSD_NORM_WARP2)
                                    : SSD_NORM_PICK_GATED(ssd_gated_norm_backward_kernel, float, false, SSD_NORM_WARP2),
                         sh, groups, p, s);
    else
        st = launch_norm(name,
                         norm_first ? SSD_NORM_PICK_GATED(ssd_gated_norm_backward_kernel, __nv_bfloat16, true, SSD_NORM_WARP3)
                                    : SSD_NORM_PICK_GATED(ssd_gated_norm_backward_kernel, __nv_bfloat16, false, SSD_NORM_WARP3),
                         sh, groups, p, s);
    if (st != SSD_OK || !dw) return st;
    return launch_dweight(static_cast<float*>(ws), dw, sh.blocks * sh.seg, D, s);
}

}  // namespace ssd
