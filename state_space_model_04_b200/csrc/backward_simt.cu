// backward_simt.cu -- gradients of the SSD prefill on the fp32 pipes: every fp32 call, and bf16
// calls whose shape the tensor-core path does not take.
//
// The recurrence h_t = e^{a_t} h_{t-1} + dt_t x_t B_t^T, y_t = h_t C_t + D x_t (a = dt A) and its
// adjoint run in the chunked dual form, kQ = 64 tokens a chunk.  With cs the prefix sum of a in
// the chunk, L_ij = exp(cs_i - cs_j) for i >= j, S = C B^T, Gm = dy x^T, h the state entering
// the chunk and dh the adjoint of the state leaving it:
//   dx_j = dt_j U_j + D dy_j,   U_j = sum_i S_ij L_ij dy_i + exp(cs_Q - cs_j) dh B_j
//   dC_i = sum_j dS_ij B_j + exp(cs_i) h^T dy_i,        dS_ij = Gm_ij L_ij dt_j
//   dB_j = sum_i dS_ij C_i + dt_j exp(cs_Q - cs_j) dh^T x_j
//   ddt_t = x_t . U_t + A da_t
//   da_t = exp(cs_Q) <h, dh> + sum_{i >= t} E_i + sum_{j < t} F_j + sum_{i >= t > j} W_ij
//   W = Gm S L dt,  E_i = exp(cs_i) dy_i . h C_i,  F_j = dt_j exp(cs_Q - cs_j) x_j . dh B_j
// da_t adds the pairs (i, j) that straddle t, as a suffix sum of W's row sums less its column
// sums over i > j: no term of the whole sequence's length enters.  Both sums are of the same fp32
// numbers and in fp64, so what has to cancel does: behind a step that erases the state nothing may be
// left, as dA takes da_t times that step.
//
// Launches: decay terms and the chunks' own states in both directions; a scan over the chunks (in
// place: slot c ends up with the state entering chunk c, or the adjoint of the state leaving
// it); the gradients per chunk, a block walking heads of one B/C group with dB and dC in
// registers; sums.  Bound by the fp32 pipes and the shared memory that feeds them: per token and
// head about 57,000 multiply-adds at N = 128 against 4 KB of state traffic (two fp32 states a chunk, each
// written twice and read twice).  4 x 2048 tokens, 48
// heads, N = 128, fp32: 1.82 ms, 25 TFLOP/s, a third of the fp32 pipes' rate.
#include <algorithm>
#include "backward.cuh"
#include "tc.cuh"

namespace ssd {
namespace {

constexpr int kQ = 64, kP = 64;
constexpr int kThreads = 256;

struct SimtBwd {
    BwdArgs a;
    int nc;       // chunks a sequence
    int splits;   // blocks a (chunk, group)
    float* dtv;   // [b nc][H][kQ] step sizes, 0 past the end
    double* cs;   // [b nc][H][kQ] inclusive prefix sums of dt A
    float* e;     // [b nc][H][kQ] exp(cs)
    float* w;     // [b nc][H][kQ] exp(cs_Q - cs)
    float* hs;    // [b nc][H][P][N] the chunk's own state, then the state entering it
    float* gs;    // [b nc][H][P][N] the chunk's own adjoint, then the adjoint of the state leaving it
    float* part;  // [2][splits][b][T][G][N] sums of dB, dC over a block's heads (splits > 1)
    float *pA, *pD, *pb;  // [b nc][H] sums of dA, dD and the bias gradient over a chunk
};

// Tiles are [rows][W] floats; the 16-byte piece c of row r sits at piece c ^ (r / 4 % 8), so that
// threads reading 8 rows 4 apart at one piece, or 8 pieces of one row, meet no bank conflict.
template <int W> __device__ __forceinline__ int at(int r, int c4) { return r * W + ((c4 ^ ((r >> 2) & 7)) << 2); }

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void st4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void st4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), c = __floats2bfloat162_rn(v.z, v.w);
    uint2 u;
    u.x = *reinterpret_cast<const uint32_t*>(&a);
    u.y = *reinterpret_cast<const uint32_t*>(&c);
    *reinterpret_cast<uint2*>(p) = u;
}

// A [kQ][W] tile from rows `stride` elements apart; rows from `valid` on are zero.
template <int W, int kThr, typename T>
__device__ __forceinline__ void load_tile(float* dst, const T* src, size_t stride, int valid) {
#pragma unroll 2
    for (int i = threadIdx.x; i < kQ * (W / 4); i += kThr) {
        const int r = i / (W / 4), c = i % (W / 4);
        const float4 v = r < valid ? ld4(src + r * stride + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(dst + at<W>(r, c)) = v;
    }
}

// acc[a][b] += sum_k A[4 ty + a][k] B[4 tx + b][k]  (both along rows)
template <int K>
__device__ __forceinline__ void mm_nt(const float* A, const float* B, int ty, int tx, float (&acc)[4][4]) {
#pragma unroll 1
    for (int k = 0; k < K / 4; ++k) {
        float4 av[4], bv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = ld4(A + at<K>(4 * ty + i, k)), bv[i] = ld4(B + at<K>(4 * tx + i, k));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = fmaf(av[i].x, bv[j].x, acc[i][j]);
                acc[i][j] = fmaf(av[i].y, bv[j].y, acc[i][j]);
                acc[i][j] = fmaf(av[i].z, bv[j].z, acc[i][j]);
                acc[i][j] = fmaf(av[i].w, bv[j].w, acc[i][j]);
            }
    }
}
__device__ __forceinline__ void axpy4(float s, float4 v, float* acc) {
    acc[0] = fmaf(s, v.x, acc[0]);
    acc[1] = fmaf(s, v.y, acc[1]);
    acc[2] = fmaf(s, v.z, acc[2]);
    acc[3] = fmaf(s, v.w, acc[3]);
}
// acc[a][...] += s_a sum_k A[4 ty + a][k] B[k][columns 4 tx .. and 64 + 4 tx ..]   (K = 64, B [64][W])
template <int W>
__device__ __forceinline__ void mm_nn(const float* A, const float* B, int ty, int tx, const float (&s)[4],
                                      float (&acc)[4][W / 16]) {
#pragma unroll 1
    for (int k = 0; k < 16; ++k) {
        float4 av[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            av[i] = ld4(A + at<64>(4 * ty + i, k));
            av[i].x *= s[i], av[i].y *= s[i], av[i].z *= s[i], av[i].w *= s[i];
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int n = 0; n < W / 64; ++n) {
                const float4 bv = ld4(B + at<W>(4 * k + kk, tx + 16 * n));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float m = kk == 0 ? av[i].x : kk == 1 ? av[i].y : kk == 2 ? av[i].z : av[i].w;
                    axpy4(m, bv, &acc[i][4 * n]);
                }
            }
    }
}
// acc[a][...] += sum_k A[k][4 ty + a] B[k][columns 4 tx .. and 64 + 4 tx ..]   (A [64][64], B [64][W])
template <int W>
__device__ __forceinline__ void mm_tn(const float* A, const float* B, int ty, int tx, float (&acc)[4][W / 16]) {
#pragma unroll (W == 64 ? 4 : 2)
    for (int k = 0; k < 64; ++k) {
        const float4 av = ld4(A + at<64>(k, ty));
#pragma unroll
        for (int n = 0; n < W / 64; ++n) {
            const float4 bv = ld4(B + at<W>(k, tx + 16 * n));
            axpy4(av.x, bv, &acc[0][4 * n]);
            axpy4(av.y, bv, &acc[1][4 * n]);
            axpy4(av.z, bv, &acc[2][4 * n]);
            axpy4(av.w, bv, &acc[3][4 * n]);
        }
    }
}

// ---- the chunk's decay terms and its own states: z = 0: sum_j dt_j w_j x_j B_j^T, z = 1:
// sum_i e_i dy_i C_i^T.  Both directions need the terms; one stores them.
template <typename TIO, int N>
__global__ void __launch_bounds__(kThreads) ssd_bwd_chunk_states_kernel(const SimtBwd p) {
    griddep_launch();
    extern __shared__ float sm[];
    float *sx = sm, *sb = sm + kQ * kP, *s_scale = sb + kQ * N;
    const int h = blockIdx.x % p.a.H, bc = blockIdx.x / p.a.H, dir = blockIdx.y;
    const int bi = bc / p.nc, t0 = (bc % p.nc) * kQ, g = h / (p.a.H / p.a.G);
    const int valid = min(kQ, p.a.T - t0);
    const size_t tok = (size_t)bi * p.a.T + t0;
    const int lane = threadIdx.x;
    float dt[2] = {};
    if (lane < 32) {  // two tokens a lane
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (2 * lane + k < valid) dt[k] = p.a.dt[(tok + 2 * lane + k) * p.a.H + h];
    }
    const TIO* xs = static_cast<const TIO*>(dir ? p.a.dy : p.a.x) + (tok * p.a.H + h) * kP;
    constexpr int kRows = kThreads / (kP / 4);  // rows of x the block reads at once
    const int xr = threadIdx.x / (kP / 4), xc = threadIdx.x % (kP / 4);
    float4 x[kQ / kRows];
#pragma unroll
    for (int i = 0; i < kQ / kRows; ++i) {
        const int r = i * kRows + xr;
        x[i] = r < valid ? ld4(xs + (size_t)r * p.a.H * kP + 4 * xc) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    load_tile<N, kThreads>(sb, static_cast<const TIO*>(dir ? p.a.C : p.a.B) + (tok * p.a.G + g) * N, (size_t)p.a.G * N, valid);
    if (lane < 32) {
        const double Ah = p.a.A[h];
#pragma unroll
        for (int k = 0; k < 2; ++k) dt[k] = 2 * lane + k < valid ? dt_value(dt[k], p.a.dtm, h) : 0.f;
        const double a0 = dt[0] * Ah, a1 = dt[1] * Ah;
        double s = a0 + a1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double v = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += v;
        }
        const double tot = __shfl_sync(0xffffffffu, s, 31);
        const size_t o = (size_t)blockIdx.x * kQ + 2 * lane;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const double c = k ? s : s - a1;
            const float e = expf((float)c), w = expf((float)(tot - c));
            s_scale[2 * lane + k] = dir ? e : w * dt[k];
            if (!dir) p.dtv[o + k] = dt[k], p.cs[o + k] = c, p.e[o + k] = e, p.w[o + k] = w;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQ / kRows; ++i) {
        const int r = i * kRows + xr;
        const float f = s_scale[r];
        x[i].x *= f, x[i].y *= f, x[i].z *= f, x[i].w *= f;
        *reinterpret_cast<float4*>(sx + at<64>(r, xc)) = x[i];
    }
    __syncthreads();
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    float acc[4][N / 16] = {};
    mm_tn<N>(sx, sb, ty, tx, acc);
    float* dst = (dir ? p.gs : p.hs) + (size_t)blockIdx.x * kP * N;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < N / 64; ++n)
            st4(dst + (4 * ty + i) * N + 64 * n + 4 * tx,
                make_float4(acc[i][4 * n], acc[i][4 * n + 1], acc[i][4 * n + 2], acc[i][4 * n + 3]));
}

// ---- scan over the chunks, four state entries a thread; z = 0 forwards, z = 1 backwards
constexpr int kAhead = 8;  // chunks loaded ahead of the dependent updates
__global__ void __launch_bounds__(kThreads) ssd_bwd_state_scan_kernel(const SimtBwd p) {
    griddep_launch();
    griddep_wait();
    const int pn = kP * p.a.N, per = pn / (4 * kThreads);
    const int u = blockIdx.x / per, el = ((blockIdx.x % per) * kThreads + threadIdx.x) * 4;
    const int h = u % p.a.H, bi = u / p.a.H, dir = blockIdx.y;
    const float* init = dir ? p.a.dhf : p.a.h0;
    float4 run = init ? ld4(init + (size_t)u * pn + el) : make_float4(0.f, 0.f, 0.f, 0.f);
    float* st = dir ? p.gs : p.hs;
    auto slot = [&](int k) {  // the k-th chunk walked
        return ((size_t)bi * p.nc + (dir ? p.nc - 1 - k : k)) * p.a.H + h;
    };
    for (int k0 = 0; k0 < p.nc; k0 += kAhead) {
        float4 v[kAhead];
        float gam[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (k0 + j < p.nc) {
                v[j] = ld4(st + slot(k0 + j) * pn + el);
                gam[j] = p.e[slot(k0 + j) * kQ + kQ - 1];
            }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (k0 + j < p.nc) {
                st4(st + slot(k0 + j) * pn + el, run);
                run.x = fmaf(gam[j], run.x, v[j].x);
                run.y = fmaf(gam[j], run.y, v[j].y);
                run.z = fmaf(gam[j], run.z, v[j].z);
                run.w = fmaf(gam[j], run.w, v[j].w);
            }
    }
    if (dir && p.a.dh0) st4(p.a.dh0 + (size_t)u * pn + el, run);
}

// 2^v, within 2 ulp
__device__ __forceinline__ float exp2_approx(float v) {
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v));
    return v;
}
__device__ __noinline__ float raw_slope(float z, float lo, float hi) { return dt_slope(z, DtMap{nullptr, lo, hi, 1}); }

// ---- gradients of a chunk
template <int N> struct MainSmem {
    static constexpr int kB = 0, kC = kB + kQ * N, kH = kC + kQ * N, kG = kH + kP * N, kX = kG + kP * N,
                         kY = kX + kQ * kP, kS = kY + kQ * kP, kM = kS + kQ * kQ, kTerms = kM + kQ * kQ;
    // per-token: cs (two floats), row sums and column parts [8] (fp64), dt, e, w, Gm S and Gm on the
    // diagonal, E, F; then the warps' sums of <h, dh>
    static constexpr int kFloats = kTerms + kQ * (2 + 2 + 16 + 3 + 2 + 2) + 16;
};

template <typename TIO, int N>
// Two groups of 256 threads, a 4 x 4 tile of a 64 x 64 product each, work side by side on an item:
//   pairs   Gm, M, dS and W's sums, then U, V, dx and F
//   states  E from C h^T, then the states' parts of dC and dB, held in registers over the heads
// One group doing both in turn took 361 us against 321 us for 4096 tokens, 24 heads, N = 64, and at
// N = 128 the two were level.  The products are rolled loops of 80 instructions: unrolled four
// times, the code outgrew the instruction cache (80 KB against 51 KB: 321 against 283 us, and 1.61
// against 1.36 ms for 4 x 2048 tokens, 48 heads, N = 128).  8 x 8 tiles read half as much shared
// memory a multiply-add but leave a warp a scheduler, or bodies of 150 instructions and more: 1.49 ms.
__global__ void __launch_bounds__(2 * kThreads, 1) ssd_bwd_chunk_kernel(const SimtBwd p) {
    using SM = MainSmem<N>;
    extern __shared__ float sm[];
    float *sB = sm + SM::kB, *sC = sm + SM::kC, *sH = sm + SM::kH, *sG = sm + SM::kG, *sX = sm + SM::kX,
          *sY = sm + SM::kY, *sS = sm + SM::kS, *sM = sm + SM::kM;
    float2* s_cs = reinterpret_cast<float2*>(sm + SM::kTerms);  // log2(e) cs in two parts
    double* s_row = reinterpret_cast<double*>(s_cs + kQ);  // [kQ] sum_j W_ij (i > j)
    double* s_col = s_row + kQ;                            // [8 warps][kQ] parts of sum_i Gm S L (i > j)
    float *s_dt = reinterpret_cast<float*>(s_col + 8 * kQ), *s_e = s_dt + kQ, *s_w = s_e + kQ;
    float* s_dia = s_w + kQ;        // [kQ] Gm_jj S_jj, and [kQ] Gm_jj behind it
    float* s_E = s_dia + 2 * kQ;    // [kQ] E_i
    float* s_F = s_E + kQ;          // [kQ] F_j / dt_j
    float* s_z = s_F + kQ;          // [16] warp sums of <h, dh>
    const int tid = threadIdx.x, ty = (tid & 255) >> 4, tx = tid & 15, warp = tid >> 5, lane = tid & 31;
    const bool pairs = tid < kThreads;
    const int H = p.a.H, G = p.a.G, T = p.a.T, hg = H / G;
    const int split = blockIdx.x % p.splits, ug = blockIdx.x / p.splits, g = ug % G, bc = ug / G;
    const int bi = bc / p.nc, t0 = (bc % p.nc) * kQ, valid = min(kQ, T - t0);
    const size_t tok = (size_t)bi * T + t0;
    const int per = hg / p.splits, more = hg % p.splits;  // heads of a split; the first `more` have one more
    const int h_lo = split * per + min(split, more), h_hi = h_lo + per + (split < more);

    load_tile<N, 2 * kThreads>(sB, static_cast<const TIO*>(p.a.B) + (tok * G + g) * N, (size_t)G * N, valid);
    load_tile<N, 2 * kThreads>(sC, static_cast<const TIO*>(p.a.C) + (tok * G + g) * N, (size_t)G * N, valid);
    __syncthreads();
    if (pairs) {
        float s[4][4] = {};
        mm_nt<N>(sC, sB, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(sS + at<64>(4 * ty + i, tx)) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    }
    griddep_launch();
    griddep_wait();  // the states; B, C and S above need none of the launches ahead
    // over the heads: the pairs' group holds dS in the first four columns of dC's registers
    float dC[4][N / 16] = {}, dB[4][N / 16] = {};
    auto& dS = dC;

    for (int hh = h_lo; hh < h_hi; ++hh) {
        const int h = g * hg + hh;
        const size_t u = (size_t)bc * H + h;
        __syncthreads();  // the head before has been read
        load_tile<kP, 2 * kThreads>(sX, static_cast<const TIO*>(p.a.x) + (tok * H + h) * kP, (size_t)H * kP, valid);
        load_tile<kP, 2 * kThreads>(sY, static_cast<const TIO*>(p.a.dy) + (tok * H + h) * kP, (size_t)H * kP, valid);
        float z = 0.f;
#pragma unroll 2
        for (int i = tid; i < kP * (N / 4); i += 2 * kThreads) {
            const int r = i / (N / 4), c = i % (N / 4);
            const float4 a = ld4(p.hs + u * kP * N + 4 * i), d = ld4(p.gs + u * kP * N + 4 * i);
            *reinterpret_cast<float4*>(sH + at<N>(r, c)) = a;
            *reinterpret_cast<float4*>(sG + at<N>(r, c)) = d;
            z = fmaf(a.x, d.x, fmaf(a.y, d.y, fmaf(a.z, d.z, fmaf(a.w, d.w, z))));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane == 0) s_z[warp] = z;
        if (tid < kQ) {
            const double c = p.cs[u * kQ + tid] * 1.4426950408889634;
            s_cs[tid] = make_float2((float)c, (float)(c - (double)(float)c));
            s_dt[tid] = p.dtv[u * kQ + tid];
            s_e[tid] = p.e[u * kQ + tid];
            s_w[tid] = p.w[u * kQ + tid];
        }
        __syncthreads();
        if (pairs) {
            // ---- Gm, M = S L, dS, W's sums (rows i = 4 ty + a, columns j = 4 tx + b)
            {
                float gm[4][4] = {}, dtj[4];
                double row[4] = {}, colp[4] = {};
                float2 cj[4];
                mm_nt<kP>(sY, sX, ty, tx, gm);
#pragma unroll
                for (int c = 0; c < 4; ++c) cj[c] = s_cs[4 * tx + c], dtj[c] = s_dt[4 * tx + c];
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const int i = 4 * ty + a;
                    const float4 s4 = ld4(sS + at<64>(i, tx));
                    const float sv[4] = {s4.x, s4.y, s4.z, s4.w};
                    const float2 ci = s_cs[i];
                    float m[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const bool low = ty > tx || (ty == tx && a >= c);  // i >= j
                        const float l = low ? exp2_approx((ci.x - cj[c].x) + (ci.y - cj[c].y)) : 0.f;
                        m[c] = sv[c] * l;
                        const float wv = a == c && ty == tx ? 0.f : gm[a][c] * m[c];  // i > j
                        dS[a][c] = fmaf(gm[a][c] * l, dtj[c], dS[a][c]);
                        row[a] = fma((double)wv, (double)dtj[c], row[a]);
                        colp[c] += (double)wv;
                    }
                    if (ty == tx) s_dia[i] = gm[a][a] * m[a], s_dia[kQ + i] = gm[a][a];
                    *reinterpret_cast<float4*>(sM + at<64>(i, tx)) = make_float4(m[0], m[1], m[2], m[3]);
                }
#pragma unroll
                for (int a = 0; a < 4; ++a) {
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) row[a] += __shfl_xor_sync(0xffffffffu, row[a], o);
                    if (tx == 0) s_row[4 * ty + a] = row[a];
                    colp[a] += __shfl_xor_sync(0xffffffffu, colp[a], 16);
                    if (lane < 16) s_col[warp * kQ + 4 * tx + a] = colp[a];
                }
            }
            asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
            // ---- dx and F (rows j = 4 ty + a, columns p = 4 tx + b)
            {
                float v[4][4] = {}, uu[4][4] = {};
                mm_nt<N>(sB, sG, ty, tx, v);
                mm_tn<kP>(sM, sY, ty, tx, uu);
                const float Dh = p.a.D[h];
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const int j = 4 * ty + a;
                    const float4 x4 = ld4(sX + at<64>(j, tx)), y4 = ld4(sY + at<64>(j, tx));
                    const float wj = s_w[j], dtj = s_dt[j];
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[a][c] *= wj;
                    float f = x4.x * v[a][0] + x4.y * v[a][1] + x4.z * v[a][2] + x4.w * v[a][3];
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
                    if (tx == 0) s_F[j] = f;
                    const float4 o4 = make_float4(fmaf(dtj, uu[a][0] + v[a][0], Dh * y4.x),
                                                  fmaf(dtj, uu[a][1] + v[a][1], Dh * y4.y),
                                                  fmaf(dtj, uu[a][2] + v[a][2], Dh * y4.z),
                                                  fmaf(dtj, uu[a][3] + v[a][3], Dh * y4.w));
                    if (j < valid) st4(static_cast<TIO*>(p.a.dx) + ((tok + j) * H + h) * kP + 4 * tx, o4);
                }
            }
        } else {
            // ---- E
            {
                float v[4][4] = {};
                mm_nt<N>(sC, sH, ty, tx, v);
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const int i = 4 * ty + a;
                    const float4 y4 = ld4(sY + at<64>(i, tx));
                    float f = y4.x * v[a][0] + y4.y * v[a][1] + y4.z * v[a][2] + y4.w * v[a][3];
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
                    if (tx == 0) s_E[i] = f * s_e[i];
                }
            }
            // ---- the states' parts of dC and dB
            {
                float sc[4], sb[4];
#pragma unroll
                for (int a = 0; a < 4; ++a) sc[a] = s_e[4 * ty + a], sb[a] = s_w[4 * ty + a] * s_dt[4 * ty + a];
                mm_nn<N>(sY, sH, ty, tx, sc, dC);
                mm_nn<N>(sX, sG, ty, tx, sb, dB);
            }
        }
        __syncthreads();
        // ---- ddt, two tokens a lane of warp 0
        if (warp == 0) {
            float zz = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) zz += s_z[k];
            zz *= s_e[kQ - 1];
            double rc[2];
            float col[2], f[2], dtv[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int t = 2 * lane + k;
                double cw = 0.0;
#pragma unroll
                for (int q = 0; q < 8; ++q) cw += s_col[q * kQ + t];
                col[k] = (float)cw;
                dtv[k] = s_dt[t];
                f[k] = s_F[t] * dtv[k];
                rc[k] = (double)s_E[t] + (s_row[t] - cw * (double)dtv[k]);
            }
            double suf = rc[0] + rc[1];  // suffix sum of rc, prefix sum of f over lanes
            float pre = f[0] + f[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double a = __shfl_down_sync(0xffffffffu, suf, o);
                const float c = __shfl_up_sync(0xffffffffu, pre, o);
                if (lane + o < 32) suf += a;
                if (lane >= o) pre += c;
            }
            // the F ahead of the lane's tokens, by a shift: less their own F, the rounding of those would stay
            pre = __shfl_up_sync(0xffffffffu, pre, 1);
            if (lane == 0) pre = 0.f;
            float sA = 0.f, sD = 0.f, sb = 0.f;
            const float Ah = p.a.A[h];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int t = 2 * lane + k;
                const float da = zz + (float)(k ? suf - rc[0] : suf) + (k ? pre + f[0] : pre);
                float ddt = fmaf(Ah, da, s_dia[t] + col[k] + s_F[t]);
                if (t < valid) {
                    const size_t o = (tok + t) * H + h;
                    if (p.a.dtm.raw) ddt *= raw_slope(p.a.dt[o] + (p.a.dtm.bias ? p.a.dtm.bias[h] : 0.f), p.a.dtm.lo, p.a.dtm.hi);
                    p.a.ddt[o] = ddt;
                    sA = fmaf(dtv[k], da, sA);
                    sD += s_dia[kQ + t];
                    sb += ddt;
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                sA += __shfl_xor_sync(0xffffffffu, sA, o);
                sD += __shfl_xor_sync(0xffffffffu, sD, o);
                sb += __shfl_xor_sync(0xffffffffu, sb, o);
            }
            if (lane == 0) {
                p.pA[u] = sA;
                p.pD[u] = sD;
                if (p.pb) p.pb[u] = sb;
            }
        }
    }
    // ---- the pairs' parts of dC and dB, from the sum of dS over the heads
    __syncthreads();
    if (pairs) {
#pragma unroll
        for (int a = 0; a < 4; ++a)
            *reinterpret_cast<float4*>(sM + at<64>(4 * ty + a, tx)) = make_float4(dS[a][0], dS[a][1], dS[a][2], dS[a][3]);
    }
    __syncthreads();
    if (pairs) return;
    const float one[4] = {1.f, 1.f, 1.f, 1.f};
    mm_nn<N>(sM, sB, ty, tx, one, dC);
    mm_tn<N>(sM, sC, ty, tx, dB);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const int r = 4 * ty + a;
        if (r >= valid) continue;
#pragma unroll
        for (int n = 0; n < N / 64; ++n) {
            const float4 vb = make_float4(dB[a][4 * n], dB[a][4 * n + 1], dB[a][4 * n + 2], dB[a][4 * n + 3]);
            const float4 vc = make_float4(dC[a][4 * n], dC[a][4 * n + 1], dC[a][4 * n + 2], dC[a][4 * n + 3]);
            const size_t o = ((tok + r) * G + g) * N + 64 * n + 4 * tx;
            if (p.splits == 1) {
                st4(static_cast<TIO*>(p.a.dB) + o, vb);
                st4(static_cast<TIO*>(p.a.dC) + o, vc);
            } else {
                const size_t all = (size_t)p.a.b * T * G * N;
                st4(p.part + split * all + o, vb);
                st4(p.part + (p.splits + split) * all + o, vc);
            }
        }
    }
}

// dB and dC from the blocks' sums, in block order (none where a group's heads are not split), and
// the sums over the chunks
template <typename TIO>
__global__ void __launch_bounds__(kThreads) ssd_bwd_sums_kernel(const SimtBwd p, const HeadSums hs, int group_blocks) {
    griddep_wait();
    if ((int)blockIdx.x >= group_blocks) return head_sum<kThreads>(hs, blockIdx.x - group_blocks);
    const size_t all = (size_t)p.a.b * p.a.T * p.a.G * p.a.N, i = ((size_t)blockIdx.x * kThreads + threadIdx.x) * 4;
    if (i >= 2 * all) return;
    const int which = i >= all;
    const size_t at = i - which * all;
    const float* src = p.part + (size_t)which * p.splits * all + at;
    float4 s = ld4(src);
#pragma unroll 4
    for (int k = 1; k < p.splits; ++k) {
        const float4 v = ld4(src + k * all);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    st4(static_cast<TIO*>(which ? p.a.dC : p.a.dB) + at, s);
}

// Carves the workspace; returns its size.  ws = nullptr: the size only.
size_t simt_layout(const BwdArgs& a, char* ws, SimtBwd* p) {
    p->a = a;
    p->nc = (a.T + kQ - 1) / kQ;
    const size_t bc = (size_t)a.b * p->nc, u = bc * a.H;
    const int hg = a.H / a.G;
    // A block holds an SM.  More blocks a group fill the last wave better, but each begins with the
    // group's S and ends with its dB and dC, about 0.8 of a head's time, and adds a part to the sums
    // (64 groups of 24 heads on 148 SMs: 239 us with 2 blocks a group, 251 with 4, 297 with 5).
    const int sms = device_sms();
    const size_t groups = bc * a.G;
    double best = 0.0;
    p->splits = 1;
    for (int n = 1; n <= hg && (n == 1 || groups * (n - 1) < 8 * (size_t)sms); ++n) {
        const double waves = (double)((groups * n + sms - 1) / sms);
        const double cost = waves * ((hg + n - 1) / n + 0.8) + (n > 1 ? 0.3 + 0.02 * n : 0.0);
        if (n == 1 || cost < best) best = cost, p->splits = n;
    }
    size_t o = 0;
    auto take = [&](size_t bytes) {
        char* r = ws ? ws + o : nullptr;
        o += round_up(bytes, 256);
        return r;
    };
    p->dtv = reinterpret_cast<float*>(take(u * kQ * 4));
    p->cs = reinterpret_cast<double*>(take(u * kQ * 8));
    p->e = reinterpret_cast<float*>(take(u * kQ * 4));
    p->w = reinterpret_cast<float*>(take(u * kQ * 4));
    p->hs = reinterpret_cast<float*>(take(u * kP * a.N * 4));
    p->gs = reinterpret_cast<float*>(take(u * kP * a.N * 4));
    p->pA = reinterpret_cast<float*>(take(u * 4));
    p->pD = reinterpret_cast<float*>(take(u * 4));
    p->pb = reinterpret_cast<float*>(take(u * 4));
    p->part = p->splits > 1 ? reinterpret_cast<float*>(take(2 * p->splits * (size_t)a.b * a.T * a.G * a.N * 4)) : nullptr;
    return o;
}

template <typename TIO, int N>
int run_simt(const SimtBwd& p, cudaStream_t s) {
    const size_t u = (size_t)p.a.b * p.nc * p.a.H;
    {
        const int smem = (kQ * kP + kQ * N + kQ) * 4;
        if (const int st = smem_limit_once((const void*)ssd_bwd_chunk_states_kernel<TIO, N>, smem)) return st;
        LaunchScope ls("ssd_bwd_chunk_states", s);
        ssd_bwd_chunk_states_kernel<TIO, N><<<dim3((unsigned)u, 2), kThreads, smem, s>>>(p);
        SSD_CUDA_TRY(cudaGetLastError());
    }
    {
        LaunchScope ls("ssd_bwd_state_scan", s);
        SSD_CUDA_TRY(launch_pdl(ssd_bwd_state_scan_kernel, dim3(p.a.b * p.a.H * (kP * N / (4 * kThreads)), 2), kThreads, 0, s, p));
    }
    {
        const int smem = MainSmem<N>::kFloats * 4;
        if (const int st = smem_limit_once((const void*)ssd_bwd_chunk_kernel<TIO, N>, smem)) return st;
        LaunchScope ls("ssd_bwd_chunk", s);
        SSD_CUDA_TRY(launch_pdl(ssd_bwd_chunk_kernel<TIO, N>, dim3((unsigned)((size_t)p.a.b * p.nc * p.a.G * p.splits)),
                                2 * kThreads, smem, s, p));
    }
    {
        const size_t all = (size_t)p.a.b * p.a.T * p.a.G * N;
        const int group_blocks = p.splits > 1 ? (int)((all / 2 + kThreads - 1) / kThreads) : 0;
        const HeadSums hs{p.pA, p.pD, p.pb, p.a.b * p.nc, p.a.H, p.a.dA, p.a.dD, p.a.dbias};
        LaunchScope ls("ssd_bwd_sums", s);
        SSD_CUDA_TRY(launch_pdl(ssd_bwd_sums_kernel<TIO>, dim3((unsigned)(group_blocks + hs.blocks())), kThreads, 0, s, p, hs,
                                group_blocks));
    }
    return SSD_OK;
}

}  // namespace

size_t backward_simt_workspace_bytes(const BwdArgs& a) {
    SimtBwd p;
    return simt_layout(a, nullptr, &p);
}

// Whether the launches' grids hold the call: (chunk, head) pairs and state entries in one
// dimension of a grid.
bool backward_simt_fits(const BwdArgs& a) {
    const unsigned long long u = (unsigned long long)a.b * ((a.T + kQ - 1) / kQ) * a.H;
    return u < (1ull << 31) && (unsigned long long)a.b * a.H * 8 < (1ull << 31) &&
           (unsigned long long)a.b * a.T * a.G * a.N / 2 / kThreads + 3ull * a.H < (1ull << 31) - 1;
}

int launch_backward_simt(const BwdArgs& a, void* ws, cudaStream_t s) {
    SimtBwd p;
    simt_layout(a, static_cast<char*>(ws), &p);
    if (!a.dbias) p.pb = nullptr;
    if (a.io == SSD_BF16)
        return a.N == 128 ? run_simt<__nv_bfloat16, 128>(p, s) : run_simt<__nv_bfloat16, 64>(p, s);
    return a.N == 128 ? run_simt<float, 128>(p, s) : run_simt<float, 64>(p, s);
}

}  // namespace ssd
