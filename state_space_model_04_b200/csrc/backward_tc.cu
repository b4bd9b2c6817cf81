// backward_tc.cu -- gradients of the SSD prefill on the sm_100a tensor cores (tcgen05 + TMEM +
// TMA), for bf16 inputs with P = 64, N = 128.  The formulas are those at the head of
// backward_simt.cu, with chunks of 128 tokens (the M of one tcgen05 MMA).
//
// Two passes over the tokens, because the state runs forwards and its adjoint backwards:
//
//   state pass   a CTA walks one (sequence, head) chunk by chunk, forwards with x, B for the state
//                h entering each chunk, backwards with dy, C for the adjoint dh of the state
//                leaving it, the running state in fp32 registers; each is written as two bf16
//                halves (hi = bf16(h), lo = bf16(h - hi), 16 bits of h together) in the layout
//                the next pass's MMAs read.
//   main pass    a CTA takes a run of (chunk, head) items, heads fastest, so that the heads of a
//                B/C group follow one another in one CTA and what they share stays on chip:
//                S^T = B C^T is computed once and held in registers, dB and dC accumulate in
//                TMEM over the heads, and the pair terms dS are summed over the heads in
//                registers and multiplied with B and C once a group.  A group's heads may lie in
//                several CTAs; each then stores its sums in fp32 and a third pass (join) adds them
//                in CTA order.
//
// Per item the main pass multiplies (rows j or i, 128 each)
//   G^T = X dY^T,   V = B dh^T (hi, lo),   Y = C h^T (hi, lo),
//   dC += (e o dY) h,   dB += (w dt o X) dh,   U = w o V + M^T dY,  M^T = S^T o L^T
// with G^T, V and Y in fp32 TMEM.  Precision: ddt, dA and dh0 are fp32 gradients, and what they
// are made of (G, S, V, Y, the states) carries 16 bits or more, the decays fp32's: V and Y take both
// halves of the states, the state pass both halves of the weighted x and dy.  dx, dB and dC are
// stored in bf16, so M, dS, the weighted rows and the states are rounded to bf16 once where they
// feed only those.
//
// Bound: memory, with the latency between a pass's roles close behind.  Per item the main pass
// moves 48 KB of x, dy, dx and 64 KB of state halves, the state pass 32 KB and 64 KB.  8 x 4096
// tokens, 80 heads, events around each launch: terms 27 us, state pass 443 us (4.5 TB/s, 69 % of a
// copy's rate), main pass 612 us (3.8 TB/s, 57 %; tensor pipe 26 %, issue slots 44 %), join 19 us; the call
// 1.09 ms.  Under a sustained load of these calls the 1000 W power limit takes the clock from 1.97 to
// 1.6 GHz, and they take 1.17 to 1.26 ms by the board.
#include <algorithm>
#include <atomic>
#include <cstring>
#include "backward.cuh"
#include "tc.cuh"

namespace ssd {
namespace {

constexpr int kP = 64, kN = 128;
constexpr uint32_t kRegion = kBlk * 128;        // one [128 rows][64 bf16] swizzled box: 16 KB
constexpr uint32_t kImage = 2 * kRegion;        // a state: hi, lo, each [128 n][64 p]
// per-token terms of an item, [kTerms][128] fp32 (a: step sizes times A; cs: its prefix sum in the
// chunk, csub: in the token's 32-token group).  csub log2(e) takes the first two places, in two parts,
// token pairs as {hi, hi, lo, lo}: a step that erases the state leaves a prefix sum in the thousands, of
// which fp32 alone keeps too little for the decay between two tokens behind it
constexpr int kTermCs2 = 0;
constexpr int kTermE = 2;                       // exp(cs)
constexpr int kTermW = 3;                       // exp(cs_last - cs)
constexpr int kTermDt = 4;                      // dt
constexpr int kTerms = 5;
// where the parts of a token's csub log2(e) are
__device__ __forceinline__ int cs2_at(int token) { return kTermCs2 * kBlk + 4 * (token >> 1) + (token & 1); }
constexpr int kCs2Lo = 2;
constexpr uint32_t kTermBytes = kTerms * kBlk * 4;

struct BwdTc {
    CUtensorMap tm_x, tm_dy, tm_B, tm_C, tm_dx;
    BwdArgs a;
    int nc;                 // chunks a sequence
    int ctas;               // of the main pass
    int per_group;          // CTAs a (chunk, group) where each CTA stays in one, or 0: an even split,
    int each, more;         // `each` items a CTA, one more in the first `more`
    int n_whole;            // (sequence, head) pairs the state pass walks whole; the others in
    int nseg, cseg;         // nseg segments of cseg chunks
    float* seg_end;         // [split pairs][2 directions][nseg - 1][P][N] end states of segments run from zero
                            // (the first from the initial state)
    float* seg_decay;       // [split pairs][2][nseg - 1] their whole decay
    long long items;        // b nc H
    float* terms;           // [items][kTerms][128]
    float* slope;           // [items][128] of dt over its raw step, or nullptr (dt is given)
    uint8_t* img_h;         // [items][kImage] state entering the chunk
    uint8_t* img_g;         // [items][kImage] adjoint of the state leaving it
    float* part;            // [ctas][2][2][128][128] sums of dB, dC of a CTA's first and last group
    float *pA, *pD, *pb;    // [b nc][H]
    int* status;
    unsigned long long wait_ns;
    int starve;
    int lag;                // role of the main pass that sleeps before it reads an item, or -1
};

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Waits.  Their slow side is one function each for a whole warp and for one thread, and all it needs
// beside the barrier lies in shared memory: a wait costs its place in the code a few instructions.
// On expiry the site goes to the status word and every other wait of the CTA gives up.
__shared__ int s_stop;
__shared__ int* s_status;
__device__ __forceinline__ bool stopped() { return *reinterpret_cast<volatile int*>(&s_stop) != 0; }
__device__ __forceinline__ bool wait_expired(unsigned long long t0, uint32_t site) {
    if (stopped()) return true;
    if (globaltimer() - t0 <= s_wait_ns) return false;
    *reinterpret_cast<volatile int*>(&s_stop) = 1;
    atomicCAS(s_status, 0, (int)(SSD_ERR_TIMEOUT | (site << 8)));
    return true;
}
__device__ __noinline__ bool wait_slow_warp(uint32_t bar, uint32_t parity_site) {
    const unsigned long long t0 = globaltimer();
    while (!__all_sync(0xffffffffu, mbar_try_sleep(bar, parity_site & 1)))
        if (__any_sync(0xffffffffu, wait_expired(t0, parity_site >> 1))) return false;
    return true;
}
__device__ __noinline__ bool wait_slow_one(uint32_t bar, uint32_t parity_site) {
    const unsigned long long t0 = globaltimer();
    while (!mbar_try_sleep(bar, parity_site & 1))
        if (wait_expired(t0, parity_site >> 1)) return false;
    return true;
}
// Phase `n` of a barrier (its parity counts).  wait_warp: all lanes together, with one result.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t n, uint32_t site) {
    return __all_sync(0xffffffffu, mbar_try(bar, n & 1)) || wait_slow_warp(bar, (n & 1) | (site << 1));
}
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t n, uint32_t site) {
    return mbar_try(bar, n & 1) || wait_slow_one(bar, (n & 1) | (site << 1));
}

// ------------------------------------------------------------------ per-token terms
// One warp per item, lane l holds tokens 32 q + l; prefix sums in fp64.
constexpr int kTermThreads = 256;
__global__ void __launch_bounds__(kTermThreads) ssd_bwd_tc_terms_kernel(const __grid_constant__ BwdTc p) {
    const int lane = threadIdx.x & 31, h = blockIdx.y * (kTermThreads / 32) + (threadIdx.x >> 5);
    griddep_launch();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = 0;
    if (h >= p.a.H) return;
    const int bc = blockIdx.x, bi = bc / p.nc, t0 = (bc % p.nc) * kBlk;
    const double Ah = p.a.A[h];
    float dt[4], slope[4];
    double cs[4], end[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int t = t0 + 32 * q + lane;
        const float raw = t < p.a.T ? p.a.dt[((size_t)bi * p.a.T + t) * p.a.H + h] : 0.f;
        dt[q] = t < p.a.T ? dt_value(raw, p.a.dtm, h) : 0.f;
        slope[q] = p.a.dtm.raw ? dt_slope(raw + (p.a.dtm.bias ? p.a.dtm.bias[h] : 0.f), p.a.dtm) : 1.f;
        cs[q] = dt[q] * Ah;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const double v = __shfl_up_sync(0xffffffffu, cs[q], o);
            if (lane >= o) cs[q] += v;
        }
    }
    double run = 0.0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        end[q] = run;  // the prefix ahead of group q
        run += __shfl_sync(0xffffffffu, cs[q], 31);
    }
    float* t = p.terms + ((size_t)bc * p.a.H + h) * kTerms * kBlk + lane;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const double c = end[q] + cs[q];
        const double c2 = cs[q] * 1.4426950408889634;
        float* two = t - lane + cs2_at(32 * q + lane);
        two[0] = (float)c2;
        two[kCs2Lo] = (float)(c2 - (double)(float)c2);
        t[kTermE * kBlk + 32 * q] = expf((float)c);
        t[kTermW * kBlk + 32 * q] = expf((float)(run - c));
        t[kTermDt * kBlk + 32 * q] = dt[q];
        if (p.slope) p.slope[((size_t)bc * p.a.H + h) * kBlk + 32 * q + lane] = slope[q];
    }
}

// ------------------------------------------------------------------ state pass
//   warp 0      TMA producer: X (or dY) and the two boxes of B (or C) of a chunk, 3-slot ring
//   warp 1      TMEM owner and MMA issuer: D[n][hi p | lo p] = B^T [wX_hi | wX_lo], one product of
//               N = 128 (the halves in products of their own would read B from shared memory twice)
//   warp 2      stores the images, one bulk copy each
//   warps 4-11  half a token row a thread: weighted into hi and lo tiles, a chunk ahead
//   warps 12-19 half a state row n a thread, 32 fp32 entries in registers: writes the entering state's
//               halves to an image, then h <- exp(cs_last) h + D_hi + D_lo
// A sequence may be cut into segments of whole chunks to fill the SMs: the ends kernel runs all but
// the last segment from zero for their end states, and the state kernel's segments start from the
// fold of the ends before them.
constexpr int kSThreads = 640;
constexpr uint32_t kSSlot = 3 * kRegion;            // X, B (n 0..63), B (n 64..127)
constexpr int kSSlots = 3;
constexpr uint32_t kSXs = kSSlots * kSSlot;         // hi, lo tiles of the weighted rows
constexpr uint32_t kSImg = kSXs + kImage;           // state image
constexpr uint32_t kSSmall = kSImg + kImage;
constexpr uint32_t kSSmem = kSSmall + 256;
static_assert(kSSmem <= 232448 - 1024, "state pass shared memory");
constexpr uint32_t kSCols = 256;                    // two accumulators of 128 columns
enum {
    SB_FULL = 0, SB_EMPTY = 3, SB_XS = 6, SB_IMG = 7, SB_IMGFREE = 8, SB_DONE = 9, SB_ACC = 10, SB_ACCFREE = 12, SB_COUNT = 14
};

template <bool kEnds>
__global__ void __launch_bounds__(kSThreads, 1) ssd_bwd_tc_state_kernel(const __grid_constant__ BwdTc p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int H = p.a.H, nc = p.nc;
    // the pairs walked whole first, being the longest, then the segments of the others
    const int segs = kEnds ? p.nseg - 1 : p.nseg, dir = blockIdx.x & 1, x = (blockIdx.x >> 1) - (kEnds ? 0 : p.n_whole);
    const bool whole = x < 0;
    const int u = p.n_whole + (whole ? x : x / segs), seg = whole ? 0 : x % segs;
    const int h = u % H, bi = u / H, g = h / (H / p.a.G);
    // this CTA's chunks in walking order: [c0, c0 + n)
    const int c0 = seg * p.cseg, n = whole ? nc : min(p.cseg, nc - c0);
    auto chunk = [&](int k) { return dir ? nc - 1 - c0 - k : c0 + k; };
    uint8_t* small = smem + kSSmall;
    uint64_t* bars = reinterpret_cast<uint64_t*>(small);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(small + 144);
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    auto wt = [&](int b, uint32_t n, uint32_t site) { return wait_warp(bar(b), n, site); };
    auto w1 = [&](int b, uint32_t n, uint32_t site) { return wait_one(bar(b), n, site); };

    if (threadIdx.x == 0) {
        const bool misaligned = (sbase & 1023u) != 0;
        if (misaligned) report_status(p.status, SSD_ERR_INTERNAL | (5 << 8));
        for (int i = 0; i < SB_COUNT; ++i)
            mbar_init(bar(i), i == SB_XS || i == SB_IMG || (i & ~1) == SB_ACCFREE ? 8 : 1);
        s_stop = misaligned ? 1 : 0;
        s_status = p.status;
        s_wait_ns = p.wait_ns;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_alloc_cta(s_tmem, kSCols, warp == 1), 0);
    if (tmem == kTmemSentinel) {
        s_stop = 1;
        report_status(p.status, SSD_ERR_INTERNAL | (6 << 8));
    }
    griddep_launch();
    griddep_wait();  // what the launches ahead wrote
    // the product of the sequence's last chunk walked only feeds the adjoint of the initial state
    const bool final = !kEnds && c0 + n == nc;
    const int products = final && !(dir && p.a.dh0) ? n - 1 : n;

    if (warp == 0) {
        if (lane == 0 && !stopped() && !p.starve) {
            int issued = 0;
#pragma unroll 1
            for (int k = 0; k < products; ++k) {
                const int s = k % kSSlots;
                if (k >= kSSlots && !w1(SB_EMPTY + s, k / kSSlots - 1, 50)) break;
                const uint32_t f = bar(SB_FULL + s), slot = sbase + s * kSSlot;
                const int t0 = chunk(k) * kBlk;
                mbar_expect_tx(f, kSSlot);
                tma_load_4d(slot, dir ? &p.tm_dy : &p.tm_x, f, 0, h, t0, bi);
                tma_load_4d(slot + kRegion, dir ? &p.tm_C : &p.tm_B, f, 0, g, t0, bi);
                tma_load_4d(slot + 2 * kRegion, dir ? &p.tm_C : &p.tm_B, f, 64, g, t0, bi);
                issued = k + 1;
            }
            for (int k = issued - kSSlots; k < issued; ++k)
                if (k >= 0) mbar_drain(bar(SB_FULL + k % kSSlots), (k / kSSlots) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t id = idesc_bf16(128, 128, 1, 1);
            const uint64_t mB = sdesc(sbase + kRegion, kRegion, 1024), mX = sdesc(sbase + kSXs, kRegion, 1024);
            bool ok = !stopped();
#pragma unroll 1
            for (int k = 0; k < products && ok; ++k) {
                const int s = k & 1, slot = k % kSSlots;
                ok = w1(SB_FULL + slot, k / kSSlots, 51) && w1(SB_XS, k, 52) &&
                     (k < 2 || w1(SB_ACCFREE + s, (k - 2) >> 1, 53));
                if (!ok) break;
                tc_fence_after();
                const uint64_t a = mB + slot * (kSSlot >> 4), b = mX;
#pragma unroll
                for (int kk = 0; kk < kBlk / 16; ++kk) mma_ss(tmem + s * 128, a + kk * 128, b + kk * 128, id, kk > 0);
                mma_commit(bar(SB_EMPTY + slot));
                mma_commit(bar(SB_ACC + s));
            }
            mma_commit(bar(SB_DONE));
            mbar_drain(bar(SB_DONE), 0);
        }
        __syncwarp();
    } else if (warp == 2) {
        if (!kEnds && lane == 0 && !stopped()) {
            uint8_t* images = (dir ? p.img_g : p.img_h) + ((size_t)bi * nc * H + h) * kImage;
#pragma unroll 1
            for (int k = 0; k < n; ++k) {
                if (!w1(SB_IMG, k, 57)) break;
                bulk_store(images + (size_t)chunk(k) * H * kImage, sbase + kSImg, kImage);
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(bar(SB_IMGFREE));
            }
            bulk_wait0();  // the stores are complete before the shared memory goes away
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 12) {
        const int r = (warp & 3) * 32 + lane, half = (warp - 4) >> 2;  // token, 32 of its columns
        const float* tm = p.terms + ((size_t)bi * nc * H + h) * kTerms * kBlk + r;
        auto weight = [&](int k) {
            if (k >= products) return 0.f;
            const float* t = tm + (size_t)chunk(k) * H * kTerms * kBlk;
            return dir ? t[kTermE * kBlk] : t[kTermW * kBlk] * t[kTermDt * kBlk];
        };
        float next = weight(0);
        bool live = __all_sync(0xffffffffu, !stopped());
#pragma unroll 1
        for (int k = 0; k < products && live; ++k) {
            const int s = k % kSSlots;
            const f32x2 w2 = pack2(next, next), minus = pack2(-1.f, -1.f);
            next = weight(k + 1);
            // the product of the chunk before has read the tiles
            live = (k < 1 || wt(SB_EMPTY + (k - 1) % kSSlots, (k - 1) / kSSlots, 54)) && wt(SB_FULL + s, k / kSSlots, 55);
            if (!live) break;
            const uint8_t* src = smem + s * kSSlot;
            uint8_t* dst = smem + kSXs;
#pragma unroll 2
            for (int c = 4 * half; c < 4 * half + 4; ++c) {
                const uint32_t o = swz(r, c);
                const uint4 v = *reinterpret_cast<const uint4*>(src + o);
                const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x2 t = mul2(pack2(bf_lo(in[j]), bf_hi(in[j])), w2);
                    float a, b;
                    unpack2(t, a, b);
                    hi[j] = pack_bf16(a, b);
                    unpack2(fma2(pack2(bf_lo(hi[j]), bf_hi(hi[j])), minus, t), a, b);
                    lo[j] = pack_bf16(a, b);
                }
                *reinterpret_cast<uint4*>(dst + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(dst + kRegion + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(SB_XS));
        }
    } else if (warp >= 12) {
        const int q = warp & 3, r = q * 32 + lane, half = (warp - 12) >> 2, p0 = 32 * half;  // state row n, columns p0 ..
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + p0;
        const size_t un = (size_t)(u - p.n_whole) * 2 + dir;  // of the split pairs
        const size_t at = (size_t)p0 * kN + r;  // [p][n]
        const float* init = dir ? p.a.dhf : p.a.h0;
        f32x2 st[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) st[i] = 0ull;
        if (init && seg == 0) {
            const float* v = init + (size_t)u * kP * kN + at;
#pragma unroll
            for (int i = 0; i < 16; ++i) st[i] = pack2(v[(2 * i) * kN], v[(2 * i + 1) * kN]);
        }
        const float* gp = p.terms + (((size_t)bi * nc * H + h) * kTerms + kTermE) * kBlk + kBlk - 1;
        auto decay = [&](int k) { return k < n ? gp[(size_t)chunk(k) * H * kTerms * kBlk] : 0.f; };
        if constexpr (!kEnds) {
            // the ends of the segments before, in order; the first already starts from the initial state
#pragma unroll 1
            for (int s = 0; s < seg; ++s) {
                const float* e = p.seg_end + (un * (p.nseg - 1) + s) * kP * kN + at;
                const float d = s ? p.seg_decay[un * (p.nseg - 1) + s] : 0.f;
                const f32x2 d2 = pack2(d, d);
#pragma unroll
                for (int i = 0; i < 16; ++i) st[i] = fma2(d2, s ? st[i] : 0ull, pack2(e[(2 * i) * kN], e[(2 * i + 1) * kN]));
            }
        }
        float next = decay(0), total = 1.f;
        bool live = __all_sync(0xffffffffu, !stopped());
#pragma unroll 1
        for (int k = 0; k < n && live; ++k) {
            const int s = k & 1;
            const float gam = next;
            next = decay(k + 1);
            total *= gam;
            if constexpr (!kEnds) {
                // the state as two bf16 halves
                live = k < 1 || wt(SB_IMGFREE, k - 1, 58);
                if (!live) break;
                uint8_t* img = smem + kSImg;
                const f32x2 minus = pack2(-1.f, -1.f);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float a, b;
                        unpack2(st[4 * c + j], a, b);
                        hi[j] = pack_bf16(a, b);
                        unpack2(fma2(pack2(bf_lo(hi[j]), bf_hi(hi[j])), minus, st[4 * c + j]), a, b);
                        lo[j] = pack_bf16(a, b);
                    }
                    const uint32_t o = swz(r, 4 * half + c);
                    *reinterpret_cast<uint4*>(img + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(img + kRegion + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(SB_IMG));
            }
            if (k < products) {
                live = wt(SB_ACC + s, k >> 1, 56);
                if (!live) break;
                tc_fence_after();
                const f32x2 g2 = pack2(gam, gam);
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    uint32_t hi[16], lo[16];
                    SSD_TMEM_LD16x2_WAIT(acc + s * 128 + 16 * o, 64, hi, lo);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        st[8 * o + j] = fma2(g2, st[8 * o + j],
                                             add2(pack2(__uint_as_float(hi[2 * j]), __uint_as_float(hi[2 * j + 1])),
                                                  pack2(__uint_as_float(lo[2 * j]), __uint_as_float(lo[2 * j + 1]))));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(SB_ACCFREE + s));
            }
        }
        float* out = kEnds ? p.seg_end + (un * (p.nseg - 1) + seg) * kP * kN : final && dir ? p.a.dh0 : nullptr;
        if (live && !stopped() && out) {
            if (!kEnds) out += (size_t)u * kP * kN;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float a, b;
                unpack2(st[i], a, b);
                out[at + (2 * i) * kN] = a;
                out[at + (2 * i + 1) * kN] = b;
            }
            if (kEnds && r == 0 && half == 0) p.seg_decay[un * (p.nseg - 1) + seg] = total;
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (warp == 1 && tmem != kTmemSentinel) {
        tc_fence_after();
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kSCols));
    }
}

// ------------------------------------------------------------------ main pass
// 20 warps; a warp's TMEM lane quadrant is q = warp % 4, and the work of the quadrants differs
// (tokens j of quadrant q meet tokens i of the 32-token groups c >= q only):
//
//   pair warps (q, c), q <= c: 10    S^T and the sum of dS^T of their 32 x 32 block in registers;
//                                    per item M^T and W from G^T; per group of heads dB, dC
//   row warps q: 4                   one token a thread: the weighted rows, F and E from V and Y, dx
//   producer                         X, dY and the terms of an item (2-slot ring), the state halves
//                                    (one slot), B and C of a group of heads
//   issuer                           TMEM owner; every tcgen05.mma
//   ddt                              ddt, the sums behind dA and dD
//   store                            the dx tiles
//   dot: 2                           <h, dh>, half of the entries each
//
// The roles' code runs at the same time and is fetched through one instruction cache: straight
// FMA code measures 2.4 cycles an instruction up to 24 KB and 6 from 48 KB on (one warp a
// scheduler), so loops stay rolled wherever registers need no constant index, and the slow side of
// every wait is one call.
constexpr int kWarps = 20, kThreads = 32 * kWarps;
enum { ROLE_PAIR, ROLE_ROW, ROLE_ISSUER, ROLE_DDT, ROLE_STORE, ROLE_PRODUCER, ROLE_DOT };
// Test hook: a role held back at every item shows whether the others wait for it where they have to.
constexpr unsigned kLagNs = 20000;  // several items' time
__device__ __forceinline__ void lag(const BwdTc& p, int role) {
    if (p.lag == role) __nanosleep(kLagNs);
}
__device__ __forceinline__ int role_of(int warp) {
    const int q = warp & 3, j = warp >> 2;
    if (j < 4 - q) return ROLE_PAIR;  // c = q + j
    if (j == 4 - q) return ROLE_ROW;
    if (q == 1) return ROLE_ISSUER;
    if (q == 2) return j == 3 ? ROLE_DDT : ROLE_STORE;
    return j == 2 ? ROLE_PRODUCER : ROLE_DOT;
}

constexpr uint32_t kMB = 0;                          // B: n 0..63, 64..127
constexpr uint32_t kMC = kMB + 2 * kRegion;          // C
constexpr uint32_t kMX = kMC + 2 * kRegion;          // [2] X, then the dx tile
constexpr uint32_t kMY = kMX + 2 * kRegion;          // [2] dY
constexpr uint32_t kMH = kMY + 2 * kRegion;          // h image; at a group's end the dS^T tile
constexpr uint32_t kMG = kMH + kImage;               // dh image
constexpr uint32_t kMW = kMG + kImage;               // e o dY, then w dt o X
constexpr uint32_t kMTerms = kMW + kRegion;          // [2] terms
constexpr uint32_t kMSums = kMTerms + 2 * kTermBytes;
// per item, fp32 [128] each: row sums of W by quadrant of j (4), column sums by group of i (4),
// S_jj, Gm_jj, E, F / dt
constexpr int kSumRow = 0, kSumCol = 4, kSumSd = 8, kSumGd = 9, kSumE = 10, kSumF = 11, kSums = 12;
constexpr uint32_t kSumBytes = kSums * kBlk * 4;
constexpr uint32_t kMSmall = kMSums + 2 * kSumBytes;
constexpr uint32_t kMSmem = kMSmall + 512;
static_assert(kMSmem <= 232448 - 1024, "main pass shared memory");

constexpr uint32_t kColB = 0, kColC = 128, kColG = 256, kColV = 384, kColY = 448;

enum {
    MB_FULLXY = 0,    // [2] X, dY, terms landed
    MB_EMPTYXY = 2,   // [2] row warps done with dY (4), dx tile read out (1)
    MB_EMPTYT = 4,    // [2] terms read: pair (10), row (4), ddt (1)
    MB_FULLST = 6,    // state halves landed
    MB_EMPTYST = 7,   // every product that reads them done (1), <h, dh> done (2)
    MB_FULLBC = 8,    // B, C landed
    MB_SFULL = 9,     // S^T accumulated
    MB_SREAD = 10,    // pair warps read it (10)
    MB_GFULL = 11,    // G^T accumulated
    MB_MREADY = 12,   // pair warps wrote M^T (10)
    MB_UDONE = 13,    // U accumulated: M^T is read too
    MB_VDONE = 14,    // V accumulated
    MB_VSCALED = 15,  // row warps replaced V by w o V (4)
    MB_UFREE = 16,    // row warps read U (4)
    MB_YDONE = 17,    // Y accumulated
    MB_YFREE = 18,    // row warps read Y (4)
    MB_EYREADY = 19,  // row warps wrote e o dY (4)
    MB_DCDONE = 20,   // dC's product done: the tile is free
    MB_WXREADY = 21,  // row warps wrote w dt o X (4)
    MB_DBDONE = 22,   // dB's product done: the tile is free
    MB_SUMFULL = 23,  // [2] sums written: pair (10), row (4), <h, dh> (2)
    MB_SUMEMPTY = 25, // [2] sums read (1)
    MB_DXSTAGED = 27, // [2] dx tile written (4)
    MB_DSREADY = 29,  // pair warps wrote the dS^T tile (10)
    MB_ACCDONE = 30,  // dB, dC complete
    MB_UNITFREE = 31, // pair warps read them (10): B, C, the accumulators and the tile are free
    MB_DONE = 32,
    MB_COUNT
};
static_assert(MB_COUNT * 8 <= 320, "barriers");
__device__ __forceinline__ uint32_t main_bar_count(int i) {
    switch (i) {
        case MB_EMPTYXY: case MB_EMPTYXY + 1: return 5;
        case MB_EMPTYT: case MB_EMPTYT + 1: return 15;
        case MB_SUMFULL: case MB_SUMFULL + 1: return 16;
        case MB_EMPTYST: return 3;
        case MB_SREAD: case MB_MREADY: case MB_DSREADY: case MB_UNITFREE: return 10;
        case MB_VSCALED: case MB_UFREE: case MB_YFREE: case MB_EYREADY: case MB_WXREADY:
        case MB_DXSTAGED: case MB_DXSTAGED + 1: return 4;
        default: return 1;
    }
}

// v[i] of every lane summed over the lanes; lane l gets the sum of v[l % 16].  Halving exchange: 16
// shuffles for 16 sums.
__device__ __forceinline__ float transpose_sum(float (&v)[16], int lane) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

// First item of CTA x: the items split evenly (the first `more` CTAs hold one more), or each group's
// heads over its CTAs.  Items are fewer than 2^31.
__device__ __forceinline__ int first_item(const BwdTc& p, int x) {
    if (p.per_group == 0) return x * p.each + min(x, p.more);
    const int hg = p.a.H / p.a.G;
    return x / p.per_group * hg + x % p.per_group * hg / p.per_group;
}

// The items of one CTA, [lo, hi) of items = b nc H (< 2^31), in order: item (chunk bc of all
// sequences' chunks, head h), the head's place hh in its group.  Divisions happen once.
struct Walk {
    int k, n, h, hh, bc;  // k-th of n
    int H, hg;
    __device__ __forceinline__ Walk(int lo, int hi, int H_, int hg_) : k(0), n(hi - lo), H(H_), hg(hg_) {
        bc = lo / H;
        h = lo - bc * H;
        hh = h % hg;
    }
    __device__ __forceinline__ bool first() const { return k == 0 || hh == 0; }  // of its group, in this CTA
    __device__ __forceinline__ bool last() const { return k + 1 == n || hh + 1 == hg; }
    __device__ __forceinline__ bool more() const { return k < n; }
    __device__ __forceinline__ void next() {
        ++k;
        if (++hh == hg) hh = 0;
        if (++h == H) h = 0, ++bc;
    }
    __device__ __forceinline__ int next_head() const { return h + 1 == H ? 0 : h + 1; }
};

__global__ void __launch_bounds__(kThreads, 1) ssd_bwd_tc_main_kernel(const __grid_constant__ BwdTc p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    // uniform for the compiler too: what a warp feeds to tcgen05 and TMA stays in uniform registers
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int role = role_of(warp), q = warp & 3;
    const int H = p.a.H, G = p.a.G, T = p.a.T, hg = H / G;
    const int lo = first_item(p, blockIdx.x), hi = first_item(p, blockIdx.x + 1);
    uint8_t* small = smem + kMSmall;
    uint64_t* bars = reinterpret_cast<uint64_t*>(small);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(small + 336);
    float* s_z = reinterpret_cast<float*>(small + 352);  // [2][2]
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    // waits of a whole warp, and of one thread
    auto wt = [&](int b, uint32_t n, uint32_t site) { return wait_warp(bar(b), n, site); };
    auto w1 = [&](int b, uint32_t n, uint32_t site) { return wait_one(bar(b), n, site); };
    // one arrival of the warp, once all its lanes are here
    auto arrive = [&](int b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b));
    };

    if (threadIdx.x == 0) {
        const bool misaligned = (sbase & 1023u) != 0;
        if (misaligned) report_status(p.status, SSD_ERR_INTERNAL | (7 << 8));
        for (int i = 0; i < MB_COUNT; ++i) mbar_init(bar(i), main_bar_count(i));
        s_stop = misaligned ? 1 : 0;
        s_status = p.status;
        s_wait_ns = p.wait_ns;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_alloc_cta(s_tmem, 512, role == ROLE_ISSUER), 0);
    if (tmem == kTmemSentinel) {
        s_stop = 1;
        report_status(p.status, SSD_ERR_INTERNAL | (8 << 8));
    }
    griddep_launch();
    griddep_wait();  // what the launches ahead wrote
    // Every role walks the same items: i.k counts them (per-item barriers complete once each), n
    // the groups begun.
    if (role == ROLE_PAIR) {
        const int c = q + (warp >> 2);  // columns i: tokens 32 c ..
        const bool diagonal = c == q;
        const int r = q * 32 + lane;    // row: token j
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16), at = lanes + kColG + c * 32;
        // the blocks of quadrant q with i < j, which its 4 - q warps keep zero between them
        const int z0 = c - q, zstep = 4 - q;
        f32x2 S[16], dS[16];  // pairs of columns
        float sd = 0.f;       // S_jj
        bool live = __all_sync(0xffffffffu, !stopped());
        int n = 0;
        for (Walk i(lo, hi, H, hg); i.more() && live; i.next()) {
            const int k = i.k, s = k & 1;
            if (i.first()) {
                live = wt(MB_SFULL, n, 100);
                if (!live) break;
                tc_fence_after();
                uint32_t raw[32];
                SSD_TMEM_LD32_WAIT(at, raw);
                tc_fence_before();
                arrive(MB_SREAD);
                ++n;
                // of the diagonal block only i > j stays: i = j, where L = 1, goes by S_jj and Gm_jj
                // (its terms of W straddle no token, and dx_j takes dt_j S_jj dy_j from the row warp)
                if (diagonal) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (j == lane) sd = __uint_as_float(raw[j]);
                        if (j <= lane) raw[j] = 0u;
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    S[j] = pack2(__uint_as_float(raw[2 * j]), __uint_as_float(raw[2 * j + 1]));
                    dS[j] = 0ull;
                }
            }
            live = wt(MB_FULLXY + s, k >> 1, 101) && (k < 2 || wt(MB_SUMEMPTY + s, (k - 2) >> 1, 102)) &&
                   wt(MB_GFULL, k, 103);
            if (!live) break;
            lag(p, ROLE_PAIR);
            tc_fence_after();
            const float* terms = reinterpret_cast<const float*>(smem + kMTerms + s * kTermBytes);
            float* sums = reinterpret_cast<float*>(smem + kMSums + s * kSumBytes);
            const float dtj = terms[kTermDt * kBlk + r];
            // L_ij = exp(cs_i - cs_j) = 2^(csub_i + d): -d is csub_j, less the totals of the groups
            // between.  The high parts' sums are exact where they cancel, and round where L is small
            float d = -terms[cs2_at(r)], dl = -terms[cs2_at(r) + kCs2Lo];
#pragma unroll 1
            for (int b = q; b < c; ++b) d += terms[cs2_at(32 * b + 31)], dl += terms[cs2_at(32 * b + 31) + kCs2Lo];
            const f32x2 d2 = pack2(d, d), dl2 = pack2(dl, dl), dt2 = pack2(dtj, dtj);
            const float4* cs2 = reinterpret_cast<const float4*>(terms + cs2_at(32 * c));
            f32x2 col2 = 0ull;
            float gd = 0.f;
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // 16 columns at a time beside S and dS
                uint32_t raw[16];
                SSD_TMEM_LD16_WAIT(at + 16 * half, raw);
                float w[16];
                uint32_t pk[8];
#pragma unroll
                for (int j = 0; j < 16; ++j) w[j] = __uint_as_float(raw[j]);
                if (diagonal) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (16 * half + j == lane) gd = w[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int m = 8 * half + j;
                    const float4 v = cs2[m];
                    float l0, l1, a, b;
                    unpack2(add2(add2(pack2(v.x, v.y), d2), add2(pack2(v.z, v.w), dl2)), l0, l1);
                    // above the diagonal S is zero and dS is dropped in the end; the bound keeps L finite
                    // there (below it L <= 1)
                    const f32x2 l = pack2(ex2(fminf(l0, 64.f)), ex2(fminf(l1, 64.f)));
                    const f32x2 t = mul2(pack2(w[2 * j], w[2 * j + 1]), l);
                    dS[m] = fma2(t, dt2, dS[m]);
                    unpack2(mul2(S[m], l), a, b);
                    pk[j] = pack_bf16(a, b);
                    const f32x2 ww = mul2(S[m], t);
                    col2 = add2(col2, ww);
                    unpack2(mul2(ww, dt2), w[2 * j], w[2 * j + 1]);
                }
                SSD_TMEM_ST8_WAIT(at + 8 * half, pk);  // over the first 16 of the block's columns
                const float row = transpose_sum(w, lane);
                if (lane < 16) sums[(kSumRow + q) * kBlk + 32 * c + 16 * half + lane] = row;
            }
            {
                uint32_t zero[16] = {};
#pragma unroll 1
                for (int z = z0; z < q; z += zstep) SSD_TMEM_ST16_WAIT(lanes + kColG + z * 32, zero);
            }
            if (diagonal) {  // ahead of M^T: the row warps read S_jj once U, which waits for it, is done
                sums[kSumSd * kBlk + r] = sd;
                sums[kSumGd * kBlk + r] = gd;
            }
            tc_fence_before();
            arrive(MB_MREADY);
            float ca, cb;
            unpack2(col2, ca, cb);
            sums[(kSumCol + c) * kBlk + r] = ca + cb;
            arrive(MB_SUMFULL + s);
            arrive(MB_EMPTYT + s);
            if (i.last()) {
                // dS^T [j][i] in bf16 over the h image, once the item's products and <h, dh> have read
                // it.  This is the one barrier not waited for at every item, and a parity alone would
                // take phase k - 2 for phase k while the <h, dh> warps still read item k - 1; V being
                // done says that its states had landed, so phase k - 1 is complete
                live = wt(MB_VDONE, k, 106) && wt(MB_EMPTYST, k, 104);
                if (!live) break;
                uint8_t* tile = smem + kMH;
                if (diagonal) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float a, b;
                        unpack2(dS[j], a, b);
                        dS[j] = pack2(2 * j >= lane ? a : 0.f, 2 * j + 1 >= lane ? b : 0.f);
                    }
                }
#pragma unroll
                for (int c4 = 0; c4 < 4; ++c4) {
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float a, b;
                        unpack2(dS[4 * c4 + j], a, b);
                        o[j] = pack_bf16(a, b);
                    }
                    *reinterpret_cast<uint4*>(tile + (c >> 1) * kRegion + swz(r, (c & 1) * 4 + c4)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
#pragma unroll 1
                for (int z = z0; z < q; z += zstep)
#pragma unroll
                    for (int c4 = 0; c4 < 4; ++c4)
                        *reinterpret_cast<uint4*>(tile + (z >> 1) * kRegion + swz(r, (z & 1) * 4 + c4)) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async();
                arrive(MB_DSREADY);
                live = wt(MB_ACCDONE, n - 1, 105);
                if (!live) break;
                tc_fence_after();
                // row r of dB, dC by 32 columns, the quadrant's warps in turn: complete if all the
                // group's heads were here, else the CTA's share.  Its first group's share lies in slot 0,
                // a later one's in slot 1
                const int g = i.h / hg, bi = i.bc / p.nc, t0 = (i.bc - bi * p.nc) * kBlk;
                const bool whole = k - i.hh >= 0 && i.hh + 1 == hg;
                const size_t row = (((size_t)bi * T + t0 + r) * G + g) * kN;
                float* part = p.part + ((size_t)blockIdx.x * 2 + (k - i.hh > 0 ? 1 : 0)) * 2 * kBlk * kN + (size_t)r * kN;
#pragma unroll 1
                for (int m = z0; m < 8; m += zstep) {
                    uint32_t raw[32];
                    const int which = m >> 2, o = (m & 3) * 32;
                    SSD_TMEM_LD32_WAIT(lanes + (which ? kColC : kColB) + o, raw);
                    if (whole) {
                        if (t0 + r < T) {
                            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(which ? p.a.dC : p.a.dB) + row + o);
#pragma unroll
                            for (int c4 = 0; c4 < 4; ++c4)
                                dst[c4] = make_uint4(
                                    pack_bf16(__uint_as_float(raw[8 * c4 + 0]), __uint_as_float(raw[8 * c4 + 1])),
                                    pack_bf16(__uint_as_float(raw[8 * c4 + 2]), __uint_as_float(raw[8 * c4 + 3])),
                                    pack_bf16(__uint_as_float(raw[8 * c4 + 4]), __uint_as_float(raw[8 * c4 + 5])),
                                    pack_bf16(__uint_as_float(raw[8 * c4 + 6]), __uint_as_float(raw[8 * c4 + 7])));
                        }
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(part + which * kBlk * kN + o);
#pragma unroll
                        for (int c4 = 0; c4 < 8; ++c4)
                            dst[c4] = make_uint4(raw[4 * c4], raw[4 * c4 + 1], raw[4 * c4 + 2], raw[4 * c4 + 3]);
                    }
                    __syncwarp();
                }
                tc_fence_before();
                arrive(MB_UNITFREE);
            }
        }
    } else if (role == ROLE_ROW) {
        const int r = q * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
        bool live = __all_sync(0xffffffffu, !stopped());
        float D_next = p.a.D[lo % H];
        for (Walk i(lo, hi, H, hg); i.more() && live; i.next()) {
            const int k = i.k, s = k & 1;
            live = wt(MB_FULLXY + s, k >> 1, 110) && (k < 1 || wt(MB_DBDONE, k - 1, 111));
            if (!live) break;
            lag(p, ROLE_ROW);
            const float* terms = reinterpret_cast<const float*>(smem + kMTerms + s * kTermBytes);
            const float er = terms[kTermE * kBlk + r], wr = terms[kTermW * kBlk + r], dtr = terms[kTermDt * kBlk + r];
            const float Dh = D_next;
            D_next = p.a.D[i.next_head()];
            arrive(MB_EMPTYT + s);
            uint8_t* xs = smem + kMX + s * kRegion;
            const uint8_t* ys = smem + kMY + s * kRegion;
            float* sums = reinterpret_cast<float*>(smem + kMSums + s * kSumBytes);
            float F = 0.f, E = 0.f;
            // the rows of dY weighted with e, then, once dC's product has read them, of X with w dt
#pragma unroll 1
            for (int round = 0; round < 2; ++round) {
                if (round) live = wt(MB_DCDONE, k, 112);
                if (!live) break;
                const uint8_t* src = round ? xs : ys;
                const float weight = round ? wr * dtr : er;
                // x w in bf16 with one rounding that counts: x w_lo first, then fused x w_hi + that
                const __nv_bfloat162 whi = __float2bfloat162_rn(weight);
                const __nv_bfloat162 wlo = __float2bfloat162_rn(weight - __low2float(whi));
#pragma unroll 2
                for (int c = 0; c < 8; ++c) {
                    uint4 v = *reinterpret_cast<const uint4*>(src + swz(r, c));
                    __nv_bfloat162* e = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[j] = __hfma2(e[j], whi, __hmul2(e[j], wlo));
                    *reinterpret_cast<uint4*>(smem + kMW + swz(r, c)) = v;
                }
                fence_proxy_async();
                arrive(round ? MB_WXREADY : MB_EYREADY);
            }
            if (!live) break;
            // V against x, with w o V in its place, then Y against dy
#pragma unroll 1
            for (int round = 0; round < 2; ++round) {
                live = wt(round ? MB_YDONE : MB_VDONE, k, 113);
                if (!live) break;
                tc_fence_after();
                const uint8_t* other = round ? ys : xs;
                const uint32_t from = lanes + (round ? kColY : kColV);
                const f32x2 wr2 = pack2(wr, wr);
                f32x2 dots[2] = {0ull, 0ull};
#pragma unroll 1
                for (int o = 0; o < 4; ++o) {
                    const uint4 rows[2] = {*reinterpret_cast<const uint4*>(other + swz(r, 2 * o)),
                                           *reinterpret_cast<const uint4*>(other + swz(r, 2 * o + 1))};
                    uint32_t raw[16];
                    SSD_TMEM_LD16_WAIT(from + 16 * o, raw);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t in[4] = {rows[c].x, rows[c].y, rows[c].z, rows[c].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t &ra = raw[8 * c + 2 * j], &rb = raw[8 * c + 2 * j + 1];
                            const f32x2 t = pack2(__uint_as_float(ra), __uint_as_float(rb));
                            dots[c] = fma2(pack2(bf_lo(in[j]), bf_hi(in[j])), t, dots[c]);
                            float a, b;
                            unpack2(mul2(t, wr2), a, b);
                            ra = __float_as_uint(a), rb = __float_as_uint(b);
                        }
                    }
                    if (!round) SSD_TMEM_ST16_WAIT(from + 16 * o, raw);
                }
                tc_fence_before();
                arrive(round ? MB_YFREE : MB_VSCALED);
                float a, b;
                unpack2(add2(dots[0], dots[1]), a, b);
                if (round) E = a + b;  // E_i = e_i dy_i . Y_i
                else F = a + b;        // F_j / dt_j = w_j x_j . V_j
            }
            live = live && (k < 2 || wt(MB_SUMEMPTY + s, (k - 2) >> 1, 115));
            if (!live) break;
            sums[kSumE * kBlk + r] = er * E;
            sums[kSumF * kBlk + r] = wr * F;
            arrive(MB_SUMFULL + s);
            // dx = dt (U + S_jj dy) + D dy, over the thread's own row of X
            live = wt(MB_UDONE, k, 116);
            if (!live) break;
            tc_fence_after();
            const float dyw = fmaf(dtr, sums[kSumSd * kBlk + r], Dh);
            const f32x2 dy2 = pack2(dyw, dyw), dt2 = pack2(dtr, dtr);
#pragma unroll 1
            for (int o = 0; o < 4; ++o) {
                const uint4 rows[2] = {*reinterpret_cast<const uint4*>(ys + swz(r, 2 * o)),
                                       *reinterpret_cast<const uint4*>(ys + swz(r, 2 * o + 1))};
                uint32_t raw[16];
                SSD_TMEM_LD16_WAIT(lanes + kColV + 16 * o, raw);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t in[4] = {rows[c].x, rows[c].y, rows[c].z, rows[c].w};
                    uint32_t out[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const f32x2 y2 = mul2(pack2(bf_lo(in[j]), bf_hi(in[j])), dy2);
                        float a, b;
                        unpack2(fma2(pack2(__uint_as_float(raw[8 * c + 2 * j]), __uint_as_float(raw[8 * c + 2 * j + 1])), dt2, y2), a, b);
                        out[j] = pack_bf16(a, b);
                    }
                    *reinterpret_cast<uint4*>(xs + swz(r, 2 * o + c)) = make_uint4(out[0], out[1], out[2], out[3]);
                }
            }
            fence_proxy_async();
            tc_fence_before();
            arrive(MB_UFREE);
            arrive(MB_DXSTAGED + s);
            arrive(MB_EMPTYXY + s);
        }
    } else if (role == ROLE_PRODUCER) {
        if (lane == 0 && !stopped() && !p.starve) {
            int nxy = 0, nst = 0, nbc = 0, n = 0;
            for (Walk i(lo, hi, H, hg); i.more(); i.next()) {
                const int k = i.k, s = k & 1, h = i.h, bi = i.bc / p.nc, t0 = (i.bc - bi * p.nc) * kBlk;
                const size_t it = (size_t)(lo + k);
                lag(p, ROLE_PRODUCER);
                if (k >= 2 && !(w1(MB_EMPTYXY + s, (k - 2) >> 1, 60) && w1(MB_EMPTYT + s, (k - 2) >> 1, 61))) break;
                const uint32_t f = bar(MB_FULLXY + s);
                mbar_expect_tx(f, 2 * kRegion + kTermBytes);
                tma_load_4d(sbase + kMX + s * kRegion, &p.tm_x, f, 0, h, t0, bi);
                tma_load_4d(sbase + kMY + s * kRegion, &p.tm_dy, f, 0, h, t0, bi);
                bulk_load(sbase + kMTerms + s * kTermBytes, p.terms + it * kTerms * kBlk, kTermBytes, f);
                nxy = k + 1;
                if (i.first()) {
                    if (n > 0 && !w1(MB_UNITFREE, n - 1, 62)) break;
                    const uint32_t fb = bar(MB_FULLBC);
                    const int g = h / hg;
                    mbar_expect_tx(fb, 4 * kRegion);
                    tma_load_4d(sbase + kMB, &p.tm_B, fb, 0, g, t0, bi);
                    tma_load_4d(sbase + kMB + kRegion, &p.tm_B, fb, 64, g, t0, bi);
                    tma_load_4d(sbase + kMC, &p.tm_C, fb, 0, g, t0, bi);
                    tma_load_4d(sbase + kMC + kRegion, &p.tm_C, fb, 64, g, t0, bi);
                    nbc = ++n;
                }
                if (k >= 1 && !w1(MB_EMPTYST, k - 1, 63)) break;
                const uint32_t fs = bar(MB_FULLST);
                mbar_expect_tx(fs, 2 * kImage);
                bulk_load(sbase + kMG, p.img_g + it * kImage, kImage, fs);
                bulk_load(sbase + kMH, p.img_h + it * kImage, kImage, fs);
                nst = k + 1;
            }
            // loads nobody may have waited for land before the CTA exits
            for (int k = nxy - 2; k < nxy; ++k)
                if (k >= 0) mbar_drain(bar(MB_FULLXY + (k & 1)), (k >> 1) & 1);
            if (nst > 0) mbar_drain(bar(MB_FULLST), (nst - 1) & 1);
            if (nbc > 0) mbar_drain(bar(MB_FULLBC), (nbc - 1) & 1);
        }
        __syncwarp();
    } else if (role == ROLE_ISSUER) {
        // One lane issues everything, in small rolled loops whose descriptors advance by constants.  (A
        // loop over products with their layouts as data took 190 cycles an instruction; unrolled, the
        // code crowds the instruction cache.)
        if (elect_one()) {
            constexpr uint32_t id_nn = idesc_bf16(128, 128, 0, 0);   // both K-major
            constexpr uint32_t id_st = idesc_bf16(128, 64, 0, 1);    // state or dY [K rows][64]: MN-major
            constexpr uint32_t id_db = idesc_bf16(128, 128, 0, 1);
            constexpr uint32_t id_dc = idesc_bf16(128, 128, 1, 1);
            // K-major operands step 16 elements along a row (32 bytes), and every 64 a region; MN-major
            // ones step 16 rows
            auto k_major = [](uint32_t a) { return sdesc(a, 16, 1024); };
            auto mn_major = [](uint32_t a) { return sdesc(a, kRegion, 1024); };
            constexpr uint32_t kCol = 2, kRow = 128, kReg = kRegion >> 4;
            auto run4 = [&](uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {  // K = 64, both K-major
#pragma unroll 1
                for (int kk = 0; kk < 4; ++kk, a += kCol, b += kCol) mma_ss(d, a, b, id, acc | kk);
            };
            // K = 128, a K-major over two regions, b MN-major
            auto run8 = [&](uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
#pragma unroll 1
                for (int kk = 0; kk < 8; ++kk, b += kRow) {
                    mma_ss(d, a, b, id, acc | kk);
                    a += kk == 3 ? kReg - 3 * kCol : kCol;
                }
            };
            // the same against both halves of a state image
            auto run8_state = [&](uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll 1
                for (int kk = 0; kk < 8; ++kk, b += kRow) {
                    mma_ss_pair(d, a, b, b + kReg, id_st, kk);
                    a += kk == 3 ? kReg - 3 * kCol : kCol;
                }
            };
            const uint64_t kB = k_major(sbase + kMB), kC = k_major(sbase + kMC), kW = k_major(sbase + kMW);
            const uint64_t kX0 = k_major(sbase + kMX), kY0 = k_major(sbase + kMY), mY0 = mn_major(sbase + kMY);
            bool ok = !stopped();
            int n = -1;
#pragma unroll 1
            for (Walk i(lo, hi, H, hg); i.more() && ok; i.next()) {
                const int k = i.k, s = k & 1;
                const bool fresh = i.first();
                const uint32_t stage = s * kReg;
                lag(p, ROLE_ISSUER);
                // G^T's columns: U of the item before has read M^T there
                ok = k < 1 || w1(MB_UDONE, k - 1, 70);
                if (!ok) break;
                if (fresh) {
                    ++n;
                    ok = w1(MB_FULLBC, n, 71);
                    if (!ok) break;
                    tc_fence_after();
                    run4(tmem + kColG, kB, kC, id_nn, 0);
                    run4(tmem + kColG, kB + kReg, kC + kReg, id_nn, 1);
                    mma_commit(bar(MB_SFULL));
                    ok = w1(MB_SREAD, n, 72);
                    if (!ok) break;
                }
                ok = w1(MB_FULLXY + s, k >> 1, 73);
                if (!ok) break;
                tc_fence_after();
                run4(tmem + kColG, kX0 + stage, kY0 + stage, id_nn, 0);
                mma_commit(bar(MB_GFULL));
                // V = B dh^T, then Y = C h^T, each from both halves
                ok = w1(MB_FULLST, k, 74) && (k < 1 || w1(MB_UFREE, k - 1, 75));
                if (!ok) break;
                tc_fence_after();
                run8_state(tmem + kColV, kB, mn_major(sbase + kMG));
                mma_commit(bar(MB_VDONE));
                // dC += (e o dY) h, dB += (w dt o X) dh: the images as K-major [n][p]
                ok = w1(MB_EYREADY, k, 77);
                if (!ok) break;
                tc_fence_after();
                run4(tmem + kColC, kW, k_major(sbase + kMH), id_nn, !fresh);
                mma_commit(bar(MB_DCDONE));
                ok = k < 1 || w1(MB_YFREE, k - 1, 76);
                if (!ok) break;
                tc_fence_after();
                run8_state(tmem + kColY, kC, mn_major(sbase + kMH));
                mma_commit(bar(MB_YDONE));
                ok = w1(MB_WXREADY, k, 78);
                if (!ok) break;
                tc_fence_after();
                run4(tmem + kColB, kW, k_major(sbase + kMG), id_nn, !fresh);
                mma_commit(bar(MB_DBDONE));
                mma_commit(bar(MB_EMPTYST));
                // U = w o V + M^T dY
                ok = w1(MB_VSCALED, k, 79) && w1(MB_MREADY, k, 80);
                if (!ok) break;
                tc_fence_after();
                {
                    uint64_t b = mY0 + stage;
                    uint32_t a = tmem + kColG;  // M^T: 16 columns of 32 hold 32 of K
#pragma unroll 1
                    for (int kk = 0; kk < 8; ++kk, b += kRow, a += kk & 1 ? 8 : 24) mma_ts(tmem + kColV, a, b, id_st, 1);
                }
                mma_commit(bar(MB_UDONE));
                if (i.last()) {  // dB += dS^T C, dC += dS B
                    ok = w1(MB_DSREADY, n, 81);
                    if (!ok) break;
                    tc_fence_after();
                    run8(tmem + kColB, k_major(sbase + kMH), mn_major(sbase + kMC), id_db, 1);
                    uint64_t a = mn_major(sbase + kMH), b = mn_major(sbase + kMB);
#pragma unroll 1
                    for (int kk = 0; kk < 8; ++kk, a += kRow, b += kRow) mma_ss(tmem + kColC, a, b, id_dc, 1);
                    mma_commit(bar(MB_ACCDONE));
                }
            }
            mma_commit(bar(MB_DONE));
            mbar_drain(bar(MB_DONE), 0);
        }
        __syncwarp();
    } else if (role == ROLE_DDT) {
        bool ok = __all_sync(0xffffffffu, !stopped());
        float A_next = p.a.A[lo % H];
        for (Walk i(lo, hi, H, hg); i.more() && ok; i.next()) {
            const int k = i.k, s = k & 1, h = i.h, bi = i.bc / p.nc, t0 = (i.bc - bi * p.nc) * kBlk;
            const float Ah = A_next;
            A_next = p.a.A[i.next_head()];
            float slope[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) slope[g] = p.slope ? p.slope[(size_t)(lo + k) * kBlk + 32 * g + lane] : 1.f;
            ok = wt(MB_FULLXY + s, k >> 1, 90) && wt(MB_SUMFULL + s, k >> 1, 91);
            if (!ok) break;
            lag(p, ROLE_DDT);
            const float* sums = reinterpret_cast<const float*>(smem + kMSums + s * kSumBytes) + lane;
            const float* terms = reinterpret_cast<const float*>(smem + kMTerms + s * kTermBytes) + lane;
            // da_t adds a prefix of F (exclusive) and a suffix of E + rows - columns.  Lane l holds
            // tokens 32 g + l; the four groups' scans run side by side
            float f[4], dt[4], suf[4], dir[4], sD = 0.f;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                dt[g] = terms[kTermDt * kBlk + 32 * g];
                const float fj = sums[kSumF * kBlk + 32 * g], gd = sums[kSumGd * kBlk + 32 * g];
                float row = sums[kSumE * kBlk + 32 * g], col = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j <= g) row += sums[(kSumRow + j) * kBlk + 32 * g];
                    if (j >= g) col += sums[(kSumCol + j) * kBlk + 32 * g];
                }
                f[g] = fj * dt[g];
                suf[g] = fmaf(-col, dt[g], row);
                dir[g] = fmaf(gd, sums[kSumSd * kBlk + 32 * g], col + fj);
                sD += gd;
            }
            float da = (s_z[2 * s] + s_z[2 * s + 1]) * (terms - lane)[kTermE * kBlk + kBlk - 1];
            arrive(MB_SUMEMPTY + s);
            arrive(MB_EMPTYT + s);
            float pre[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) pre[g] = f[g];
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float a = __shfl_up_sync(0xffffffffu, pre[g], o), b = __shfl_down_sync(0xffffffffu, suf[g], o);
                    if (lane >= o) pre[g] += a;
                    if (lane + o < 32) suf[g] += b;
                }
            }
            float sA = 0.f, sb = 0.f, carry[4], run = da;
#pragma unroll
            for (int g = 3; g >= 0; --g) {
                carry[g] = run;  // <h, dh> and the suffix behind group g
                run += __shfl_sync(0xffffffffu, suf[g], 0);
            }
            run = 0.f;
            float* out = p.a.ddt + ((size_t)bi * T + t0 + lane) * H + h;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                // the F ahead of the token, by a shift: less its own F, the rounding of that would stay
                const float up = __shfl_up_sync(0xffffffffu, pre[g], 1);
                // every pair that straddles a token has its decay as a factor: where that is zero in fp32, so
                // is da, of which the suffix sums leave a rounding that dA would take times a large step
                da = dt[g] * Ah < -104.f ? 0.f : carry[g] + suf[g] + (lane ? run + up : run);
                run += __shfl_sync(0xffffffffu, pre[g], 31);
                const float ddt = fmaf(Ah, da, dir[g]) * slope[g];
                if (t0 + 32 * g + lane < T) {
                    out[(size_t)(32 * g) * H] = ddt;
                    sA = fmaf(dt[g], da, sA);
                    sb += ddt;
                }
            }
#pragma unroll 1
            for (int o = 16; o > 0; o >>= 1) {
                sA += __shfl_xor_sync(0xffffffffu, sA, o);
                sD += __shfl_xor_sync(0xffffffffu, sD, o);
                sb += __shfl_xor_sync(0xffffffffu, sb, o);
            }
            if (lane == 0) {
                p.pA[lo + k] = sA;
                p.pD[lo + k] = sD;
                if (p.pb) p.pb[lo + k] = sb;
            }
            __syncwarp();
        }
    } else if (role == ROLE_STORE) {
        if (lane == 0 && !stopped()) {
            for (Walk i(lo, hi, H, hg); i.more(); i.next()) {
                const int k = i.k, s = k & 1, bi = i.bc / p.nc, t0 = (i.bc - bi * p.nc) * kBlk;
                if (!w1(MB_DXSTAGED + s, k >> 1, 92)) break;
                lag(p, ROLE_STORE);
                tma_store_4d(sbase + kMX + s * kRegion, &p.tm_dx, 0, i.h, t0, bi);
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(bar(MB_EMPTYXY + s));
            }
            bulk_wait0();
        }
        __syncwarp();
    } else {
        // <h, dh>, half of the entries a warp.  hi hi' in fp32; the cross terms, 2^-8 of that, in packed
        // bf16 over the 8 entries of a vector (their error 2^-8 of them again); lo lo' is below both
        const int mine = (warp >> 2) - 3;
        bool ok = __all_sync(0xffffffffu, !stopped());
        for (int k = 0; k < hi - lo && ok; ++k) {
            const int s = k & 1;
            ok = wt(MB_FULLST, k, 95);
            if (!ok) break;
            lag(p, ROLE_DOT);
            const uint4 *h4 = reinterpret_cast<const uint4*>(smem + kMH), *g4 = reinterpret_cast<const uint4*>(smem + kMG);
            f32x2 z2 = 0ull, c2 = 0ull;
#pragma unroll 2
            for (int i = mine * 32 + lane; i < (int)(kRegion / 16); i += 64) {
                const uint4 a = h4[i], al = h4[i + kRegion / 16], b = g4[i], bl = g4[i + kRegion / 16];
                const uint32_t ah[4] = {a.x, a.y, a.z, a.w}, ao[4] = {al.x, al.y, al.z, al.w};
                const uint32_t bh[4] = {b.x, b.y, b.z, b.w}, bo[4] = {bl.x, bl.y, bl.z, bl.w};
                __nv_bfloat162 t = __float2bfloat162_rn(0.f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    auto v = [](const uint32_t& u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
                    z2 = fma2(pack2(bf_lo(ah[j]), bf_hi(ah[j])), pack2(bf_lo(bh[j]), bf_hi(bh[j])), z2);
                    t = __hfma2(v(ah[j]), v(bo[j]), __hfma2(v(ao[j]), v(bh[j]), t));
                }
                const uint32_t tu = *reinterpret_cast<const uint32_t*>(&t);
                c2 = add2(c2, pack2(bf_lo(tu), bf_hi(tu)));
            }
            arrive(MB_EMPTYST);
            float z, z1;
            unpack2(add2(z2, c2), z, z1);
            z += z1;
#pragma unroll 1
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            ok = k < 2 || wt(MB_SUMEMPTY + s, k / 2 - 1, 96);
            if (!ok) break;
            if (lane == 0) s_z[2 * s + mine] = z;
            arrive(MB_SUMFULL + s);
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (role == ROLE_ISSUER && tmem != kTmemSentinel) {
        tc_fence_after();
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

// ------------------------------------------------------------------ dB, dC of split groups
// kJoinSplit blocks a (chunk, group), or, split evenly, for every place where one CTA's items end and the
// next one's begin; where that is the first such place inside a group, they add up its parts.  One
// vector of 4 a thread keeps enough loads in flight for few groups of many parts (8 groups of 16
// parts: 17 us, with two vectors 24 us).
constexpr int kJoinThreads = 256, kJoinSplit = 2 * kBlk * kN / 4 / kJoinThreads;
__global__ void __launch_bounds__(kJoinThreads) ssd_bwd_tc_join_kernel(const __grid_constant__ BwdTc p, const HeadSums hs,
                                                                       unsigned join_blocks) {
    griddep_wait();
    if (blockIdx.x >= join_blocks) return head_sum<kJoinThreads>(hs, (int)(blockIdx.x - join_blocks));
    const int hg = p.a.H / p.a.G;
    int x0 = blockIdx.x / kJoinSplit, x1, unit, slot = 0;  // the group, and the CTAs that hold its items
    if (p.per_group) {
        unit = x0, x0 = unit * p.per_group, x1 = x0 + p.per_group - 1;
    } else {
        const int cut = first_item(p, x0 + 1);
        unit = cut / hg;
        const int from = first_item(p, x0), it0 = unit * hg, last = it0 + hg - 1, longer = p.more * (p.each + 1);
        if (cut == it0 || from > it0) return;
        x1 = last < longer ? last / (p.each + 1) : p.more + (last - longer) / p.each;
        slot = from < it0;  // a CTA's first group sits in its slot 0, a later one (its last) in slot 1
    }
    const int g = unit % p.a.G, bc = unit / p.a.G, bi = bc / p.nc, t0 = (bc % p.nc) * kBlk;
    const int rows = min(kBlk, p.a.T - t0);
    const int i = (int)(blockIdx.x % kJoinSplit) * kJoinThreads + threadIdx.x;
    const int which = i / (kBlk * kN / 4), e = (i % (kBlk * kN / 4)) * 4, r = e / kN, c = e % kN;
    if (r >= rows) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int x = x0; x <= x1; ++x) {
        const float4 v = *reinterpret_cast<const float4*>(p.part + (((size_t)x * 2 + (x == x0 ? slot : 0)) * 2 + which) * kBlk * kN + e);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(which ? p.a.dC : p.a.dB) + (((size_t)bi * p.a.T + t0 + r) * p.a.G + g) * kN + c;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
}

// CTAs of the main pass.  An even split of the items loads the SMs best, but a CTA whose run crosses
// from one (chunk, group) into the next begins two of them, and the groups cut are joined afterwards.
// With few groups each can have CTAs of its own.  In units of an item's 3.2 us a crossing costs about
// 2.5 and its join as much, a join of k parts of whole groups 0.6 + 0.07 k.  Main pass and join, split
// evenly and by groups: 1024 items in 128 groups 71 and 54 us, 768 in 32 groups 61 and 52 us, 3072 in 64
// groups 127 and 122 us; more groups than SMs leave the even split only.
void plan_main(BwdTc* p) {
    const int sms = device_sms(), hg = p->a.H / p->a.G, items = (int)p->items, groups = items / hg;
    p->ctas = std::min(items, sms);
    p->per_group = 0;
    const int most = (items + p->ctas - 1) / p->ctas;
    double best = most + 5.0;
    for (int k = 1; k <= hg && groups * (long long)k <= sms; ++k) {
        const double cost = (hg + k - 1) / k + (k > 1 ? 0.6 + 0.07 * k : 0.0);
        if (cost < best) best = cost, p->per_group = k;
    }
    if (p->per_group) p->ctas = groups * p->per_group;
    p->each = items / p->ctas, p->more = items % p->ctas;
}

// Pairs of the state pass walked whole, and segments of the others.  A CTA walks its chunks one after
// another, which costs a chunk's time each and a start of about two.  Segments fill the SMs that whole
// pairs leave idle in their last wave, but the ends kernel walks all but the last of them once more
// (without the stores: 16 us against 20 us for 11 chunks), and each fold of an end is taken as a
// quarter of a chunk.  Whole pairs are scheduled first; the cheapest of a few dozen plans wins.
void plan_segments(int b, int H, int nc, int* n_whole, int* nseg, int* cseg) {
    const int sms = device_sms(), pairs = b * H, waves = 2 * pairs / sms;
    double best = 0.0;
    bool first = true;
    auto consider = [&](int whole, int n) {
        const int len = (nc + n - 1) / n, split = pairs - whole;
        if ((nc + len - 1) / len != n) return;
        const double wt = nc + 2.0, st = len + 2.0 + 0.25 * (n - 1), et = 0.8 * len + 2.0;
        const int q = 2 * whole / sms, r = 2 * whole % sms;  // full waves of whole pairs, and the SMs of one more
        const double s = 2.0 * split * n;
        double cost = q * wt;
        if (s > 0.0) {
            const double beside = (sms - r) * std::floor(r ? wt / st : 0.0);  // segments done beside the last wave
            if (r && s <= beside) cost += std::max(wt, std::ceil(s / (sms - r)) * st);
            else cost += (r ? wt : 0.0) + std::ceil((s - beside) / sms) * st;
            if (n > 1) cost += std::ceil(2.0 * split * (n - 1) / sms) * et + 5.0;
        } else if (r) {
            cost += wt;
        }
        if (first || cost < best) best = cost, *n_whole = whole, *nseg = n, *cseg = len, first = false;
    };
    consider(pairs, 1);
    for (int n = 2; n <= std::min(nc, 64); ++n) {
        consider(0, n);
        for (int w = std::max(0, waves - 1); w <= waves; ++w)
            for (int f = 0; f < 8; ++f) {  // w waves of whole pairs and f eighths of one more
                const int whole = (w * sms + f * sms / 8) / 2;
                if (whole > 0 && whole < pairs) consider(whole, n);
            }
    }
    if (*n_whole == pairs) *nseg = 1, *cseg = nc;
}

size_t tc_layout(const BwdArgs& a, char* ws, BwdTc* p) {
    p->a = a;
    p->nc = (a.T + kBlk - 1) / kBlk;
    p->items = (long long)a.b * p->nc * a.H;
    plan_main(p);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        char* r = ws ? ws + o : nullptr;
        o += round_up(bytes, 256);
        return r;
    };
    const size_t n = (size_t)p->items;
    p->terms = reinterpret_cast<float*>(take(n * kTermBytes));
    p->slope = reinterpret_cast<float*>(take(n * kBlk * 4));
    p->img_h = reinterpret_cast<uint8_t*>(take(n * kImage));
    p->img_g = reinterpret_cast<uint8_t*>(take(n * kImage));
    plan_segments(a.b, a.H, p->nc, &p->n_whole, &p->nseg, &p->cseg);
    const size_t ends = ((size_t)a.b * a.H - p->n_whole) * 2 * (p->nseg - 1);
    p->seg_end = reinterpret_cast<float*>(take(ends * kP * kN * 4));
    p->seg_decay = reinterpret_cast<float*>(take(ends * 4));
    p->part = reinterpret_cast<float*>(take((size_t)p->ctas * 4 * kBlk * kN * 4));
    p->pA = reinterpret_cast<float*>(take(n * 4));
    p->pD = reinterpret_cast<float*>(take(n * 4));
    p->pb = reinterpret_cast<float*>(take(n * 4));
    return o;
}

std::atomic<unsigned long long> g_starve_bwd{0};
std::atomic<int> g_lag_bwd{-1};

}  // namespace

bool backward_tc_supported(int P, int N, int io) { return io == SSD_BF16 && P == kP && N == kN; }

size_t backward_tc_workspace_bytes(const BwdArgs& a) {
    BwdTc p;
    return tc_layout(a, nullptr, &p);
}

void backward_tc_starve_next(unsigned long long wait_ns) { g_starve_bwd.store(wait_ns); }

int backward_tc_lag_next(int role) {
    if (role < 0 || role > ROLE_DOT)
        return set_error(SSD_ERR_INVALID_ARG, "role %d outside [0, %d]", role, (int)ROLE_DOT);
    g_lag_bwd.store(role);
    return SSD_OK;
}

// ws: the status word at its start, the passes' scratch `offset` bytes behind it
int launch_backward_tc(const BwdArgs& a, void* ws, size_t offset, cudaStream_t s) {
    BwdTc p;
    memset(&p, 0, sizeof(p));
    tc_layout(a, static_cast<char*>(ws) + offset, &p);
    if (!a.dbias) p.pb = nullptr;
    if (!a.dtm.raw) p.slope = nullptr;
    p.status = static_cast<int*>(ws);
    const unsigned long long starve = g_starve_bwd.exchange(0);
    p.starve = starve != 0;
    p.wait_ns = starve ? starve : kWaitLimitNs;
    p.lag = g_lag_bwd.exchange(-1);
    int st;
    if ((st = make_map(&p.tm_x, a.x, kP, a.H, a.T, a.b)) != SSD_OK) return st;
    if ((st = make_map(&p.tm_dy, a.dy, kP, a.H, a.T, a.b)) != SSD_OK) return st;
    if ((st = make_map(&p.tm_B, a.B, kN, a.G, a.T, a.b)) != SSD_OK) return st;
    if ((st = make_map(&p.tm_C, a.C, kN, a.G, a.T, a.b)) != SSD_OK) return st;
    if ((st = make_map(&p.tm_dx, a.dx, kP, a.H, a.T, a.b)) != SSD_OK) return st;
    if ((st = smem_limit_once((const void*)ssd_bwd_tc_state_kernel<false>, (int)kSSmem)) != SSD_OK) return st;
    if ((st = smem_limit_once((const void*)ssd_bwd_tc_state_kernel<true>, (int)kSSmem)) != SSD_OK) return st;
    if ((st = smem_limit_once((const void*)ssd_bwd_tc_main_kernel, (int)kMSmem)) != SSD_OK) return st;
    {
        LaunchScope ls("ssd_bwd_tc_terms", s);
        ssd_bwd_tc_terms_kernel<<<dim3(a.b * p.nc, (a.H + 7) / 8), kTermThreads, 0, s>>>(p);
        SSD_CUDA_TRY(cudaGetLastError());
    }
    const int split = a.b * a.H - p.n_whole;
    if (p.nseg > 1) {
        LaunchScope ls("ssd_bwd_tc_ends", s);
        SSD_CUDA_TRY(launch_pdl(ssd_bwd_tc_state_kernel<true>, dim3(2 * split * (p.nseg - 1)), kSThreads, kSSmem, s, p));
    }
    {
        LaunchScope ls("ssd_bwd_tc_state", s);
        SSD_CUDA_TRY(launch_pdl(ssd_bwd_tc_state_kernel<false>, dim3(2 * (p.n_whole + split * p.nseg)), kSThreads, kSSmem, s, p));
    }
    {
        LaunchScope ls("ssd_bwd_tc_main", s);
        SSD_CUDA_TRY(launch_pdl(ssd_bwd_tc_main_kernel, dim3(p.ctas), kThreads, kMSmem, s, p));
    }
    {
        const unsigned join_blocks = p.per_group == 1 ? 0 : (unsigned)(kJoinSplit * (p.per_group ? p.ctas / p.per_group : p.ctas - 1));
        const HeadSums hs{p.pA, p.pD, p.pb, a.b * p.nc, a.H, a.dA, a.dD, a.dbias};
        LaunchScope ls("ssd_bwd_tc_join", s);
        SSD_CUDA_TRY(launch_pdl(ssd_bwd_tc_join_kernel, dim3(join_blocks + hs.blocks()), kJoinThreads, 0, s, p, hs, join_blocks));
    }
    return SSD_OK;
}

}  // namespace ssd
