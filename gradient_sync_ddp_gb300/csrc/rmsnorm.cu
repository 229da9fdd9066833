// RMS norm with the residual's addition, forward (fp32 / bf16 or 8-bit
// output) and backward.
//
//   h = x + residual,  rstd = 1/sqrt(mean(h²) + eps),  y = h·rstd·γ
//   8 bits: scale = max|y| / 127, q = y / scale to the nearest integer
//   backward: n = h·rstd, c = mean(dy·γ·n),
//             dx = rstd·(dy·γ − n·c) + dh,  dγ = Σ_rows dy·n
//
// Sums and statistics are fp32; h is rounded to its type only where it is
// stored, the statistics and y use the unrounded sum.
//
// Bound by HBM (16384 x 4096 bf16 with residual: 537 MB in 84 us, 0.96 of the
// copy rate; with 8 bits out 470 MB in 81 us; backward 8192 x 4096 268 MB in
// 49 us, 0.82; one row of 768 in 1.9 us, a launch): forward reads x and residual and writes h and y once,
// backward reads dy, h and dh and writes dx once.  A row stays in registers
// between the reduction and the output: a warp per row (narrow rows) or a CTA
// per row, 16-byte vectors.  Where rows do not start on 16-byte boundaries (an
// odd width) but all matrices of the call lie alike, the vectors are those of
// the aligned grid and up to 2·(VEC − 1) elements at the row's ends go one per
// thread (16384 x 4099 bf16 124 us, 0.65: γ's columns shift against the
// vectors).  Matrices that lie differently, and rows wider than the registers
// hold, take the element loop (two passes over the row).
// Backward keeps a CTA's rows alike (its grid is a multiple of VEC), so that
// the vectors' columns stay a thread's own there too (5000 x 4099 bf16 46 us,
// 0.53; 4099 x 2051 fp32 30 us, 0.67; by elements 72 and 32, which matrices that
// lie differently still take).  Tried: blocks of fixed columns shifted out of
// two aligned pieces, 4099 x 2051 fp32 86 us.
// dγ: every thread owns the same columns of all its rows, a CTA's part goes to
// the workspace and a second kernel adds the parts in their order.
#include <cstdint>

#include "row_grid.h"
#include "rows.cuh"

namespace ddp {
namespace {

constexpr int kNormThreads = 256;

struct NormParams {
    const void* x;
    const void* res;
    const float* gamma;
    void* h;
    void* y;        // fp32 / bf16, or int8
    float* scale;   // 8-bit output only
    float* rstd;
    int64_t ldx, ldr, ldh, ldy, rows;
    int32_t D;
    float eps;
};

enum { kOutF32 = 0, kOutBf16 = 1, kOutQ8 = 2 };

// A CTA per row (grid-stride), two passes over the row; every element is read
// and written by the same thread, so y and h may lie on x or residual.
template <bool BF16, int OUT>
__global__ void __launch_bounds__(kNormThreads) norm_loop_kernel(const __grid_constant__ NormParams a) {
    __shared__ float sh[32];
    pdl_enter();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const void* x = row_ptr<BF16>(a.x, row, a.ldx);
        const void* r = a.res ? row_ptr<BF16>(a.res, row, a.ldr) : nullptr;
        float ss = 0.0f, mx = 0.0f;
        for (int d = threadIdx.x; d < a.D; d += kNormThreads) {
            float h = load_elem<BF16>(x, d);
            if (r) h += load_elem<BF16>(r, d);
            ss = fmaf(h, h, ss);
            if constexpr (OUT == kOutQ8) mx = max_nan(mx, fabsf(a.gamma ? h * a.gamma[d] : h));
        }
        ss = block_all<SumOp>(ss, sh);
        const float rstd = 1.0f / sqrtf(ss / a.D + a.eps);
        float inv = 0.0f, up = 1.0f;
        if constexpr (OUT == kOutQ8) {
            mx = block_all<MaxNanOp>(mx, sh);
            // a row of zeros has the scale 0; one that is not finite has a scale that is not, and zeros
            const float sc = mx * rstd / 127.0f;
            up = mx < 1.0e-30f ? 0x1p64f : 1.0f;         // 127 / mx would overflow
            inv = sc > 0.0f && sc < INFINITY ? 127.0f / (mx * up) : 0.0f;
            if (threadIdx.x == 0) a.scale[row] = sc;
        }
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
        for (int d = threadIdx.x; d < a.D; d += kNormThreads) {
            float h = load_elem<BF16>(x, d);
            if (r) h += load_elem<BF16>(r, d);
            const float hg = a.gamma ? h * a.gamma[d] : h;
            if (a.h) store_elem<BF16>(row_ptr<BF16>(a.h, row, a.ldh), d, h);
            if constexpr (OUT == kOutQ8) {
                const float q = rintf(hg * up * inv);
                static_cast<int8_t*>(a.y)[row * a.ldy + d] = static_cast<int8_t>(inv > 0.0f ? q : 0.0f);
            } else {
                store_elem<OUT == kOutBf16>(row_ptr<OUT == kOutBf16>(a.y, row, a.ldy), d, hg * rstd);
            }
        }
    }
}

// What one thread holds of a row: vectors threadIdx-strided, one element at the row's ends.
struct RowShape {
    int lead, nvec, edges;
};
template <bool BF16, bool EDGE>
__device__ __forceinline__ RowShape row_shape(const char* p, int D) {
    constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES;
    RowShape s{0, D / VEC, 0};
    if constexpr (EDGE) {
        s.lead = min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / ES, D);
        s.nvec = (D - s.lead) / VEC;
        s.edges = D - s.nvec * VEC;
    }
    return s;
}
template <int VEC>
__device__ __forceinline__ int edge_elem(const RowShape& s, int e) {
    return e < s.lead ? e : e + s.nvec * VEC;
}

// N consecutive values of a matrix, N·size a power of two up to 32 bytes and p aligned to it (or to 16).
template <bool BF16, int N>
__device__ __forceinline__ void load_n(const char* p, float (&o)[N]) {
    if constexpr (!BF16) {
#pragma unroll
        for (int q = 0; q < N / 4; ++q) {
            const uint4 v = ld16<false>(p + 16 * q);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[4 * q + e] = vec_elem<false>(v, e);
        }
    } else if constexpr (N == 8) {
        const uint4 v = ld16<false>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = vec_elem<true>(v, e);
    } else {
        uint2 v;
        asm volatile("ld.global.cs.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
        o[0] = bf16_lo(v.x);
        o[1] = bf16_hi(v.x);
        o[2] = bf16_lo(v.y);
        o[3] = bf16_hi(v.y);
    }
}
template <bool BF16, int N>
__device__ __forceinline__ void store_n(char* p, const float (&o)[N]) {
    if constexpr (!BF16) {
#pragma unroll
        for (int q = 0; q < N / 4; ++q) *reinterpret_cast<float4*>(p + 16 * q) = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
    } else if constexpr (N == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
    } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    }
}
// γ of VEC columns from d on (1 without γ).  EDGE: d is any column, the same
// modulo 4 for a row's vectors; the 16-byte pieces that cover them, shifted
// (one 4-byte load per column instead cost 8 passes of 32 sectors per warp).
template <bool EDGE, int VEC>
__device__ __forceinline__ void load_gamma(const float* gamma, int D, int d, float (&o)[VEC]) {
    if (gamma == nullptr) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = 1.0f;
        return;
    }
    const int s = EDGE ? (d + static_cast<int>(reinterpret_cast<uintptr_t>(gamma) / 4)) & 3 : 0, b = d - s;
    if (EDGE && (b < 0 || b + VEC + 4 > D)) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = __ldg(gamma + d + e);
        return;
    }
    float f[VEC + 4];
#pragma unroll
    for (int q = 0; q < VEC / 4 + (EDGE ? 1 : 0); ++q) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(gamma + b) + q);
        f[4 * q] = v.x;
        f[4 * q + 1] = v.y;
        f[4 * q + 2] = v.z;
        f[4 * q + 3] = v.w;
    }
    if constexpr (EDGE) {
#pragma unroll
        for (int e = 0; e < VEC + 3; ++e) f[e] = s & 1 ? f[e + 1] : f[e];
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = s & 2 ? f[e + 2] : f[e];
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = f[e];
}

constexpr int kWarpRows = 8;      // rows per CTA of the warp-per-row forward kernels
constexpr int max_group(bool bf16, int vpt) { return vpt * (bf16 ? 8 : 4) > 16 ? 512 : 1024; }

// Forward: VPT vectors per thread.  WARP: a warp per row, kWarpRows per CTA; else a CTA per row.
template <bool BF16, int OUT, int VPT, bool EDGE, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : max_group(BF16, VPT))
    norm_kernel(const __grid_constant__ NormParams a) {
    constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES, YS = OUT == kOutQ8 ? 1 : OUT == kOutBf16 ? 2 : 4;
    __shared__ float2 sh[32];
    pdl_enter();
    const int G = WARP ? 32 : blockDim.x;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.rows) return;       // whole warps
    const char* x = row_ptr<BF16>(a.x, row, a.ldx);
    const char* r = a.res ? row_ptr<BF16>(a.res, row, a.ldr) : nullptr;
    const RowShape s = row_shape<BF16, EDGE>(x, a.D);
    float h[VPT][VEC], he = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = t + i * G;
        if (v < s.nvec) load_n<BF16, VEC>(x + (s.lead + v * VEC) * ES, h[i]);
        else
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[i][e] = 0.0f;
    }
    if (r != nullptr) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + i * G;
            if (v >= s.nvec) break;
            float rr[VEC];
            load_n<BF16, VEC>(r + (s.lead + v * VEC) * ES, rr);
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[i][e] += rr[e];
        }
    }
    // the last warp has the fewest vectors: elsewhere the ends would cost the row a second memory latency
    const int te = G - 1 - t;
    const bool has_edge = EDGE && te < s.edges;
    const int de = EDGE ? edge_elem<VEC>(s, te) : 0;
    if (has_edge) he = load_elem<BF16>(x, de) + (r ? load_elem<BF16>(r, de) : 0.0f);
    float ss = he * he, mx = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = fmaf(h[i][e], h[i][e], ss);
    if (a.h != nullptr) {
        char* ho = row_ptr<BF16>(a.h, row, a.ldh);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + i * G;
            if (v < s.nvec) store_n<BF16, VEC>(ho + (s.lead + v * VEC) * ES, h[i]);
        }
        if (has_edge) store_elem<BF16>(ho, de, he);
    }
    // h·γ
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = t + i * G;
        if (v >= s.nvec) break;
        float g[VEC];
        load_gamma<EDGE, VEC>(a.gamma, a.D, s.lead + v * VEC, g);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            h[i][e] *= g[e];
            if constexpr (OUT == kOutQ8) mx = max_nan(mx, fabsf(h[i][e]));
        }
    }
    if (has_edge) {
        he = a.gamma ? he * a.gamma[de] : he;
        if constexpr (OUT == kOutQ8) mx = max_nan(mx, fabsf(he));
    }
    if constexpr (OUT == kOutQ8) {
        if constexpr (WARP) ss = warp_all<SumOp>(ss), mx = warp_all<MaxNanOp>(mx);
        else block_all2<SumOp, MaxNanOp>(ss, mx, sh);
    } else {
        ss = WARP ? warp_all<SumOp>(ss) : block_all<SumOp>(ss, reinterpret_cast<float*>(sh));
    }
    const float rstd = 1.0f / sqrtf(ss / a.D + a.eps);
    if (t == 0 && a.rstd) a.rstd[row] = rstd;
    if constexpr (OUT == kOutQ8) {
        const float sc = mx * rstd / 127.0f;
        if (t == 0) a.scale[row] = sc;
        const bool some = sc > 0.0f && sc < INFINITY;
        if (mx < 1.0e-30f) {             // 127 / mx would overflow
            mx *= 0x1p64f;
            he *= 0x1p64f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) h[i][e] *= 0x1p64f;
        }
        // q = y / sc = (h·γ)·127 / max|h·γ|.  The product is at most 127 up to rounding, so that adding 1.5·2^23 leaves
        // the nearest integer (ties to even) in the low byte, with one rounding and no conversion instruction (those
        // run at a quarter of the rate: 16384 x 4096 bf16 92 -> 89 us).
        constexpr float kMagic = 12582912.0f;
        const float inv = 127.0f / mx;
        auto quant = [&](float v) { return some ? __float_as_uint(fmaf(v, inv, kMagic)) : 0u; };
        char* y = static_cast<char*>(a.y) + row * a.ldy;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + i * G;
            if (v >= s.nvec) break;
            uint32_t w[VEC / 4];
#pragma unroll
            for (int q = 0; q < VEC / 4; ++q)
                w[q] = __byte_perm(__byte_perm(quant(h[i][4 * q]), quant(h[i][4 * q + 1]), 0x0040),
                                   __byte_perm(quant(h[i][4 * q + 2]), quant(h[i][4 * q + 3]), 0x0040), 0x5410);
            char* d = y + s.lead + v * VEC;
            if constexpr (VEC == 8) *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[VEC / 4 - 1]);
            else *reinterpret_cast<uint32_t*>(d) = w[0];
        }
        if (has_edge) y[de] = static_cast<char>(quant(he) & 0xffu);
    } else {
        char* y = row_ptr<OUT == kOutBf16>(a.y, row, a.ldy);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + i * G;
            if (v >= s.nvec) break;
            float o[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = h[i][e] * rstd;
            store_n<OUT == kOutBf16, VEC>(y + (s.lead + v * VEC) * YS, o);
        }
        if (has_edge) store_elem<OUT == kOutBf16>(y, de, he * rstd);
    }
}

struct NormGradParams {
    const void* dy;
    const void* h;
    const float* rstd;
    const float* gamma;
    const void* dh;
    void* dx;
    float* partial;   // [gridDim.x][D] or NULL
    int64_t lddy, ldh, lddh, lddx, rows;
    int32_t D;
};

// A CTA per row (grid-stride); each thread owns the same columns of every
// row, so its CTA's part of dγ needs no atomics: it is kept in the workspace.
template <bool BF16, bool DYBF16>
__global__ void __launch_bounds__(kNormThreads) norm_grad_loop_kernel(const __grid_constant__ NormGradParams a) {
    __shared__ float sh[32];
    pdl_enter();
    float* part = a.partial ? a.partial + static_cast<int64_t>(blockIdx.x) * a.D : nullptr;
    bool first = true;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, first = false) {
        const void* dy = row_ptr<DYBF16>(a.dy, row, a.lddy);
        const void* hp = row_ptr<BF16>(a.h, row, a.ldh);
        const void* dh = a.dh ? row_ptr<BF16>(a.dh, row, a.lddh) : nullptr;
        void* dx = row_ptr<BF16>(a.dx, row, a.lddx);
        const float rstd = a.rstd[row];
        float s = 0.0f;
        for (int d = threadIdx.x; d < a.D; d += kNormThreads) {
            const float g = load_elem<DYBF16>(dy, d), n = load_elem<BF16>(hp, d) * rstd;
            s = fmaf(a.gamma ? g * a.gamma[d] : g, n, s);
        }
        const float c = block_all<SumOp>(s, sh) / a.D;
        for (int d = threadIdx.x; d < a.D; d += kNormThreads) {
            const float g = load_elem<DYBF16>(dy, d), n = load_elem<BF16>(hp, d) * rstd;
            float v = rstd * ((a.gamma ? g * a.gamma[d] : g) - n * c);
            if (dh) v += load_elem<BF16>(dh, d);
            store_elem<BF16>(dx, d, v);
            if (part) part[d] = first ? g * n : fmaf(g, n, part[d]);
        }
    }
}

// N values of a matrix as they lie in memory.
template <bool BF16, int N>
struct Packed {
    static constexpr int W = N * (BF16 ? 2 : 4) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const char* p) {
        if constexpr (W == 2) {
            asm volatile("ld.global.cs.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p) : "memory");
        } else {
#pragma unroll
            for (int q = 0; q < W / 4; ++q) {
                const uint4 v = ld16<false>(p + 16 * q);
                w[4 * q] = v.x;
                w[4 * q + 1] = v.y;
                w[4 * q + 2] = v.z;
                w[4 * q + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float at(int e) const {
        if constexpr (BF16) return e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
        else return __uint_as_float(w[e]);
    }
};

// Backward, aligned rows, grid-stride: a row's dy, h and dh are all on their
// way before the first is used, and stay packed in registers.  A thread's
// columns are the same for every row, so its part of dγ is in registers too.
// AHEAD: the next row is fetched before this one is reduced.  EDGE: rows off
// the 16-byte boundaries that lie alike; the grid is a multiple of VEC, so a
// thread's columns still do not change from row to row.
// Rows per CTA of the warp-per-row kernel: one CTA per SM, so that dγ has few
// parts and a warp has 128 registers (8192 x 768 bf16: 13.9 us with 16 warps, 14.6 with 8 and two CTAs per SM, 16.0 with
// 4 and four; three CTAs of 8 spill).
constexpr int kGradRows = 16;

template <bool BF16, bool DYBF16, int VPT, bool WARP, bool AHEAD, bool EDGE>
__global__ void __launch_bounds__(WARP ? 32 * kGradRows : AHEAD ? 512 : max_group(BF16, VPT))
    norm_grad_kernel(const __grid_constant__ NormGradParams a) {
    constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES, YS = DYBF16 ? 2 : 4;
    extern __shared__ float part_sh[];   // WARP and a.partial: [kGradRows][D]
    __shared__ float sh[32];
    pdl_enter();
    const int G = WARP ? 32 : blockDim.x;
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int w = WARP ? threadIdx.x >> 5 : 0;
    const bool want = a.partial != nullptr;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * (WARP ? kGradRows : 1) + w;
    const RowShape s = row_shape<BF16, EDGE>(row_ptr<BF16>(a.h, row0, a.ldh), a.D);
    const int te = G - 1 - t, de = EDGE ? edge_elem<VEC>(s, te) : 0;
    const bool has_edge = EDGE && te < s.edges;
    const float gme = has_edge && a.gamma ? __ldg(a.gamma + de) : 1.0f;
    float acc[VPT][VEC] = {}, acc_e = 0.0f, ge = 0.0f, he = 0.0f, re = 0.0f, ge2 = 0.0f, he2 = 0.0f, re2 = 0.0f;
    float gk[EDGE && !WARP ? VPT : 1][VEC];          // γ of the thread's columns, where there is room for it
    auto gamma_of = [&](int i, int v, float (&gm)[VEC]) {
        if constexpr (EDGE && !WARP) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) gm[e] = gk[i][e];
        } else {
            load_gamma<EDGE, VEC>(a.gamma, a.D, s.lead + v * VEC, gm);
        }
    };
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (WARP ? kGradRows : 1);
    Packed<DYBF16, VEC> g[VPT], g2[AHEAD ? VPT : 1];
    Packed<BF16, VEC> h[VPT], r[VPT], h2[AHEAD ? VPT : 1], r2[AHEAD ? VPT : 1];
    float rstd = 0.0f, rstd2 = 0.0f;
    auto fetch = [&](int64_t row, Packed<DYBF16, VEC>* gg, Packed<BF16, VEC>* hh, Packed<BF16, VEC>* rr, float& rs, float& eg, float& eh, float& er) {
        const char* dy = row_ptr<DYBF16>(a.dy, row, a.lddy);
        const char* hp = row_ptr<BF16>(a.h, row, a.ldh);
        const char* dh = a.dh ? row_ptr<BF16>(a.dh, row, a.lddh) : nullptr;
        rs = a.rstd[row];
        if (has_edge) {
            eg = load_elem<DYBF16>(dy, de);
            eh = load_elem<BF16>(hp, de);
            if (dh) er = load_elem<BF16>(dh, de);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + i * G;
            if (v < s.nvec) {
                gg[i].load(dy + (s.lead + v * VEC) * YS);
                hh[i].load(hp + (s.lead + v * VEC) * ES);
                if (dh) rr[i].load(dh + (s.lead + v * VEC) * ES);
                else rr[i].zero();
            }
        }
    };
    int64_t row = row0;
    if (AHEAD && row < a.rows) fetch(row, g, h, r, rstd, ge, he, re);
    for (; row < a.rows; row += stride) {
        if constexpr (AHEAD) {
            if (row + stride < a.rows) fetch(row + stride, g2, h2, r2, rstd2, ge2, he2, re2);
        } else {
            fetch(row, g, h, r, rstd, ge, he, re);
        }
        if constexpr (EDGE && !WARP) {
            if (row == row0) {                       // behind the first row's loads
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (t + i * G < s.nvec) load_gamma<true, VEC>(a.gamma, a.D, s.lead + (t + i * G) * VEC, gk[i]);
            }
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + i * G;
            if (v >= s.nvec) break;
            float gm[VEC];
            gamma_of(i, v, gm);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float gn = g[i].at(e) * (h[i].at(e) * rstd);
                acc[i][e] += gn;
                sum = fmaf(gn, gm[e], sum);
            }
        }
        if constexpr (EDGE) {
            const float gn = ge * (he * rstd);
            acc_e += gn;
            sum = fmaf(gn, gme, sum);
        }
        const float c = (WARP ? warp_all<SumOp>(sum) : block_all<SumOp>(sum, sh)) / a.D;
        char* dx = row_ptr<BF16>(a.dx, row, a.lddx);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = t + i * G;
            if (v >= s.nvec) break;
            float gm[VEC], o[VEC];
            gamma_of(i, v, gm);
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = fmaf(rstd, g[i].at(e) * gm[e] - h[i].at(e) * rstd * c, r[i].at(e));
            store_n<BF16, VEC>(dx + (s.lead + v * VEC) * ES, o);
        }
        if (has_edge) store_elem<BF16>(dx, de, fmaf(rstd, ge * gme - he * rstd * c, re));
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                g[i] = g2[i];
                h[i] = h2[i];
                r[i] = r2[i];
            }
            rstd = rstd2;
            ge = ge2;
            he = he2;
            re = re2;
        }
    }
    if (!want) return;
    float* out = a.partial + static_cast<int64_t>(blockIdx.x) * a.D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = t + i * G;
        if (v >= s.nvec) break;
        float* d = (WARP ? part_sh + w * a.D : out) + s.lead + v * VEC;
        if constexpr (EDGE) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) d[e] = acc[i][e];
        } else {
#pragma unroll
            for (int q = 0; q < VEC / 4; ++q)
                reinterpret_cast<float4*>(d)[q] = make_float4(acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]);
        }
    }
    if (has_edge) ((WARP ? part_sh + w * a.D : out))[de] = acc_e;
    if constexpr (WARP) {
        __syncthreads();
        for (int d = threadIdx.x; d < a.D; d += 32 * kGradRows) {
            float v = part_sh[d];
#pragma unroll
            for (int i = 1; i < kGradRows; ++i) v += part_sh[i * a.D + d];
            out[d] = v;
        }
    }
}

// Backward, rows that lie anywhere: an element at a time, each thread the
// same EPT columns of every row (γ and its part of dγ in registers), G threads.
template <bool BF16, bool DYBF16, int G, int EPT>
__global__ void __launch_bounds__(G, G * EPT <= 512 ? 1024 / G : G <= 512 ? (EPT <= 4 ? 3 : 2) : 1)
    norm_grad_elem_kernel(const __grid_constant__ NormGradParams a) {
    constexpr int ES = BF16 ? 2 : 4, YS = DYBF16 ? 2 : 4;
    __shared__ float sh[32];
    pdl_enter();
    const int t = threadIdx.x;
    float acc[EPT] = {}, gm[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) gm[i] = t + i * G < a.D && a.gamma ? __ldg(a.gamma + t + i * G) : 1.0f;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char* dy = row_ptr<DYBF16>(a.dy, row, a.lddy) + t * YS;
        const char* hp = row_ptr<BF16>(a.h, row, a.ldh) + t * ES;
        const char* dh = row_ptr<BF16>(a.dh, row, a.lddh) + t * ES;
        float g[EPT], n[EPT], r[EPT];
        const float rstd = a.rstd[row];
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const bool in = t + i * G < a.D;
            g[i] = in ? load_elem<DYBF16>(dy + i * G * YS, 0) : 0.0f;
            n[i] = in ? load_elem<BF16>(hp + i * G * ES, 0) : 0.0f;
            r[i] = in && a.dh ? load_elem<BF16>(dh + i * G * ES, 0) : 0.0f;
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            n[i] *= rstd;
            acc[i] = fmaf(g[i], n[i], acc[i]);
            g[i] *= gm[i];
            sum = fmaf(g[i], n[i], sum);
        }
        const float c = block_all<SumOp>(sum, sh) / a.D;
        char* dx = row_ptr<BF16>(a.dx, row, a.lddx) + t * ES;
#pragma unroll
        for (int i = 0; i < EPT; ++i)
            if (t + i * G < a.D) store_elem<BF16>(dx + i * G * ES, 0, fmaf(rstd, g[i] - n[i] * c, r[i]));
    }
    if (a.partial == nullptr) return;
#pragma unroll
    for (int i = 0; i < EPT; ++i)
        if (t + i * G < a.D) a.partial[static_cast<int64_t>(blockIdx.x) * a.D + t + i * G] = acc[i];
}

struct GammaParams {
    const float* partial;
    float* dgamma;
    int32_t n, D;
};

// dγ[d] = Σ over the CTAs' parts, in a fixed order: 16 columns per CTA, 64
// threads per column over interleaved parts, then those 64 by halves.
__global__ void __launch_bounds__(1024) norm_gamma_kernel(const __grid_constant__ GammaParams a) {
    __shared__ float sh[64][17];
    pdl_enter();
    const int c = threadIdx.x & 15, w = threadIdx.x >> 4;
    const int d = blockIdx.x * 16 + c;
    float s = 0.0f;
    if (d < a.D) {
#pragma unroll 10
        for (int i = w; i < a.n; i += 64) s += a.partial[static_cast<int64_t>(i) * a.D + d];
    }
    sh[w][c] = s;
    __syncthreads();
    if (threadIdx.x >= 512) return;
    const int col = threadIdx.x >> 5, l = threadIdx.x & 31;      // a warp per column
    s = warp_all<SumOp>(sh[l][col] + sh[l + 32][col]);
    if (l == 0 && blockIdx.x * 16 + col < a.D) a.dgamma[blockIdx.x * 16 + col] = s;
}

constexpr int kGradCtas = 608;   // at most this many parts of dγ

int grad_parts(int64_t rows) { return static_cast<int>(rows < kGradCtas ? (rows < 1 ? 1 : rows) : kGradCtas); }

bool dtype_ok(int32_t t) { return t == DDP_F32 || t == DDP_BF16; }
int dsize(int32_t t) { return t == DDP_BF16 ? 2 : 4; }

// How the rows of a call's matrices lie on the grid of VEC elements (16 bytes of x's type).
enum class Lay { kAligned, kAlike, kDifferent };
Lay layout(const Mat* const* mats, int n, int D, int vec, const float* gamma) {
    bool aligned = D % vec == 0 && aligned16(gamma), alike = true;
    for (int i = 0; i < n; ++i) {
        const Mat &m = *mats[i], &f = *mats[0];
        if (m.p == nullptr) continue;
        const uintptr_t e = reinterpret_cast<uintptr_t>(m.p) / m.esz, e0 = reinterpret_cast<uintptr_t>(f.p) / f.esz;
        const bool one = m.rows <= 1;
        alike &= e % vec == e0 % vec && (one || m.ld % vec == f.ld % vec);
        aligned &= e % vec == 0 && (one || m.ld % vec == 0);
    }
    return aligned ? Lay::kAligned : alike ? Lay::kAlike : Lay::kDifferent;
}

// Vectors per thread and threads per row.  Many rows: a warp per row up to 128
// vectors, then two vectors per thread; few rows (they do not fill the GPU):
// as many threads as the row has vectors.  0 threads: the row does not fit.
struct Group {
    int vpt, threads;
    bool warp;
};
Group pick_group(int64_t rows, int D, bool bf16, int sms) {
    const int vec = bf16 ? 8 : 4, nv = (D + vec - 1) / vec;
    if (nv <= 32) return {1, 32, true};
    const bool few = rows < 2ll * sms;
    if (!few && nv <= 128) return {(nv + 31) / 32, 32, true};
    for (int vpt = few ? 1 : 2; vpt <= 4; vpt *= 2) {
        const int t = ((nv + vpt - 1) / vpt + 31) / 32 * 32;
        if (t <= max_group(bf16, vpt)) return {vpt, t, false};
    }
    return {0, 0, false};
}

template <bool BF16, int OUT, bool EDGE>
void (*fwd_kernel(const Group& g))(NormParams) {
    if (g.warp) return g.vpt == 1 ? norm_kernel<BF16, OUT, 1, EDGE, true> : g.vpt == 2 ? norm_kernel<BF16, OUT, 2, EDGE, true> : g.vpt == 3 ? norm_kernel<BF16, OUT, 3, EDGE, true> : norm_kernel<BF16, OUT, 4, EDGE, true>;
    return g.vpt == 1 ? norm_kernel<BF16, OUT, 1, EDGE, false> : g.vpt == 2 ? norm_kernel<BF16, OUT, 2, EDGE, false> : norm_kernel<BF16, OUT, 4, EDGE, false>;
}
template <bool BF16, int OUT>
void (*fwd_kernel(Lay lay, const Group& g))(NormParams) {
    if (lay == Lay::kDifferent || g.threads == 0) return norm_loop_kernel<BF16, OUT>;
    return lay == Lay::kAligned ? fwd_kernel<BF16, OUT, false>(g) : fwd_kernel<BF16, OUT, true>(g);
}
template <bool BF16, bool DYBF16, bool EDGE>
void (*bwd_vec(const Group& g))(NormGradParams) {
    if (g.warp) return g.vpt == 1 ? norm_grad_kernel<BF16, DYBF16, 1, true, false, EDGE> : g.vpt == 2 ? norm_grad_kernel<BF16, DYBF16, 2, true, false, EDGE> : g.vpt == 3 ? norm_grad_kernel<BF16, DYBF16, 3, true, false, EDGE> : norm_grad_kernel<BF16, DYBF16, 4, true, false, EDGE>;
    // fetching ahead needs more than 64 registers: 8192 x 4096 bf16 at 52 us with it, 53 without; off the boundaries
    // 5000 x 4099 bf16 71 with it, 46 without
    if (g.threads <= 512 && g.vpt <= 2) return g.vpt == 1 ? norm_grad_kernel<BF16, DYBF16, 1, false, !EDGE, EDGE> : norm_grad_kernel<BF16, DYBF16, 2, false, !EDGE, EDGE>;
    return g.vpt == 1 ? norm_grad_kernel<BF16, DYBF16, 1, false, false, EDGE> : g.vpt == 2 ? norm_grad_kernel<BF16, DYBF16, 2, false, false, EDGE> : norm_grad_kernel<BF16, DYBF16, 4, false, false, EDGE>;
}

// Element kernels by width: threads, kernel.
template <bool BF16, bool DYBF16>
int bwd_elem(int D, void (**k)(NormGradParams)) {
    if (D <= 128) return *k = norm_grad_elem_kernel<BF16, DYBF16, 128, 1>, 128;
    if (D <= 512) return *k = norm_grad_elem_kernel<BF16, DYBF16, 128, 4>, 128;
    if (D <= 1024) return *k = norm_grad_elem_kernel<BF16, DYBF16, 256, 4>, 256;
    if (D <= 2048) return *k = norm_grad_elem_kernel<BF16, DYBF16, 512, 4>, 512;
    if (D <= 512 * 6) return *k = norm_grad_elem_kernel<BF16, DYBF16, 512, 6>, 512;
    if (D <= 4608) return *k = norm_grad_elem_kernel<BF16, DYBF16, 512, 9>, 512;
    if (D <= 8192) return *k = norm_grad_elem_kernel<BF16, DYBF16, 1024, 8>, 1024;
    return *k = norm_grad_loop_kernel<BF16, DYBF16>, kNormThreads;
}

// How rmsnorm_backward runs: kernel, threads, CTAs, shared memory.
struct GradPlan {
    void (*kernel)(NormGradParams);
    int threads, ctas;
    size_t smem;
};
template <bool BF16, bool DYBF16>
int grad_plan(Lay lay, int64_t rows, int D, bool want, int sms, GradPlan* p) {
    const Group g = pick_group(rows, D, BF16, sms);
    int64_t rows_per_cta = 1;
    p->smem = 0;
    const bool vec = lay != Lay::kDifferent && g.threads != 0;
    if (vec) {
        p->kernel = lay == Lay::kAligned ? bwd_vec<BF16, DYBF16, false>(g) : bwd_vec<BF16, DYBF16, true>(g);
        p->threads = g.warp ? 32 * kGradRows : g.threads;
        rows_per_cta = g.warp ? kGradRows : 1;
        p->smem = g.warp && want ? static_cast<size_t>(kGradRows) * D * 4 : 0;
    } else {
        p->threads = bwd_elem<BF16, DYBF16>(D, &p->kernel);
    }
    // one wave, and few enough parts of dγ
    const int64_t ctas = (rows + rows_per_cta - 1) / rows_per_cta;
    const int st = one_wave_grid(reinterpret_cast<const void*>(p->kernel), p->threads, ctas, &p->ctas);
    if (p->ctas > kGradCtas) p->ctas = kGradCtas;
    if (vec && lay == Lay::kAlike) p->ctas = alike_grid(p->ctas, ctas);
    return st;
}

int forward(const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t in_dtype, const float* gamma,
            int64_t rows, int32_t D, float eps, void* h_out, int64_t ldh, void* y, int64_t ldy, int out,
            float* scale, float* rstd_out, void* stream) {
    if (!dtype_ok(in_dtype) || rows < 0 || D < 1 || !(eps >= 0.0f) || !(eps < 3.0e38f)) return DDP_ERR_INVALID_ARG;
    if (D > kMaxWidth) return DDP_ERR_UNSUPPORTED;
    const int es = dsize(in_dtype), ys = out == kOutQ8 ? 1 : out == kOutBf16 ? 2 : 4;
    const Mat mx{x, rows, D, ldx, es}, mr{residual, rows, D, ldr, es}, mh{h_out, rows, D, ldh, es},
        my{y, rows, D, ldy, ys}, mg{gamma, 1, D, D, 4}, ms{scale, 1, rows, rows, 4}, mt{rstd_out, 1, rows, rows, 4};
    if (!mat_valid(mx) || !mat_valid(my) || (residual && !mat_valid(mr)) || (h_out && !mat_valid(mh)))
        return DDP_ERR_INVALID_ARG;
    if (rows > 0 && (x == nullptr || y == nullptr || (out == kOutQ8 && scale == nullptr))) return DDP_ERR_INVALID_ARG;
    for (const Mat* m : {&mx, &mr, &mh, &my, &mg, &ms, &mt})
        if (!mat_aligned(*m)) return DDP_ERR_ALIGNMENT;
    for (const Mat* o : {&my, &mh}) {
        for (const Mat* i : {&mx, &mr})
            if (!mats_same(*o, *i) && mats_overlap(*o, *i)) return DDP_ERR_INVALID_ARG;
        for (const Mat* i : {&mg, &ms, &mt})
            if (mats_overlap(*o, *i)) return DDP_ERR_INVALID_ARG;
    }
    if (mats_overlap(my, mh) || mats_overlap(ms, mt)) return DDP_ERR_INVALID_ARG;
    for (const Mat* o : {&ms, &mt})
        for (const Mat* i : {&mx, &mr, &mg})
            if (mats_overlap(*o, *i)) return DDP_ERR_INVALID_ARG;
    if (rows == 0) return DDP_OK;
    const NormParams p{x, residual, gamma, h_out, y, scale, rstd_out, ldx, ldr, ldh, ldy, rows, D, eps};
    DeviceInfo d;
    const int st = current_device_info(&d);
    if (st != DDP_OK) return st;
    const bool b = in_dtype == DDP_BF16;
    const Mat* const mats[4] = {&mx, &mr, &mh, &my};
    const Lay lay = layout(mats, 4, D, b ? 8 : 4, gamma);
    const Group g = pick_group(rows, D, b, d.sm_count);
    void (*kernel)(NormParams) = out == kOutQ8    ? (b ? fwd_kernel<true, kOutQ8>(lay, g) : fwd_kernel<false, kOutQ8>(lay, g))
                                 : out == kOutBf16 ? (b ? fwd_kernel<true, kOutBf16>(lay, g) : fwd_kernel<false, kOutBf16>(lay, g))
                                                   : (b ? fwd_kernel<true, kOutF32>(lay, g) : fwd_kernel<false, kOutF32>(lay, g));
    const bool loop = lay == Lay::kDifferent || g.threads == 0;
    const int64_t ctas = loop ? (rows < (1 << 16) ? rows : 1 << 16) : g.warp ? (rows + kWarpRows - 1) / kWarpRows : rows;
    if (ctas > INT32_MAX) return DDP_ERR_UNSUPPORTED;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), loop ? kNormThreads : g.warp ? 32 * kWarpRows : g.threads,
                      static_cast<cudaStream_t>(stream), p);
}

}  // namespace
}  // namespace ddp

using namespace ddp;

extern "C" int rmsnorm_forward(const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t in_dtype,
                               const float* gamma, int64_t rows, int32_t D, float eps, void* h_out, int64_t ldh,
                               void* y, int64_t ldy, int32_t out_dtype, float* rstd_out, void* stream) {
    if (!dtype_ok(out_dtype)) return DDP_ERR_INVALID_ARG;
    return forward(x, ldx, residual, ldr, in_dtype, gamma, rows, D, eps, h_out, ldh, y, ldy,
                   out_dtype == DDP_BF16 ? kOutBf16 : kOutF32, nullptr, rstd_out, stream);
}

extern "C" int rmsnorm_forward_q8(const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t in_dtype,
                                  const float* gamma, int64_t rows, int32_t D, float eps, void* h_out, int64_t ldh,
                                  int8_t* q, int64_t ldq, float* scale, float* rstd_out, void* stream) {
    return forward(x, ldx, residual, ldr, in_dtype, gamma, rows, D, eps, h_out, ldh, q, ldq, kOutQ8, scale, rstd_out,
                   stream);
}

extern "C" size_t rmsnorm_backward_workspace_bytes(int64_t rows, int32_t D) {
    return rows < 0 || D < 1 || D > kMaxWidth ? 0 : static_cast<size_t>(grad_parts(rows)) * static_cast<size_t>(D) * 4;
}

extern "C" int rmsnorm_backward(const void* dy, int64_t lddy, int32_t dy_dtype, const void* h, int64_t ldh,
                                int32_t h_dtype, const float* rstd, const float* gamma, const void* dh, int64_t lddh,
                                int64_t rows, int32_t D, void* dx, int64_t lddx, float* dgamma, void* workspace,
                                size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dy_dtype) || !dtype_ok(h_dtype) || rows < 0 || D < 1) return DDP_ERR_INVALID_ARG;
    if (D > kMaxWidth) return DDP_ERR_UNSUPPORTED;
    const int es = dsize(h_dtype);
    const size_t need = dgamma ? rmsnorm_backward_workspace_bytes(rows, D) : 0;
    const Mat my{dy, rows, D, lddy, dsize(dy_dtype)}, mh{h, rows, D, ldh, es}, md{dh, rows, D, lddh, es},
        mo{dx, rows, D, lddx, es}, mr{rstd, 1, rows, rows, 4}, mg{gamma, 1, D, D, 4}, mw{dgamma, 1, D, D, 4},
        ws{dgamma ? workspace : nullptr, 1, static_cast<int64_t>(need / 4), static_cast<int64_t>(need / 4), 4};
    if (!mat_valid(my) || !mat_valid(mh) || !mat_valid(mo) || (dh && !mat_valid(md))) return DDP_ERR_INVALID_ARG;
    if (rows > 0 && (dy == nullptr || h == nullptr || rstd == nullptr || dx == nullptr)) return DDP_ERR_INVALID_ARG;
    if (dgamma && workspace == nullptr) return DDP_ERR_INVALID_ARG;
    for (const Mat* m : {&my, &mh, &md, &mo, &mr, &mg, &mw})
        if (!mat_aligned(*m)) return DDP_ERR_ALIGNMENT;
    if (!aligned16(ws.p)) return DDP_ERR_ALIGNMENT;
    if (dgamma && workspace_bytes < need) return DDP_ERR_CAPACITY;
    for (const Mat* i : {&my, &mh, &md})
        if (!mats_same(mo, *i) && mats_overlap(mo, *i)) return DDP_ERR_INVALID_ARG;
    for (const Mat* o : {&mo, &mw, &ws})
        for (const Mat* i : {&mr, &mg})
            if (mats_overlap(*o, *i)) return DDP_ERR_INVALID_ARG;
    for (const Mat* o : {&mw, &ws})
        for (const Mat* i : {&my, &mh, &md, &mo})
            if (mats_overlap(*o, *i)) return DDP_ERR_INVALID_ARG;
    if (mats_overlap(mw, ws)) return DDP_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int parts = 0;
    if (rows > 0) {
        const NormGradParams p{dy, h, rstd, gamma, dh, dx, dgamma ? static_cast<float*>(workspace) : nullptr,
                               lddy, ldh, lddh, lddx, rows, D};
        DeviceInfo d;
        int st = current_device_info(&d);
        if (st != DDP_OK) return st;
        const bool b = h_dtype == DDP_BF16, c = dy_dtype == DDP_BF16;
        const Mat* const mats[4] = {&mh, &my, &md, &mo};
        const Lay lay = layout(mats, 4, D, b ? 8 : 4, gamma);
        const bool want = dgamma != nullptr;
        GradPlan g;
        st = b ? (c ? grad_plan<true, true>(lay, rows, D, want, d.sm_count, &g) : grad_plan<true, false>(lay, rows, D, want, d.sm_count, &g))
               : (c ? grad_plan<false, true>(lay, rows, D, want, d.sm_count, &g) : grad_plan<false, false>(lay, rows, D, want, d.sm_count, &g));
        if (st != DDP_OK) return st;
        parts = g.ctas;
        if ((st = launch_smem(g.kernel, static_cast<unsigned>(g.ctas), g.threads, g.smem, s, p)) != DDP_OK) return st;
    }
    if (dgamma) {
        const GammaParams q{static_cast<const float*>(workspace), dgamma, parts, D};
        return launch_pdl(norm_gamma_kernel, dim3(static_cast<unsigned>((D + 15) / 16)), 1024, s, q);
    }
    return DDP_OK;
}
