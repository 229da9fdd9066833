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
#include <cstdint>

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
        float inv = 0.0f;
        if constexpr (OUT == kOutQ8) {
            mx = block_all<MaxNanOp>(mx, sh);
            // a row of zeros has the scale 0; one that is not finite has a scale that is not, and zeros
            const float sc = mx * rstd / 127.0f;
            inv = sc > 0.0f && sc < INFINITY ? rstd / sc : 0.0f;
            if (threadIdx.x == 0) a.scale[row] = sc;
        }
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
        for (int d = threadIdx.x; d < a.D; d += kNormThreads) {
            float h = load_elem<BF16>(x, d);
            if (r) h += load_elem<BF16>(r, d);
            const float hg = a.gamma ? h * a.gamma[d] : h;
            if (a.h) store_elem<BF16>(row_ptr<BF16>(a.h, row, a.ldh), d, h);
            if constexpr (OUT == kOutQ8) {
                const float q = fminf(fmaxf(rintf(hg * inv), -127.0f), 127.0f);
                static_cast<int8_t*>(a.y)[row * a.ldy + d] = static_cast<int8_t>(inv > 0.0f ? q : 0.0f);
            } else {
                store_elem<OUT == kOutBf16>(row_ptr<OUT == kOutBf16>(a.y, row, a.ldy), d, hg * rstd);
            }
        }
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

struct GammaParams {
    const float* partial;
    float* dgamma;
    int32_t n, D;
};

// dγ[d] = Σ over the CTAs' parts, in their order: 32 columns per CTA, 8
// threads per column over interleaved parts, then those 8 in order.
__global__ void __launch_bounds__(kNormThreads) norm_gamma_kernel(const __grid_constant__ GammaParams a) {
    __shared__ float sh[8][32];
    pdl_enter();
    const int c = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + c;
    float s = 0.0f;
    if (d < a.D)
        for (int i = w; i < a.n; i += 8) s += a.partial[static_cast<int64_t>(i) * a.D + d];
    sh[w][c] = s;
    __syncthreads();
    if (w == 0 && d < a.D) {
        for (int i = 1; i < 8; ++i) s += sh[i][c];
        a.dgamma[d] = s;
    }
}

constexpr int kGradCtas = 608;   // at most this many parts of dγ

int grad_parts(int64_t rows) { return static_cast<int>(rows < kGradCtas ? (rows < 1 ? 1 : rows) : kGradCtas); }

bool dtype_ok(int32_t t) { return t == DDP_F32 || t == DDP_BF16; }
int dsize(int32_t t) { return t == DDP_BF16 ? 2 : 4; }

int forward(const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t in_dtype, const float* gamma,
            int64_t rows, int32_t D, float eps, void* h_out, int64_t ldh, void* y, int64_t ldy, int out,
            float* scale, float* rstd_out, void* stream) {
    if (!dtype_ok(in_dtype) || rows < 0 || D < 1 || !(eps >= 0.0f) || !(eps < 3.0e38f)) return DDP_ERR_INVALID_ARG;
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
    const bool b = in_dtype == DDP_BF16;
    void (*kernel)(NormParams) = out == kOutQ8    ? (b ? norm_loop_kernel<true, kOutQ8> : norm_loop_kernel<false, kOutQ8>)
                                 : out == kOutBf16 ? (b ? norm_loop_kernel<true, kOutBf16> : norm_loop_kernel<false, kOutBf16>)
                                                   : (b ? norm_loop_kernel<true, kOutF32> : norm_loop_kernel<false, kOutF32>);
    const int64_t cap = 1 << 16;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(rows < cap ? rows : cap)), kNormThreads,
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
    return rows < 0 || D < 1 ? 0 : static_cast<size_t>(grad_parts(rows)) * static_cast<size_t>(D) * 4;
}

extern "C" int rmsnorm_backward(const void* dy, int64_t lddy, int32_t dy_dtype, const void* h, int64_t ldh,
                                int32_t h_dtype, const float* rstd, const float* gamma, const void* dh, int64_t lddh,
                                int64_t rows, int32_t D, void* dx, int64_t lddx, float* dgamma, void* workspace,
                                size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dy_dtype) || !dtype_ok(h_dtype) || rows < 0 || D < 1) return DDP_ERR_INVALID_ARG;
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
    const int parts = grad_parts(rows);
    if (rows > 0) {
        const NormGradParams p{dy, h, rstd, gamma, dh, dx, dgamma ? static_cast<float*>(workspace) : nullptr,
                               lddy, ldh, lddh, lddx, rows, D};
        const bool b = h_dtype == DDP_BF16, c = dy_dtype == DDP_BF16;
        void (*kernel)(NormGradParams) = b ? (c ? norm_grad_loop_kernel<true, true> : norm_grad_loop_kernel<true, false>)
                                           : (c ? norm_grad_loop_kernel<false, true> : norm_grad_loop_kernel<false, false>);
        const int st = launch_pdl(kernel, dim3(static_cast<unsigned>(parts)), kNormThreads, s, p);
        if (st != DDP_OK) return st;
    }
    if (dgamma) {
        const GammaParams q{static_cast<const float*>(workspace), dgamma, rows > 0 ? parts : 0, D};
        return launch_pdl(norm_gamma_kernel, dim3(static_cast<unsigned>((D + 31) / 32)), kNormThreads, s, q);
    }
    return DDP_OK;
}
