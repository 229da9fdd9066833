// Shared by the row operators (RMS norm, 8-bit product, distillation loss):
// rows of a strided matrix read and written as fp32, CTA reductions, and the
// host's checks of matrices against one another.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "host_common.h"

namespace ddp {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <bool BF16>
__device__ __forceinline__ void store_elem(void* base, int64_t e, float v) {
    if constexpr (BF16) reinterpret_cast<__nv_bfloat16*>(base)[e] = __float2bfloat16_rn(v);
    else reinterpret_cast<float*>(base)[e] = v;
}

// First byte of row `row` of a matrix with `ld` elements between rows.
template <bool BF16>
__device__ __forceinline__ const char* row_ptr(const void* base, int64_t row, int64_t ld) {
    return static_cast<const char*>(base) + row * ld * (BF16 ? 2 : 4);
}
template <bool BF16>
__device__ __forceinline__ char* row_ptr(void* base, int64_t row, int64_t ld) {
    return static_cast<char*>(base) + row * ld * (BF16 ? 2 : 4);
}

// Two values rounded to bf16 by one instruction, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Pairs of fp32 values in one register pair: one instruction for two multiply-adds or additions.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Sum / maximum over the CTA, in every thread; MaxOp leaves NaN out (its
// callers carry NaN through a sum), MaxNanOp carries it.  `sh` holds one float per
// warp and is free again when the call returns.
struct SumOp {
    __device__ __forceinline__ static float id() { return 0.0f; }
    __device__ __forceinline__ static float f(float a, float b) { return a + b; }
};
struct MaxOp {
    __device__ __forceinline__ static float id() { return -INFINITY; }
    __device__ __forceinline__ static float f(float a, float b) { return fmaxf(a, b); }
};

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
struct MaxNanOp {
    __device__ __forceinline__ static float id() { return -INFINITY; }
    __device__ __forceinline__ static float f(float a, float b) { return max_nan(a, b); }
};

template <class Op>
__device__ __forceinline__ float warp_all(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = Op::f(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

template <class Op>
__device__ __forceinline__ float block_all(float v, float* sh) {
    v = warp_all<Op>(v);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    const int nw = (blockDim.x + 31) >> 5;
    float r = (threadIdx.x & 31) < nw ? sh[threadIdx.x & 31] : Op::id();
    r = warp_all<Op>(r);
    __syncthreads();
    return r;
}

// Two values over the CTA at once, in every thread; `sh`, one pair per warp, as in block_all.
template <class OpA, class OpB>
__device__ __forceinline__ void block_all2(float& a, float& b, float2* sh) {
    a = warp_all<OpA>(a);
    b = warp_all<OpB>(b);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const bool in = (threadIdx.x & 31) < (blockDim.x + 31) >> 5;
    const float2 v = in ? sh[threadIdx.x & 31] : make_float2(OpA::id(), OpB::id());
    a = warp_all<OpA>(v.x);
    b = warp_all<OpB>(v.y);
    __syncthreads();
}

// ---- host: a matrix argument of a call --------------------------------

inline bool dtype_ok(int32_t t) { return t == DDP_F32 || t == DDP_BF16; }
inline int dsize(int32_t t) { return t == DDP_BF16 ? 2 : 4; }

// Columns of a row: their numbers, rounded up to what a CTA takes at a time, fit 32 bits.
constexpr int64_t kMaxWidth = (1ll << 31) - 65536;

struct Mat {
    const void* p;
    int64_t rows, cols, ld;   // ld in elements
    int esz;                  // bytes per element
};

inline bool mat_valid(const Mat& m) {
    return m.rows >= 0 && m.cols >= 0 && (m.rows <= 1 || m.ld >= m.cols) && m.ld >= 0 && m.ld <= INT64_MAX / 64 &&
           (m.rows == 0 || m.ld == 0 || m.rows <= INT64_MAX / 64 / m.ld) && m.cols <= INT64_MAX / 64;
}

inline bool mat_aligned(const Mat& m) { return (reinterpret_cast<uintptr_t>(m.p) & (m.esz - 1)) == 0; }

inline size_t mat_span(const Mat& m) {
    return m.rows <= 0 || m.cols <= 0 ? 0 : static_cast<size_t>(((m.rows - 1) * m.ld + m.cols) * m.esz);
}

// Whether two matrices share a byte.  Two column slices of one buffer
// (the same pitch, disjoint columns) do not; matrices of different pitch
// whose spans meet are taken to.
inline bool mats_overlap(const Mat& a, const Mat& b) {
    if (a.p == nullptr || b.p == nullptr || !overlaps(a.p, mat_span(a), b.p, mat_span(b))) return false;
    const int64_t pitch = a.ld * a.esz;
    if (pitch != b.ld * b.esz || pitch == 0 || a.rows <= 1 || b.rows <= 1) return true;
    const int64_t wa = a.cols * a.esz, wb = b.cols * b.esz;
    const intptr_t d = reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p);
    const int64_t off = ((d % pitch) + pitch) % pitch;   // b's columns start here in a's pitch
    return off < wa || off + wb > pitch;
}

inline bool mats_same(const Mat& a, const Mat& b) {
    return a.p == b.p && a.esz == b.esz && (a.ld == b.ld || a.rows <= 1);
}

// Launch with dynamic shared memory, in clusters where asked, and programmatic stream serialisation allowed (the kernels begin with
// pdl_enter()); the opt-in beyond 48 KB is asked for only where it is needed.
template <typename Params>
int launch_smem(void (*kernel)(Params), unsigned grid, int block, size_t smem, cudaStream_t s, const Params& params,
                unsigned cluster = 1) {
    cudaError_t e;
    if (smem > 48 * 1024 - 1024) {
        // always the most there is: a smaller call of the same kernel on another thread would take back what this one needs
        cudaFuncAttributes f;
        if ((e = cudaFuncGetAttributes(&f, reinterpret_cast<const void*>(kernel))) != cudaSuccess) return cuda_fail(e);
        if (static_cast<size_t>(f.maxDynamicSharedSizeBytes) < smem &&
            (e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      227 * 1024 - static_cast<int>(f.sharedSizeBytes))) != cudaSuccess)
            return cuda_fail(e);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, params)) != cudaSuccess) return cuda_fail(e);
    return check_launch();
}

}  // namespace ddp
