// Orthogonalisation of matrices by Newton-Schulz steps, alone and as the
// optimizer step of a model's matrices behind the replicas' average.
//
//   X = U / (‖U‖ + eps)                    (Frobenius; a tall U transposed: m rows <= n columns)
//   A = X·Xᵀ,  B = bA + cA²,  X ← aX + B·X    `steps` times, (a, b, c) = (3.4445, −4.7750, 2.0315)
//   optimizer: g = average of the replicas, buf ← μ·buf + g, U = g + μ·buf (or buf),
//              θ ← θ·(1 − lr·wd) − lr·scale·X
//
// The polynomial takes singular values between 1e-3 and 1 to about 1; it grows
// small ones by up to 3.4445^steps, and with them whatever X was rounded by.
// Products run in fp16 with fp32 accumulators: 11 bits where bf16 has 8, at the
// same rate.  Nothing leaves fp16's range: X has singular values up to about
// 1.2, and U is stored times a power of two (exact) that brings its entries to
// about 1; the norm's reciprocal is applied to the accumulators.  While more than two
// steps remain X also keeps what fp16 rounded off (a second fp16 number, used
// in aX, through which nearly all of a small singular value passes).  Relative error
// of X (768 x 768, by the 2-norm): 1.3e-3 for a random matrix, 3.5e-4 for singular
// values falling as 1/i, 4e-4 as 1/i²; in bf16 1e-2, 2.7e-2 and 0.16, in fp16
// without the second number 1.2e-3, 3.4e-3 and 2e-2.
//
// Matrices of one shape run together, so that a step of many small ones fills
// the GPU.  A and B are symmetric: tiles on and above the diagonal are
// computed and stored twice, the second time transposed, 3mn·m + m³ operations
// per step instead of 4mn·m + 2m³.
//   update_kernel / square_kernel   average, momentum, U; parts of ‖U‖²
//   split_kernel   ‖U‖ from its parts, U to fp16 (and the rest), transposed where tall
//   step_kernel    persistent tcgen05 tiles, 3 launches per step (Gram matrix,
//                  polynomial, product with X; the last one writes the result): a pair of
//                  CTAs per tile of 256 x 256, or a CTA per tile of 128 x 128 where pairs would leave
//                  SMs without work.  Roles by warp: a TMA producer (64 of K a stage, 128-byte
//                  swizzle, six stages), an issuer of tcgen05.mma, eight
//                  epilogue warps; two accumulators in TMEM, so that a tile's
//                  epilogue runs under the next one's products.
// Every wait on a barrier is bounded; a tile whose wait ran out is written as NaN.
#include <algorithm>
#include <cstdint>

#include <cuda_fp16.h>

#include "tile.cuh"

namespace ddp {
namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr int kGroup = DDP_NS_GROUP;   // matrices per launch
constexpr int kMaxSide = 65536;
constexpr int kMaxSteps = 16;
constexpr int kPad = 64;               // sides are padded to blocks of K
constexpr int kParts = 1024;           // of a matrix's ‖U‖², at most
constexpr int kPartElems = 8192;       // a part has at least so many elements
constexpr int kMaxReplicas = 16;

// ---- average, momentum, sums of squares ------------------------------------

struct UpdateParams {
    const void* replica[kMaxReplicas];
    int64_t offset[kGroup];
    float* buf;
    float* u;              // [count][pitch]
    float* part;           // [count][kParts]
    int64_t size, pitch, per;   // per: elements per part, a multiple of 8
    float inv_n, momentum;
    int32_t n, pow2, nesterov, vec;   // vec: every matrix of every buffer lies on 16 bytes
};

__device__ __forceinline__ void block_part(float ss, float* out) {
    __shared__ float sh[32];
    ss = block_all<SumOp>(ss, sh);
    if (threadIdx.x == 0) *out = ss;
}

// A CTA per part of a matrix.  g as the bucket average has it: summed in rank order, then divided by N (times 1/N where
// that is exact).
template <bool BF16>
__global__ void __launch_bounds__(kThreads) update_kernel(const __grid_constant__ UpdateParams p) {
    constexpr int VEC = 4;
    pdl_enter();
    const int64_t off = p.offset[blockIdx.y], e0 = blockIdx.x * p.per, e1 = min(p.size, e0 + p.per);
    float* buf = p.buf + off;
    float* u = p.u + blockIdx.y * p.pitch;
    float ss = 0.0f;
    auto one = [&](float g, float& b) {                  // g: the sum over the replicas; returns U
        g = p.pow2 ? g * p.inv_n : __fdiv_rn(g, static_cast<float>(p.n));
        b = fmaf(p.momentum, b, g);
        const float v = p.nesterov ? fmaf(p.momentum, b, g) : b;
        ss = fmaf(v, v, ss);
        return v;
    };
    if (p.vec) {
        const int64_t whole = e0 + (e1 - e0) / VEC * VEC;
        for (int64_t e = e0 + threadIdx.x * VEC; e < whole; e += kThreads * VEC) {
            float4 b = *reinterpret_cast<const float4*>(buf + e);
            float s[VEC] = {};
#pragma unroll 8
            for (int r = 0; r < p.n; ++r) {
                if constexpr (BF16) {
                    uint2 v;
                    asm volatile("ld.global.cs.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(static_cast<const char*>(p.replica[r]) + (off + e) * 2) : "memory");
                    s[0] += bf16_lo(v.x);
                    s[1] += bf16_hi(v.x);
                    s[2] += bf16_lo(v.y);
                    s[3] += bf16_hi(v.y);
                } else {
                    const uint4 v = ld16<false>(static_cast<const char*>(p.replica[r]) + (off + e) * 4);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) s[i] += vec_elem<false>(v, i);
                }
            }
            float4 v;
            v.x = one(s[0], b.x);
            v.y = one(s[1], b.y);
            v.z = one(s[2], b.z);
            v.w = one(s[3], b.w);
            *reinterpret_cast<float4*>(buf + e) = b;
            *reinterpret_cast<float4*>(u + e) = v;
        }
        for (int64_t e = whole + threadIdx.x; e < e1; e += kThreads) {
            float s = 0.0f, b = buf[e];
            for (int r = 0; r < p.n; ++r) s += load_elem<BF16>(p.replica[r], off + e);
            u[e] = one(s, b);
            buf[e] = b;
        }
    } else {
        for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads) {
            float s = 0.0f, b = buf[e];
#pragma unroll 8
            for (int r = 0; r < p.n; ++r) s += load_elem<BF16>(p.replica[r], off + e);
            u[e] = one(s, b);
            buf[e] = b;
        }
    }
    block_part(ss, p.part + blockIdx.y * kParts + blockIdx.x);
}

struct SplitParams {
    const void* x[kGroup];   // the matrices, or one buffer of them: x[0] + pitch·b
    int64_t ldx, pitch;
    const float* part;
    float* alpha;            // [count]: 1 / ((‖U‖ + eps)·scale)
    __half* hi;              // [count][mp][np]
    __half* lo;              // or NULL
    int64_t size;
    float eps;
    int32_t rows, cols, parts, mp, np, tall, vec, listed;
};

__device__ __forceinline__ const void* matrix_of(const SplitParams& p, int b, bool bf16) {
    return p.listed ? p.x[b] : static_cast<const char*>(p.x[0]) + b * p.pitch * (bf16 ? 2 : 4);
}

// A CTA per part: rows in turn.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) square_kernel(const __grid_constant__ SplitParams p, float* part) {
    constexpr int VEC = BF16 ? 8 : 4;
    pdl_enter();
    const char* x = static_cast<const char*>(matrix_of(p, blockIdx.y, BF16));
    float ss = 0.0f;
    // a warp per row
    const int lane = threadIdx.x & 31, w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), n = gridDim.x * (kThreads / 32);
    for (int r = w; r < p.rows; r += n) {
        const char* row = row_ptr<BF16>(static_cast<const void*>(x), r, p.ldx);
        if (p.vec) {
            for (int c = lane; c < p.cols / VEC; c += 32) {
                const uint4 v = ld16_keep(row + static_cast<int64_t>(c) * 16);
#pragma unroll
                for (int e = 0; e < VEC; ++e) ss = fmaf(vec_elem<BF16>(v, e), vec_elem<BF16>(v, e), ss);
            }
        } else {
#pragma unroll 4
            for (int c = lane; c < p.cols; c += 32) {
                const float v = load_elem<BF16>(row, c);
                ss = fmaf(v, v, ss);
            }
        }
    }
    block_part(ss, part + blockIdx.y * kParts + blockIdx.x);
}

// A tile of 64 x 64 of X, read along the rows of the matrix it comes from.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) split_kernel(const __grid_constant__ SplitParams p) {
    __shared__ float tile[64][65];
    __shared__ float sh[32];
    pdl_enter();
    const int b = blockIdx.z, i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
    const char* x = static_cast<const char*>(matrix_of(p, b, BF16));
    const int r0 = p.tall ? j0 : i0, c0 = p.tall ? i0 : j0;      // in the matrix
    const int tc = threadIdx.x & 63, tr = threadIdx.x >> 6;
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int r = r0 + tr + 4 * k, c = c0 + tc;
        v[k] = r < p.rows && c < p.cols ? load_elem<BF16>(row_ptr<BF16>(static_cast<const void*>(x), r, p.ldx), c) : 0.0f;
    }
    float ss = 0.0f;
    for (int i = threadIdx.x; i < p.parts; i += kThreads) ss += p.part[b * kParts + i];
    const float norm = sqrtf(block_all<SumOp>(ss, sh));
    // the power of two that brings the entries to about 1, and none of them, at most the norm, past 32768
    float scale = 1.0f, alpha = __int_as_float(0x7fffffff);
    if (norm < INFINITY) {
        const float want = fminf(sqrtf(static_cast<float>(p.size)), 32768.0f) / norm;
        scale = want < 0x1p126f ? exp2f(floorf(log2f(fmaxf(want, 0x1p-126f)))) : norm > 0.0f ? 0x1p126f : 1.0f;
        alpha = norm > 0.0f ? 1.0f / (norm + p.eps) / scale : 0.0f;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) p.alpha[b] = alpha;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const float s = v[k] * scale;
        if (p.tall) tile[tc][tr + 4 * k] = s;
        else tile[tr + 4 * k][tc] = s;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = (threadIdx.x >> 3) + 32 * k, j = (threadIdx.x & 7) * 8;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float s0 = tile[i][j + 2 * q], s1 = tile[i][j + 2 * q + 1];
            const __half2 h = __floats2half2_rn(s0, s1);
            const float2 f = __half22float2(h);
            const __half2 l = __floats2half2_rn(s0 - f.x, s1 - f.y);
            hi[q] = *reinterpret_cast<const uint32_t*>(&h);
            lo[q] = *reinterpret_cast<const uint32_t*>(&l);
        }
        const int64_t at = (static_cast<int64_t>(b) * p.mp + i0 + i) * p.np + j0 + j;
        *reinterpret_cast<uint4*>(p.hi + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (p.lo) *reinterpret_cast<uint4*>(p.lo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// ---- products ------------------------------------------------------------

constexpr int kBlockK = 64;            // a row of 128 bytes
constexpr int kRows = 128;             // rows of either operand that a CTA holds
constexpr int kOperandBytes = kRows * 128, kStageBytes = 2 * kOperandBytes, kStages = 6;
constexpr int kStepThreads = 384;      // 4 warps of single roles, 8 of the epilogue
constexpr size_t kStepSmem = kStages * kStageBytes + 1024;   // more than half of an SM's: a CTA takes all of its TMEM

enum { kGram = 0, kPoly = 1, kApply = 2, kLast = 3 };
enum { kOutF32 = 0, kOutBf16 = 1, kOutParam = 2 };

struct StepParams {
    CUtensorMap ta, tb;
    const float* alpha;       // of the first step, or NULL: 1
    const __half* e_hi;       // kPoly: A; kApply and kLast: X
    const __half* e_lo;       // or NULL
    __half* o_hi;             // kGram: A; kPoly: B; kApply: X
    __half* o_lo;             // or NULL
    void* out[kGroup];        // kLast: results, or parameters
    void* out2[kGroup];       // parameters in bf16
    int64_t ldo;
    float decay, step;        // kOutParam
    float shift, ca, cb;      // of this step: A − shift·I, (a, b) of the polynomial of it
    int32_t kind, tall, vec, has2;
    int32_t m, n, mp, ld, cols;   // ld, cols: of what is read and written here (mp, or the padded n)
    int32_t blocks, tm, tn, per, pieces;
};

struct StepShared {
    uint64_t ready[kStages];   // of the first CTA: both CTAs' operands are in shared memory
    uint64_t done[kStages];    // a stage's MMAs: it may be overwritten
    uint64_t d_full[2], d_empty[2], idle;
    uint32_t tmem;
    volatile int failed;
};

template <bool PAIR>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if constexpr (PAIR) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"(static_cast<uint32_t>(add))
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"(static_cast<uint32_t>(add))
            : "memory");
    }
}
template <bool PAIR, bool BOTH = true>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (PAIR) mma_commit<BOTH>(bar);
    else asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The same operand by columns: 64 of them, 128 bytes, in each of the block's 64 rows of K (128-byte swizzle), the next
// 64 columns 8 KB on; groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_columns(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (512ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// The u-th tile: matrix, tile row and column; on and above the diagonal of a symmetric result.
struct Tile {
    int b, i, j;
};
template <int MODE>
__device__ __forceinline__ Tile tile_of(const StepParams& p, int u) {
    Tile t;
    t.b = u / p.per;
    int r = u - t.b * p.per;
    if constexpr (MODE == kGram || MODE == kPoly) {
        t.i = 0;
        for (int w = p.tm; r >= w; --w) {
            r -= w;
            ++t.i;
        }
        t.j = t.i + r;
    } else {
        t.i = r % p.tm;
        t.j = r / p.tm;
    }
    return t;
}

__device__ __forceinline__ float2 half_pair(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Sixteen columns of a result's row (of a column, where tall) to where the caller keeps them.
__device__ __forceinline__ void write_out(const StepParams& p, int b, int row, int col, const float (&v)[16]) {
    if (row >= p.m) return;
    const int cols = min(16, p.n - col);
    const int64_t at = p.tall ? static_cast<int64_t>(col) * p.ldo + row : static_cast<int64_t>(row) * p.ldo + col, by = p.tall ? p.ldo : 1;
    if (p.kind == kOutBf16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out[b]) + at;
        if (!p.tall && p.vec && cols == 16) {
            reinterpret_cast<uint4*>(o)[0] = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
            reinterpret_cast<uint4*>(o)[1] = make_uint4(pack2(v[8], v[9]), pack2(v[10], v[11]), pack2(v[12], v[13]), pack2(v[14], v[15]));
            return;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (e < cols) o[e * by] = __float2bfloat16_rn(v[e]);
        return;
    }
    float* o = static_cast<float*>(p.out[b]) + at;
    float w[16];
    const bool whole = !p.tall && p.vec && cols == 16;
    if (p.kind == kOutParam) {
        if (whole) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 t = reinterpret_cast<const float4*>(o)[q];
                w[4 * q] = t.x;
                w[4 * q + 1] = t.y;
                w[4 * q + 2] = t.z;
                w[4 * q + 3] = t.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = e < cols ? o[e * by] : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = fmaf(-p.step, v[e], w[e] * p.decay);
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = v[e];
    }
    if (whole) {
#pragma unroll
        for (int q = 0; q < 4; ++q) reinterpret_cast<float4*>(o)[q] = make_float4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (e < cols) o[e * by] = w[e];
    }
    if (p.has2) {
        __nv_bfloat16* c = static_cast<__nv_bfloat16*>(p.out2[b]) + at;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (e < cols) c[e * by] = __float2bfloat16_rn(w[e]);
    }
}

template <int MODE, bool PAIR>
__global__ void __launch_bounds__(kStepThreads, 1) step_kernel(const __grid_constant__ StepParams p) {
    extern __shared__ unsigned char raw[];
    __shared__ StepShared s;
    constexpr int SIDE = PAIR ? 256 : 128;               // of a tile
    constexpr int ARRIVALS = PAIR ? 16 : 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? blockIdx.x & 1 : 0;
    const uint32_t pad = (1024u - (smem_u32(raw) & 1023u)) & 1023u;
    unsigned char* ring = raw + pad;                     // [stages][2][128][128]
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(&s.ready[i], 1);
            bar_init(&s.done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&s.d_full[i], 1);
            bar_init(&s.d_empty[i], ARRIVALS);
        }
        bar_init(&s.idle, 1);
        s.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s.tmem)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s.tmem)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    fence_before();
    __syncthreads();
    if constexpr (PAIR) pair_sync();
    fence_after();
    // all 512 columns are this CTA's (this pair's), from address 0 on
    const uint32_t ring_addr = smem_u32(ring);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // every thread waits itself: what the launches before wrote is visible to a thread that has waited, and to no other
    pdl_wait();
    const int first = PAIR ? blockIdx.x >> 1 : blockIdx.x, step = PAIR ? gridDim.x >> 1 : gridDim.x;

    if (warp == 0 && lane == 0) {                        // producer
        Ring r;
        int issued = 0;
        bool ok = true;
        for (int u = first; u < p.pieces && ok; u += step) {
            const Tile t = tile_of<MODE>(p, u);
            const int ya = t.b * p.mp + t.i * SIDE + rank * kRows;
            const int jb = t.j * SIDE + rank * kRows;
            for (int k = 0; k < p.blocks; ++k) {
                if (!(ok = bar_wait(&s.done[r.i], r.ph ^ 1, s))) break;
                unsigned char* d = ring + r.i * kStageBytes;
                if (rank == 0) bar_expect(&s.ready[r.i], (PAIR ? 2 : 1) * kStageBytes);
                auto load = [&](unsigned char* to, const CUtensorMap* map, int x, int y) {
                    if constexpr (PAIR) tma_load_pair(to, map, x, y, first_of_pair(&s.ready[r.i]));
                    else tma_load(to, map, x, y, &s.ready[r.i]);
                };
                load(d, &p.ta, k * kBlockK, ya);
                if constexpr (MODE == kGram || MODE == kPoly) {
                    load(d + kOperandBytes, &p.tb, k * kBlockK, t.b * p.mp + jb);
                } else {
                    load(d + kOperandBytes, &p.tb, jb, t.b * p.mp + k * kBlockK);
                    load(d + kOperandBytes + kOperandBytes / 2, &p.tb, jb + 64, t.b * p.mp + k * kBlockK);
                }
                r.next(kStages);
                ++issued;
            }
        }
        // every copy has landed, and been multiplied, before the CTA gives its shared memory back
        for (int j = 0; j < kStages && j < issued; ++j) {
            r.back(kStages);
            bar_drain(&s.done[r.i], r.ph, s);
        }
    } else if (warp == 1 && rank == 0) {                 // issuer: the whole warp, so that descriptors stay in uniform registers
        Ring x, d;
        constexpr uint32_t idesc = (1u << 4) | (MODE == kGram || MODE == kPoly ? 0u : 1u << 16) |
                                   (static_cast<uint32_t>(SIDE / 8) << 17) | (static_cast<uint32_t>(SIDE / 16) << 24);
        const bool one = elect();
        bool ok = true, there = false;
        for (int u = first; u < p.pieces && ok; u += step) {
            if (!(ok = __all_sync(0xffffffffu, bar_wait(&s.d_empty[d.i], d.ph ^ 1, s)))) break;
            fence_after();
            const uint32_t acc = d.i * SIDE;
            for (int k = 0; k < p.blocks; ++k) {
                if (!there && !(ok = __all_sync(0xffffffffu, bar_wait_pair(&s.ready[x.i], x.ph, s)))) break;
                fence_after();
                const uint32_t at = ring_addr + x.i * kStageBytes;
                const uint64_t a = smem_desc(at);
                const uint64_t b = MODE == kGram || MODE == kPoly ? smem_desc(at + kOperandBytes) : smem_desc_columns(at + kOperandBytes);
                constexpr int bstep = MODE == kGram || MODE == kPoly ? 2 : 128;   // 16 of K, in 16 bytes
                if (one) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) mma_ss<PAIR>(acc, a + 2 * q, b + bstep * q, idesc, k > 0 || q > 0);
                }
                // a look at the next stage while these run
                Ring y = x;
                y.next(kStages);
                there = __all_sync(0xffffffffu, bar_test_pair(&s.ready[y.i], y.ph));
                if (one) commit<PAIR>(&s.done[x.i]);
                __syncwarp();
                x = y;
            }
            if (ok && one) commit<PAIR>(&s.d_full[d.i]);
            d.next(2);
        }
        if (one) {
            commit<PAIR, false>(&s.idle);
            bar_drain(&s.idle, 0, s);
        }
    } else if (warp >= 4) {                              // epilogue: 32 rows, half of the columns
        Ring d;
        constexpr int COLS = SIDE / 2;
        const int q = warp & 3, half = (warp - 4) >> 2;
        for (int u = first; u < p.pieces; u += step) {
            const Tile t = tile_of<MODE>(p, u);
            const int row = t.i * SIDE + rank * kRows + q * 32 + lane;
            const bool in = row < p.mp;
            const float alpha = p.alpha ? p.alpha[t.b] : 1.0f;
            const int64_t base = (static_cast<int64_t>(t.b) * p.mp + row) * p.ld;
            const uint32_t acc = d.i * SIDE + (static_cast<uint32_t>(q * 32) << 16);
            bool ok = true;
            for (int c0 = 0; c0 < COLS; c0 += 64) {
                const int col0 = t.j * SIDE + half * COLS + c0;
                const bool cols = col0 < p.cols;         // padded to 64: all or none
                uint4 hi[8], lo[8];
                if constexpr (MODE != kGram) {           // fetched while the tile is still being summed
                    if (in && cols) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) hi[i] = ld16_keep(p.e_hi + base + col0 + 8 * i);
                        if (MODE != kPoly && p.e_lo) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) lo[i] = ld16_keep(p.e_lo + base + col0 + 8 * i);
                        }
                    }
                }
                if (c0 == 0) {
                    ok = bar_wait(&s.d_full[d.i], d.ph, s) && !s.failed;
                    fence_after();
                }
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    float v[16];
                    __syncwarp();
                    tmem_ld16(acc + half * COLS + c0 + 16 * h, v);
                    if (c0 + 64 >= COLS && h == 3) {     // the accumulator is free before its last columns are stored
                        fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if constexpr (PAIR) bar_arrive_first(&s.d_empty[d.i]);
                            else bar_arrive(&s.d_empty[d.i]);
                        }
                    }
                    if (!in || !cols) continue;
                    const int col = col0 + 16 * h;
                    if (!ok) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = __int_as_float(0x7fffffff);
                    }
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        if constexpr (MODE == kGram) {
                            v[e] = fmaf(v[e], alpha * alpha, row == col + e ? -p.shift : 0.0f);
                            v[e + 1] = fmaf(v[e + 1], alpha * alpha, row == col + e + 1 ? -p.shift : 0.0f);
                        } else {
                            float2 f = half_pair(word(hi[2 * h + e / 8], e / 2 % 4));
                            if constexpr (MODE == kPoly) {
                                v[e] = fmaf(kC, v[e], p.cb * f.x);
                                v[e + 1] = fmaf(kC, v[e + 1], p.cb * f.y);
                            } else {
                                if (p.e_lo) {
                                    const float2 g = half_pair(word(lo[2 * h + e / 8], e / 2 % 4));
                                    f.x += g.x;
                                    f.y += g.y;
                                }
                                v[e] = alpha * fmaf(p.ca, f.x, v[e]);
                                v[e + 1] = alpha * fmaf(p.ca, f.y, v[e + 1]);
                            }
                        }
                    }
                    if constexpr (MODE == kLast) {
                        if (col < p.n) write_out(p, t.b, row, col, v);
                    } else {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const __half2 x = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
                            w[e] = *reinterpret_cast<const uint32_t*>(&x);
                        }
                        uint4* o = reinterpret_cast<uint4*>(p.o_hi + base + col);
                        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        if constexpr (MODE == kApply) {
                            if (p.o_lo) {
                                uint32_t z[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const float2 f = half_pair(w[e]);
                                    const __half2 x = __floats2half2_rn(v[2 * e] - f.x, v[2 * e + 1] - f.y);
                                    z[e] = *reinterpret_cast<const uint32_t*>(&x);
                                }
                                uint4* ol = reinterpret_cast<uint4*>(p.o_lo + base + col);
                                ol[0] = make_uint4(z[0], z[1], z[2], z[3]);
                                ol[1] = make_uint4(z[4], z[5], z[6], z[7]);
                            }
                        } else if (t.i != t.j) {         // the tile below the diagonal
                            unsigned short* m = reinterpret_cast<unsigned short*>(p.o_hi) + (static_cast<int64_t>(t.b) * p.mp + col) * p.ld + row;
#pragma unroll
                            for (int e = 0; e < 16; ++e) m[static_cast<int64_t>(e) * p.ld] = static_cast<unsigned short>(w[e / 2] >> (16 * (e & 1)));
                        }
                    }
                }
            }
            d.next(2);
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if constexpr (PAIR) pair_sync();                     // nothing of the pair's is in flight any more
    fence_after();
    if (warp == 0) {
        if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(s.tmem) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(s.tmem) : "memory");
    }
}

// ---- host ----------------------------------------------------------------

// Where everything lies in the workspace, for a group of `count` matrices.
struct Layout {
    int m, n, mp, np;
    bool tall;
    int64_t size, pitch;      // of U
    size_t u, part, alpha, x0, x1, lo, a, b, total;
};
Layout layout_of(int count, int rows, int cols) {
    Layout l{};
    l.tall = rows > cols;
    l.m = l.tall ? cols : rows;
    l.n = l.tall ? rows : cols;
    l.mp = static_cast<int>(round_up(l.m, kPad));
    l.np = static_cast<int>(round_up(l.n, kPad));
    l.size = static_cast<int64_t>(rows) * cols;
    l.pitch = round_up(l.size, 8);
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += static_cast<size_t>(round_up(bytes * count, 256));
        return here;
    };
    const int64_t x = static_cast<int64_t>(l.mp) * l.np * 2, a = static_cast<int64_t>(l.mp) * l.mp * 2;
    l.u = take(l.pitch * 4);
    l.part = take(kParts * 4);
    l.alpha = take(4);
    l.x0 = take(x);
    l.x1 = take(x);
    l.lo = take(x);
    l.a = take(a);
    l.b = take(a);
    l.total = at;
    return l;
}

// Tiles by pairs of CTAs or by single ones: the less time, in K blocks of a 128 x 128 tile.  A pair's 256 x 256 tile
// takes two such times of the tensor cores, a CTA's 128 x 128 one a little more than one (its operands come at
// twice the bytes per product).
struct Tiling {
    bool pair;
    int tm, tn, per, ctas;
};
Tiling tiling(int count, int rows, int cols, bool symmetric, int sms) {
    auto tiles = [&](int side) {
        const int64_t tm = (rows + side - 1) / side, tn = (cols + side - 1) / side;
        return symmetric ? tm * (tm + 1) / 2 : tm * tn;
    };
    auto waves = [](int64_t n, int at) { return (n + at - 1) / at; };
    const int64_t two = tiles(256) * count, one = tiles(128) * count;
    const bool pair = waves(two, sms / 2) * 20 <= waves(one, sms) * 13;
    const int side = pair ? 256 : 128;
    Tiling t{pair, (rows + side - 1) / side, (cols + side - 1) / side, static_cast<int>(tiles(side)), 0};
    const int64_t n = pair ? two : one, most = pair ? sms / 2 : sms;
    t.ctas = static_cast<int>(std::min(n, most)) * (pair ? 2 : 1);
    return t;
}

struct Call {
    int count, rows, cols, steps;
    float eps;
    unsigned char* ws;
    cudaStream_t s;
};

// What the last product writes: one pointer per matrix.
struct Results {
    int kind;
    int64_t ld;
    bool vec;
    float decay, step;
    void* const* out;
    void* const* out2;
};

template <int MODE>
int launch_step(const StepParams& p, const Tiling& t, cudaStream_t s) {
    return launch_smem(t.pair ? step_kernel<MODE, true> : step_kernel<MODE, false>, static_cast<unsigned>(t.ctas), kStepThreads,
                       kStepSmem, s, p, t.pair ? 2 : 1);
}

// The steps on a group of matrices that split_kernel has laid out.
int run_steps(const Call& c, const Layout& l, const Results& r) {
    DeviceInfo d;
    int st = current_device_info(&d);
    if (st != DDP_OK) return st;
    __half* x[2] = {reinterpret_cast<__half*>(c.ws + l.x0), reinterpret_cast<__half*>(c.ws + l.x1)};
    __half* lo = reinterpret_cast<__half*>(c.ws + l.lo);
    __half* a = reinterpret_cast<__half*>(c.ws + l.a);
    __half* b = reinterpret_cast<__half*>(c.ws + l.b);
    const int64_t all = static_cast<int64_t>(c.count) * l.mp;
    auto map = [&](CUtensorMap* t, const __half* base, int cols, int box_rows) {
        return encode(t, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, cols, all, static_cast<int64_t>(cols) * 2, kBlockK, box_rows,
                      CU_TENSOR_MAP_SWIZZLE_128B);
    };
    CUtensorMap xk[2], xn[2], ak, bk;
    for (int i = 0; i < 2; ++i) {
        if ((st = map(&xk[i], x[i], l.np, kRows)) != DDP_OK) return st;
        if ((st = map(&xn[i], x[i], l.np, kBlockK)) != DDP_OK) return st;
    }
    if ((st = map(&ak, a, l.mp, kRows)) != DDP_OK) return st;
    if ((st = map(&bk, b, l.mp, kRows)) != DDP_OK) return st;
    const Tiling sym = tiling(c.count, l.mp, l.mp, true, d.sm_count), full = tiling(c.count, l.mp, l.np, false, d.sm_count);
    StepParams p{};
    p.m = l.m;
    p.n = l.n;
    p.mp = l.mp;
    auto shape = [&](const Tiling& t, int cols, int blocks) {
        p.ld = p.cols = cols;
        p.blocks = blocks;
        p.tm = t.tm;
        p.tn = t.tn;
        p.per = t.per;
        p.pieces = t.per * c.count;
    };
    for (int i = 0; i < c.steps; ++i) {
        const int from = i & 1;
        // once A is near I: of A' = A − I, B = (b + c)I + (b + 2c)A' + cA'²
        const bool near = i >= std::max(c.steps - 2, 2);
        p.shift = near ? 1.0f : 0.0f;
        p.ca = near ? kA + kB + kC : kA;
        p.cb = near ? kB + 2.0f * kC : kB;
        p.alpha = i == 0 ? reinterpret_cast<const float*>(c.ws + l.alpha) : nullptr;
        shape(sym, l.mp, l.np / kBlockK);
        p.ta = xk[from];
        p.tb = xk[from];
        p.o_hi = a;
        if ((st = launch_step<kGram>(p, sym, c.s)) != DDP_OK) return st;
        p.alpha = nullptr;
        shape(sym, l.mp, l.mp / kBlockK);
        p.ta = ak;
        p.tb = ak;
        p.e_hi = a;
        p.o_hi = b;
        if ((st = launch_step<kPoly>(p, sym, c.s)) != DDP_OK) return st;
        p.alpha = i == 0 ? reinterpret_cast<const float*>(c.ws + l.alpha) : nullptr;
        shape(full, l.np, l.mp / kBlockK);
        p.ta = bk;
        p.tb = xn[from];
        p.e_hi = x[from];
        p.e_lo = i < c.steps - 2 ? lo : nullptr;
        if (i + 1 < c.steps) {
            p.o_hi = x[from ^ 1];
            p.o_lo = i + 1 < c.steps - 2 ? lo : nullptr;
            if ((st = launch_step<kApply>(p, full, c.s)) != DDP_OK) return st;
        } else {
            p.kind = r.kind;
            p.tall = l.tall;
            p.vec = r.vec;
            p.has2 = r.out2 != nullptr;
            p.ldo = r.ld;
            p.decay = r.decay;
            p.step = r.step;
            for (int k = 0; k < c.count; ++k) {
                p.out[k] = r.out[k];
                p.out2[k] = r.out2 ? r.out2[k] : nullptr;
            }
            if ((st = launch_step<kLast>(p, full, c.s)) != DDP_OK) return st;
        }
    }
    return DDP_OK;
}

int split(const Call& c, const Layout& l, SplitParams& p, bool bf16) {
    p.part = reinterpret_cast<const float*>(c.ws + l.part);
    p.alpha = reinterpret_cast<float*>(c.ws + l.alpha);
    p.hi = reinterpret_cast<__half*>(c.ws + l.x0);
    p.lo = c.steps > 2 ? reinterpret_cast<__half*>(c.ws + l.lo) : nullptr;
    p.size = l.size;
    p.eps = c.eps;
    p.rows = c.rows;
    p.cols = c.cols;
    p.mp = l.mp;
    p.np = l.np;
    p.tall = l.tall;
    return launch_pdl(bf16 ? split_kernel<true> : split_kernel<false>,
                      dim3(static_cast<unsigned>(l.np / 64), static_cast<unsigned>(l.mp / 64), static_cast<unsigned>(c.count)), kThreads, c.s, p);
}

bool sizes_ok(int32_t count, int32_t rows, int32_t cols) { return count >= 0 && rows >= 0 && cols >= 0; }

}  // namespace
}  // namespace ddp

using namespace ddp;

extern "C" size_t newton_schulz_workspace_bytes(int32_t count, int32_t rows, int32_t cols) {
    if (!sizes_ok(count, rows, cols) || rows > kMaxSide || cols > kMaxSide) return 0;
    if (count == 0 || rows == 0 || cols == 0) return 16;
    return layout_of(std::min(count, kGroup), rows, cols).total;
}

namespace ddp {
namespace {

// launch_pdl with a second argument for square_kernel
template <typename Params, typename Arg>
int launch_pdl2(void (*kernel)(Params, Arg), dim3 grid, int block, cudaStream_t s, const Params& params, Arg arg) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, params, arg);
    return e == cudaSuccess ? check_launch() : cuda_fail(e);
}

}  // namespace
}  // namespace ddp

extern "C" int newton_schulz(const void* const* x, int64_t ldx, int32_t x_dtype, void* const* out, int64_t ldo,
                             int32_t out_dtype, int32_t count, int32_t rows, int32_t cols, int32_t steps, float eps,
                             void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype) || !sizes_ok(count, rows, cols) || steps < 1 || steps > kMaxSteps ||
        !(eps >= 0.0f) || !(eps < 3.0e38f))
        return DDP_ERR_INVALID_ARG;
    if (rows > kMaxSide || cols > kMaxSide) return DDP_ERR_UNSUPPORTED;
    if (count == 0 || rows == 0 || cols == 0) return DDP_OK;
    if (x == nullptr || out == nullptr || workspace == nullptr) return DDP_ERR_INVALID_ARG;
    const size_t need = newton_schulz_workspace_bytes(count, rows, cols);
    const Mat ws{workspace, 1, static_cast<int64_t>(need), static_cast<int64_t>(need), 1};
    const bool bf16 = x_dtype == DDP_BF16;
    bool in_vec = cols % (bf16 ? 8 : 4) == 0, out_vec = true;
    for (int i = 0; i < count; ++i) {
        const Mat mx{x[i], rows, cols, ldx, dsize(x_dtype)}, mo{out[i], rows, cols, ldo, dsize(out_dtype)};
        if (!mat_valid(mx) || !mat_valid(mo) || x[i] == nullptr || out[i] == nullptr) return DDP_ERR_INVALID_ARG;
        if (!mat_aligned(mx) || !mat_aligned(mo)) return DDP_ERR_ALIGNMENT;
        if (mats_overlap(mx, ws) || mats_overlap(mo, ws)) return DDP_ERR_INVALID_ARG;
        for (int j = 0; j < count; ++j) {
            const Mat oj{out[j], rows, cols, ldo, dsize(out_dtype)};
            if ((i != j && mats_overlap(mo, oj)) || (mats_overlap(mx, oj) && !(i == j && mats_same(mx, oj)))) return DDP_ERR_INVALID_ARG;
        }
        in_vec &= aligned16(x[i]) && (rows == 1 || ldx * dsize(x_dtype) % 16 == 0);
        out_vec &= aligned16(out[i]) && (rows == 1 || ldo * dsize(out_dtype) % 16 == 0);
    }
    if (!aligned16(workspace)) return DDP_ERR_ALIGNMENT;
    if (workspace_bytes < need) return DDP_ERR_CAPACITY;
    for (int i = 0; i < count; i += kGroup) {
        const Call c{std::min(kGroup, count - i), rows, cols, steps, eps, static_cast<unsigned char*>(workspace), static_cast<cudaStream_t>(stream)};
        const Layout l = layout_of(c.count, rows, cols);
        SplitParams p{};
        for (int k = 0; k < c.count; ++k) p.x[k] = x[i + k];
        p.listed = 1;
        p.ldx = ldx;
        p.vec = in_vec;
        p.rows = rows;
        p.cols = cols;
        // a CTA takes eight rows at a time
        p.parts = static_cast<int32_t>(std::min<int64_t>(kParts, std::min<int64_t>((rows + 7) / 8, (l.size + kPartElems - 1) / kPartElems)));
        float* part = reinterpret_cast<float*>(c.ws + l.part);
        int st = launch_pdl2(bf16 ? square_kernel<true> : square_kernel<false>,
                             dim3(static_cast<unsigned>(p.parts), static_cast<unsigned>(c.count)), kThreads, c.s, p, part);
        if (st != DDP_OK || (st = split(c, l, p, bf16)) != DDP_OK) return st;
        const Results r{out_dtype == DDP_BF16 ? kOutBf16 : kOutF32, ldo, out_vec, 0.0f, 0.0f, out + i, nullptr};
        if ((st = run_steps(c, l, r)) != DDP_OK) return st;
    }
    return DDP_OK;
}

extern "C" int ddp_bucket_allreduce_muon(const void* const* replicas, int32_t n_replicas, int32_t dtype,
                                         const int64_t* offsets, int32_t count, int32_t rows, int32_t cols, float* param,
                                         float* momentum_buf, float lr, float momentum, float weight_decay,
                                         float update_scale, int32_t nesterov, int32_t steps, float eps,
                                         void* param_bf16, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dtype) || n_replicas < 1 || n_replicas > kMaxReplicas || !sizes_ok(count, rows, cols) || steps < 1 ||
        steps > kMaxSteps || !(eps >= 0.0f) || !(eps < 3.0e38f))
        return DDP_ERR_INVALID_ARG;
    if (rows > kMaxSide || cols > kMaxSide) return DDP_ERR_UNSUPPORTED;
    if (count == 0 || rows == 0 || cols == 0) return DDP_OK;
    if (replicas == nullptr || offsets == nullptr || param == nullptr || momentum_buf == nullptr || workspace == nullptr)
        return DDP_ERR_INVALID_ARG;
    const int es = dsize(dtype);
    const int64_t size = static_cast<int64_t>(rows) * cols;
    // matrices do not share elements; the buffers' ranges that hold them do not meet
    int64_t low = INT64_MAX, high = 0;
    bool on4 = true;
    for (int i = 0; i < count; ++i) {
        if (offsets[i] < 0 || offsets[i] > INT64_MAX / 16 - size) return DDP_ERR_INVALID_ARG;
        low = std::min(low, offsets[i]);
        high = std::max(high, offsets[i] + size);
        on4 &= offsets[i] % 4 == 0;
        for (int j = 0; j < i; ++j)
            if (offsets[i] < offsets[j] + size && offsets[j] < offsets[i] + size) return DDP_ERR_INVALID_ARG;
    }
    const size_t need = newton_schulz_workspace_bytes(count, rows, cols);
    struct Range {
        const char* p;
        size_t n;
    };
    auto range = [&](const void* p, int bytes) {
        return Range{p ? static_cast<const char*>(p) + low * bytes : nullptr, static_cast<size_t>(high - low) * bytes};
    };
    const Range outs[4] = {range(param, 4), range(momentum_buf, 4), range(param_bf16, 2), {static_cast<const char*>(workspace), need}};
    for (int r = 0; r < n_replicas; ++r) {
        if (replicas[r] == nullptr) return DDP_ERR_INVALID_ARG;
        if (!aligned16(replicas[r])) return DDP_ERR_ALIGNMENT;
        const Range in = range(replicas[r], es);
        for (const Range& o : outs)
            if (overlaps(o.p, o.n, in.p, in.n)) return DDP_ERR_INVALID_ARG;
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return DDP_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(param), static_cast<const void*>(momentum_buf), static_cast<const void*>(param_bf16), static_cast<const void*>(workspace)})
        if (!aligned16(p)) return DDP_ERR_ALIGNMENT;
    if (workspace_bytes < need) return DDP_ERR_CAPACITY;
    for (int i = 0; i < count; i += kGroup) {
        const Call c{std::min(kGroup, count - i), rows, cols, steps, eps, static_cast<unsigned char*>(workspace), static_cast<cudaStream_t>(stream)};
        const Layout l = layout_of(c.count, rows, cols);
        UpdateParams u{};
        for (int r = 0; r < n_replicas; ++r) u.replica[r] = replicas[r];
        void *out[kGroup], *out2[kGroup];
        for (int k = 0; k < c.count; ++k) {
            u.offset[k] = offsets[i + k];
            out[k] = param + offsets[i + k];
            out2[k] = param_bf16 ? static_cast<char*>(param_bf16) + offsets[i + k] * 2 : nullptr;
        }
        u.buf = momentum_buf;
        u.u = reinterpret_cast<float*>(c.ws + l.u);
        u.part = reinterpret_cast<float*>(c.ws + l.part);
        u.size = l.size;
        u.pitch = l.pitch;
        const int64_t parts = std::min<int64_t>(kParts, (l.size + kPartElems - 1) / kPartElems);
        u.per = round_up((l.size + parts - 1) / parts, 8);
        const int used = static_cast<int>((l.size + u.per - 1) / u.per);
        u.inv_n = 1.0f / static_cast<float>(n_replicas);
        u.momentum = momentum;
        u.n = n_replicas;
        u.pow2 = (n_replicas & (n_replicas - 1)) == 0;
        u.nesterov = nesterov != 0;
        u.vec = on4;
        int st = launch_pdl(dtype == DDP_BF16 ? update_kernel<true> : update_kernel<false>,
                            dim3(static_cast<unsigned>(used), static_cast<unsigned>(c.count)), kThreads, c.s, u);
        if (st != DDP_OK) return st;
        SplitParams p{};
        p.x[0] = u.u;
        p.ldx = cols;
        p.pitch = l.pitch;
        p.parts = used;
        if ((st = split(c, l, p, false)) != DDP_OK) return st;
        const Results r{kOutParam, cols, on4 && cols % 4 == 0, 1.0f - lr * weight_decay, lr * update_scale, out, param_bf16 ? out2 : nullptr};
        if ((st = run_steps(c, l, r)) != DDP_OK) return st;
    }
    return DDP_OK;
}
