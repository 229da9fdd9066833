// Product of 8-bit integers with a scale for each token and each channel:
//   out[m, n] = (Σ_k a[m, k]·w[n, k]) · a_scale[m] · w_scale[n]
//
// The sum is an exact 32-bit integer (K <= 131071 keeps |Σ| < 2^31).
#include <cstdint>

#include "rows.cuh"

namespace ddp {
namespace {

constexpr int kMaxK = 131071;

struct Q8Params {
    const int8_t* a;
    const int8_t* w;
    const float* sa;
    const float* sw;
    void* out;
    int64_t lda, ldw, ldo, M, N;
    int32_t K;
};

// 32 x 32 outputs per CTA, 32 bytes of K at a time in shared memory, four
// products per dp4a.
template <bool BF16>
__global__ void __launch_bounds__(256) q8_tile_kernel(const __grid_constant__ Q8Params p) {
    __shared__ int sa[32][9], sw[32][9];
    pdl_enter();
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 32, n0 = static_cast<int64_t>(blockIdx.x) * 32;
    const int t = threadIdx.x, row = t >> 3, q = t & 7;
    int acc[4] = {0, 0, 0, 0};
    for (int k0 = 0; k0 < p.K; k0 += 32) {
        uint32_t va = 0, vw = 0;
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + 4 * q + j;
            if (k >= p.K) break;
            if (m0 + row < p.M) va |= static_cast<uint32_t>(static_cast<uint8_t>(p.a[(m0 + row) * p.lda + k])) << (8 * j);
            if (n0 + row < p.N) vw |= static_cast<uint32_t>(static_cast<uint8_t>(p.w[(n0 + row) * p.ldw + k])) << (8 * j);
        }
        sa[row][q] = static_cast<int>(va);
        sw[row][q] = static_cast<int>(vw);
        __syncthreads();
        for (int j = 0; j < 8; ++j)
            for (int i = 0; i < 4; ++i) acc[i] = __dp4a(sa[(t >> 5) * 4 + i][j], sw[t & 31][j], acc[i]);
        __syncthreads();
    }
    const int64_t n = n0 + (t & 31);
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + (t >> 5) * 4 + i;
        if (m < p.M && n < p.N)
            store_elem<BF16>(p.out, m * p.ldo + n, static_cast<float>(acc[i]) * p.sa[m] * p.sw[n]);
    }
}

}  // namespace
}  // namespace ddp

using namespace ddp;

extern "C" size_t q8_matmul_workspace_bytes(int64_t M, int64_t N, int32_t K) {
    return M < 0 || N < 0 || K < 0 || K > kMaxK ? 0 : 16;
}

extern "C" int q8_matmul(const int8_t* a, int64_t lda, const float* a_scale, const int8_t* w, int64_t ldw,
                         const float* w_scale, int64_t M, int64_t N, int32_t K, void* out, int64_t ldo,
                         int32_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if ((out_dtype != DDP_F32 && out_dtype != DDP_BF16) || M < 0 || N < 0 || K < 0) return DDP_ERR_INVALID_ARG;
    if (K > kMaxK || M > INT32_MAX || N > INT32_MAX) return DDP_ERR_UNSUPPORTED;
    const Mat ma{a, M, K, lda, 1}, mw{w, N, K, ldw, 1}, mo{out, M, N, ldo, out_dtype == DDP_BF16 ? 2 : 4},
        msa{a_scale, 1, M, M, 4}, msw{w_scale, 1, N, N, 4};
    if (!mat_valid(ma) || !mat_valid(mw) || !mat_valid(mo)) return DDP_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && (out == nullptr || a_scale == nullptr || w_scale == nullptr ||
                           (K > 0 && (a == nullptr || w == nullptr))))
        return DDP_ERR_INVALID_ARG;
    const size_t need = q8_matmul_workspace_bytes(M, N, K);
    const Mat ws{workspace, 1, static_cast<int64_t>(need), static_cast<int64_t>(need), 1};
    for (const Mat* m : {&mo, &msa, &msw})
        if (!mat_aligned(*m)) return DDP_ERR_ALIGNMENT;
    for (const Mat* i : {&ma, &mw, &msa, &msw})
        if (mats_overlap(mo, *i) || mats_overlap(ws, *i)) return DDP_ERR_INVALID_ARG;
    if (mats_overlap(mo, ws)) return DDP_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return DDP_OK;
    if (workspace == nullptr) return DDP_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return DDP_ERR_ALIGNMENT;
    if (workspace_bytes < need) return DDP_ERR_CAPACITY;
    const Q8Params p{a, w, a_scale, w_scale, out, lda, ldw, ldo, M, N, K};
    if ((M + 31) / 32 > 65535) return DDP_ERR_UNSUPPORTED;
    void (*kernel)(Q8Params) = out_dtype == DDP_BF16 ? q8_tile_kernel<true> : q8_tile_kernel<false>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>((N + 31) / 32), static_cast<unsigned>((M + 31) / 32)), 256,
                      static_cast<cudaStream_t>(stream), p);
}
