// Distillation from a teacher's top logits: loss and gradient.
//
// For a token with student logits z[0..V) and the teacher's k entries
// (index, logit) at the temperature τ:
//   p = softmax(teacher / τ) over the entries whose index lies in [0, V)
//   q = softmax(z / τ) over the vocabulary, lse = ln Σ exp(z / τ)
//   loss = τ² Σ_j p_j (ln p_j − ln q[index_j])
//   dz_v = dloss·τ·(q_v − Σ_{j: index_j = v} p_j)
// (τ² · d(z/τ)/dz = τ).  A token without entries (none in the vocabulary, or
// all of them -infinity) has loss and gradient 0, and the gradient of one
// whose dloss is 0 is 0, whatever its logits hold.
#include <cstdint>

#include "rows.cuh"

namespace ddp {
namespace {

constexpr int kDistillThreads = 512;
constexpr int kMaxTop = DDP_DISTILL_MAX_TOP;

struct DistillParams {
    const void* z;
    const void* index;
    const void* teacher;
    const float* lse_in;   // backward alone
    const float* dloss;    // NULL: 1
    float* loss;
    float* lse;
    void* dz;
    int64_t ldz, ldi, ldt, lddz, T;
    int32_t V, k;
    float tau, c;          // c = log2(e) / τ
};

// A CTA per token.  All exponentials are powers of two of z·c − M with
// M = c·max z, so that loss and gradient see differences of logits only.
template <bool BF16, bool TBF16, bool I64, bool FWD, bool BWD>
__global__ void __launch_bounds__(kDistillThreads) distill_loop_kernel(const __grid_constant__ DistillParams a) {
    __shared__ float sh[32];
    __shared__ int s_idx[kMaxTop];
    __shared__ float s_p[kMaxTop], s_z[kMaxTop];
    pdl_enter();
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const void* z = row_ptr<BF16>(a.z, row, a.ldz);
        // the teacher's entries: p_j, and ln p_j kept as a power of two in registers
        float tm = -INFINITY;
        int n_valid = 0;
        for (int j = threadIdx.x; j < a.k; j += kDistillThreads) {
            const int64_t e = row * a.ldi + j;
            const int64_t i = I64 ? static_cast<const int64_t*>(a.index)[e]
                                  : static_cast<int64_t>(static_cast<const int32_t*>(a.index)[e]);
            const bool ok = i >= 0 && i < a.V;
            const float t = load_elem<TBF16>(row_ptr<TBF16>(a.teacher, row, a.ldt), j) * a.c;
            s_idx[j] = ok ? static_cast<int>(i) : -1;
            s_p[j] = ok ? t : -INFINITY;
            s_z[j] = ok ? load_elem<BF16>(z, i) : 0.0f;
            if (ok) {
                tm = max_nan(tm, t);
                n_valid += t == -INFINITY ? 0 : 1;
            }
        }
        const bool some = __syncthreads_or(n_valid) != 0;
        tm = block_all<MaxNanOp>(tm, sh);
        float ts = 0.0f;
        for (int j = threadIdx.x; j < a.k; j += kDistillThreads) ts += some && s_idx[j] >= 0 ? exp2f(s_p[j] - tm) : 0.0f;
        ts = block_all<SumOp>(ts, sh);
        const float g = (a.dloss ? a.dloss[row] : 1.0f) * a.tau;
        const bool zero = !some || g == 0.0f;

        float M = 0.0f, ls = 0.0f;   // q_v = 2^(z·c − M − ls)
        if constexpr (FWD) {
            float m = -INFINITY;
            for (int v = threadIdx.x; v < a.V; v += kDistillThreads) m = fmaxf(m, load_elem<BF16>(z, v));
            m = block_all<MaxOp>(m, sh);
            M = m == -INFINITY ? 0.0f : m * a.c;
            float s = 0.0f;
            for (int v = threadIdx.x; v < a.V; v += kDistillThreads) s += exp2f(fmaf(load_elem<BF16>(z, v), a.c, -M));
            s = block_all<SumOp>(s, sh);
            ls = log2f(s);
            float l = 0.0f;
            for (int j = threadIdx.x; j < a.k; j += kDistillThreads) {
                if (!some || s_idx[j] < 0) continue;
                const float p = exp2f(s_p[j] - tm) / ts;
                if (p == 0.0f) continue;
                l += p * ((s_p[j] - tm) - log2f(ts) - (fmaf(s_z[j], a.c, -M) - ls));
            }
            l = block_all<SumOp>(l, sh);
            if (threadIdx.x == 0) {
                a.loss[row] = some ? l * kLn2 * a.tau * a.tau : 0.0f;
                if (a.lse) a.lse[row] = (M + ls) * kLn2;
            }
        } else {
            M = a.lse_in[row] * kLog2e;
        }
        if constexpr (BWD) {
            void* dz = row_ptr<BF16>(a.dz, row, a.lddz);
            __syncthreads();
            for (int v = threadIdx.x; v < a.V; v += kDistillThreads)
                store_elem<BF16>(dz, v, zero ? 0.0f : g * exp2f(fmaf(load_elem<BF16>(z, v), a.c, -M) - ls));
            __syncthreads();
            for (int j = threadIdx.x; j < a.k && !zero; j += kDistillThreads) {
                const int i = s_idx[j];
                if (i < 0) continue;
                bool first = true;
                float p = 0.0f;
                for (int u = 0; u < a.k; ++u) {
                    if (s_idx[u] != i) continue;
                    if (u < j) first = false;
                    p += exp2f(s_p[u] - tm) / ts;
                }
                if (first) store_elem<BF16>(dz, i, g * (exp2f(fmaf(s_z[j], a.c, -M) - ls) - p));
            }
        }
        __syncthreads();
    }
}

bool dtype_ok(int32_t t) { return t == DDP_F32 || t == DDP_BF16; }
int dsize(int32_t t) { return t == DDP_BF16 ? 2 : 4; }

template <bool BF16, bool TBF16, bool I64>
void (*pick_dir(bool fwd, bool bwd))(DistillParams) {
    return fwd ? (bwd ? distill_loop_kernel<BF16, TBF16, I64, true, true> : distill_loop_kernel<BF16, TBF16, I64, true, false>)
               : distill_loop_kernel<BF16, TBF16, I64, false, true>;
}
template <bool BF16>
void (*pick(bool tb, bool i64, bool fwd, bool bwd))(DistillParams) {
    return tb ? (i64 ? pick_dir<BF16, true, true>(fwd, bwd) : pick_dir<BF16, true, false>(fwd, bwd))
              : (i64 ? pick_dir<BF16, false, true>(fwd, bwd) : pick_dir<BF16, false, false>(fwd, bwd));
}

int distill(const void* z, int64_t ldz, int32_t dtype, const void* index, int64_t ldi, int32_t index_bits,
            const void* teacher, int64_t ldt, int32_t t_dtype, int64_t T, int32_t V, int32_t k, float tau,
            const float* lse_in, const float* dloss, float* loss, float* lse, void* dz, int64_t lddz, bool fwd, bool bwd,
            void* stream) {
    if (!dtype_ok(dtype) || !dtype_ok(t_dtype) || (index_bits != 32 && index_bits != 64) || T < 0 || V < 1 || k < 0 ||
        !(tau > 0.0f) || !(tau < 3.0e38f))
        return DDP_ERR_INVALID_ARG;
    const float c = static_cast<float>(1.4426950408889634 / static_cast<double>(tau));
    if (!(c > 1.2e-38f) || !(c < 3.0e38f)) return DDP_ERR_INVALID_ARG;
    if (k > kMaxTop) return DDP_ERR_UNSUPPORTED;
    const int es = dsize(dtype);
    const Mat mz{z, T, V, ldz, es}, mi{index, T, k, ldi, index_bits / 8}, mt{teacher, T, k, ldt, dsize(t_dtype)},
        mli{lse_in, 1, T, T, 4}, mdl{dloss, 1, T, T, 4}, ml{loss, 1, T, T, 4}, mle{lse, 1, T, T, 4},
        md{dz, T, V, lddz, es};
    if (!mat_valid(mz) || !mat_valid(mi) || !mat_valid(mt) || (bwd && !mat_valid(md))) return DDP_ERR_INVALID_ARG;
    if (T > 0 && (z == nullptr || (k > 0 && (index == nullptr || teacher == nullptr)) || (fwd && loss == nullptr) ||
                  (!fwd && lse_in == nullptr) || (bwd && dz == nullptr)))
        return DDP_ERR_INVALID_ARG;
    for (const Mat* m : {&mz, &mi, &mt, &mli, &mdl, &ml, &mle, &md})
        if (!mat_aligned(*m)) return DDP_ERR_ALIGNMENT;
    if (!mats_same(md, mz) && mats_overlap(md, mz)) return DDP_ERR_INVALID_ARG;
    for (const Mat* o : {&ml, &mle, &md})
        for (const Mat* i : {&mi, &mt, &mli, &mdl})
            if (mats_overlap(*o, *i)) return DDP_ERR_INVALID_ARG;
    if (mats_overlap(ml, mz) || mats_overlap(mle, mz) || mats_overlap(ml, mle) || mats_overlap(ml, md) ||
        mats_overlap(mle, md))
        return DDP_ERR_INVALID_ARG;
    if (T == 0) return DDP_OK;
    const DistillParams p{z, index, teacher, lse_in, dloss, loss, lse, dz, ldz, ldi, ldt, lddz, T, V, k, tau, c};
    void (*kernel)(DistillParams) = dtype == DDP_BF16 ? pick<true>(t_dtype == DDP_BF16, index_bits == 64, fwd, bwd)
                                                      : pick<false>(t_dtype == DDP_BF16, index_bits == 64, fwd, bwd);
    const int64_t cap = 1 << 16;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(T < cap ? T : cap)), kDistillThreads,
                      static_cast<cudaStream_t>(stream), p);
}

}  // namespace
}  // namespace ddp

using namespace ddp;

extern "C" int distill_topk_forward(const void* logits, int64_t ldz, int32_t dtype, const void* index, int64_t ldi,
                                    int32_t index_bits, const void* teacher, int64_t ldt, int32_t teacher_dtype,
                                    int64_t T, int32_t V, int32_t k, float temperature, float* loss, float* lse,
                                    void* stream) {
    return distill(logits, ldz, dtype, index, ldi, index_bits, teacher, ldt, teacher_dtype, T, V, k, temperature,
                   nullptr, nullptr, loss, lse, nullptr, 0, true, false, stream);
}

extern "C" int distill_topk_backward(const void* logits, int64_t ldz, int32_t dtype, const void* index, int64_t ldi,
                                     int32_t index_bits, const void* teacher, int64_t ldt, int32_t teacher_dtype,
                                     int64_t T, int32_t V, int32_t k, float temperature, const float* lse,
                                     const float* dloss, void* dlogits, int64_t lddz, void* stream) {
    return distill(logits, ldz, dtype, index, ldi, index_bits, teacher, ldt, teacher_dtype, T, V, k, temperature, lse,
                   dloss, nullptr, nullptr, dlogits, lddz, false, true, stream);
}

extern "C" int distill_topk_forward_backward(const void* logits, int64_t ldz, int32_t dtype, const void* index,
                                             int64_t ldi, int32_t index_bits, const void* teacher, int64_t ldt,
                                             int32_t teacher_dtype, int64_t T, int32_t V, int32_t k,
                                             float temperature, const float* dloss, float* loss, float* lse,
                                             void* dlogits, int64_t lddz, void* stream) {
    return distill(logits, ldz, dtype, index, ldi, index_bits, teacher, ldt, teacher_dtype, T, V, k, temperature,
                   nullptr, dloss, loss, lse, dlogits, lddz, true, true, stream);
}
