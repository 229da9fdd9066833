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
//
// One launch.  A CTA takes a token (a cluster of CTAs, each a slice of the
// vocabulary, when tokens are too few to fill the GPU or too long for the rows
// in hand to stay in L2): one pass over z sums exponentials about a reference
// per thread; the CTA (cluster) joins them; a second pass writes dz =
// dloss·τ·q, reading z again while it is still in L2; last, the at most k
// entries of dz that hold a p are rewritten.  HBM sees z once and dz once:
// 8192 x 50257 bf16, 1.65 GB in 297 us, 0.83 of the copy rate; gradient alone
// 2049 x 32003 46 us, 0.86; loss alone 129 x 50257 fp32 7.4 us.  What bounds it
// is the time a token's dependent steps take (loads, two sums over the CTA,
// loads from L2) with four tokens in hand per SM: more of them miss L2, and rows
// kept in shared memory instead (two per SM) took 373 us.  Rows need not start
// on 16-byte boundaries (an odd vocabulary): a row is its 16-byte vectors and up
// to 2·(VEC − 1) elements at its ends.
#include <cstdint>

#include "rows.cuh"

namespace ddp {
namespace {

constexpr int kDistillThreads = 256;
constexpr int kMaxTop = DDP_DISTILL_MAX_TOP;
constexpr int kTopPerThread = kMaxTop / kDistillThreads;
constexpr int kMaxCluster = 8;
constexpr int kHash = 2 * kMaxTop;
constexpr int kScanTop = 32;          // up to this many entries repeats are found by scanning all pairs
constexpr float kLog2eLow = 1.9259629911e-8f;   // log2(e) − kLog2e
constexpr int64_t kRowsInL2 = 90ll << 20;   // of the rows in hand, so that the second pass finds them there
constexpr float kSlack = 100.0f;      // what lies 2^100 below the token's reference is nothing beside it
constexpr float kHuge = 3.4028235e38f;   // the largest finite number
constexpr float kNear = 4096.0f;      // of m·c: beyond, its spacing is felt beside ln V and ln|dloss|: (z − m)·c then

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
    float tau, c, top;     // c = log2(e) / τ; top·c a little below kNear
    int32_t t_bf16, i_64, cluster;
};

// 2^x; results under 2^-126 are 0.
__device__ __forceinline__ float pow2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint64_t pow2_pair(uint64_t x) {
    float lo, hi;
    unpair(x, lo, hi);
    return pair(pow2(lo), pow2(hi));
}
// The e-th pair of a vector's values.
template <bool BF16>
__device__ __forceinline__ uint64_t vec_pair(const uint4& v, int e) {
    return pair(vec_elem<BF16>(v, 2 * e), vec_elem<BF16>(v, 2 * e + 1));
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float cluster_read(const float* p, uint32_t rank) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
    return v;
}

// Largest m of z, kept finite, and Σ 2^((z − m)·c): of differences, for m·c itself may round by more than any exponent.
struct Running {
    float m = -kHuge, s = 0.0f;
    __device__ __forceinline__ void raise(float to, float c) {
        if (to > m) {
            to = fminf(to, kHuge);
            s *= pow2((m - to) * c);
            m = to;
        }
    }
};

// The slice [v0, v1) of a row, v1 > v0: `lead` elements before its first
// 16-byte boundary, `nvec` whole vectors, `tail` elements after them.
struct Slice {
    const char* base;   // of the row
    int v0, lead, nvec, tail;
};
template <bool BF16>
__device__ __forceinline__ Slice make_slice(const char* row, int v0, int v1) {
    constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES;
    const uintptr_t a = reinterpret_cast<uintptr_t>(row) + static_cast<uintptr_t>(v0) * ES;
    Slice s;
    s.base = row;
    s.v0 = v0;
    s.lead = min(static_cast<int>(((16 - (a & 15)) & 15) / ES), v1 - v0);
    s.nvec = (v1 - v0 - s.lead) / VEC;
    s.tail = v1 - v0 - s.lead - s.nvec * VEC;
    return s;
}
// Index of the slice's e-th element outside its vectors (e < lead + tail).
template <bool BF16>
__device__ __forceinline__ int edge(const Slice& s, int e) {
    return s.v0 + (e < s.lead ? e : e + s.nvec * (BF16 ? 8 : 4));
}

// body(vector index, values) for every 16-byte vector of the slice that is this thread's, U loads in flight.
template <bool BF16, bool KEEP, class F>
__device__ __forceinline__ void each_vector(const Slice& s, F body) {
    constexpr int U = 6;
    const char* zv = s.base + static_cast<int64_t>(s.v0 + s.lead) * (BF16 ? 2 : 4);
    int i = threadIdx.x;
    for (; i + (U - 1) * kDistillThreads < s.nvec; i += U * kDistillThreads) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const char* p = zv + static_cast<int64_t>(i + u * kDistillThreads) * 16;
            v[u] = KEEP ? ld16_keep(p) : ld16<false>(p);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) body(i + u * kDistillThreads, v[u]);
    }
    uint4 v[U - 1];
#pragma unroll
    for (int u = 0; u < U - 1; ++u) {
        const char* p = zv + static_cast<int64_t>(i + u * kDistillThreads) * 16;
        if (i + u * kDistillThreads < s.nvec) v[u] = KEEP ? ld16_keep(p) : ld16<false>(p);
    }
#pragma unroll
    for (int u = 0; u < U - 1; ++u)
        if (i + u * kDistillThreads < s.nvec) body(i + u * kDistillThreads, v[u]);
}

// A vector of dz to an address that is not on 16 bytes.
template <bool BF16>
__device__ __forceinline__ void store_vec_anywhere(char* d, const uint4& w) {
#pragma unroll
    for (int e = 0; e < (BF16 ? 8 : 4); ++e) {
        const int q = BF16 ? e / 2 : e;
        const uint32_t x = q == 0 ? w.x : q == 1 ? w.y : q == 2 ? w.z : w.w;
        if constexpr (BF16) reinterpret_cast<unsigned short*>(d)[e] = static_cast<unsigned short>(x >> (16 * (e & 1)));
        else reinterpret_cast<uint32_t*>(d)[e] = x;
    }
}

// A probability's exponent: a kept lse of far logits, rounded by more than ln V, would allow any number.
__device__ __forceinline__ float at_most_one(float x) { return x > 0.0f ? 0.0f : x; }   // NaN stays

// dz = g·q over a slice; the exponent of q as FAR says.  A bf16 dz has |g| in the exponent and its sign set
// afterwards; an fp32 dz keeps them apart, for the larger exponent would round more.
template <bool BF16, bool FAR, bool KEEP>
__device__ __forceinline__ void write_grad(const Slice& s, char* dz, float c, float M, float m, float ls, float g, bool has_edge, int ve, float xe) {
    constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES;
    const float lg = log2f(fabsf(g)), off = M + ls - lg;
    const uint32_t sign = BF16 && g < 0.0f ? 0x80008000u : 0u;
    const uint64_t c2 = pair(c, c), n2 = pair(-off, -off);
    auto f = [&](float z) {
        if constexpr (FAR) {
            const float x = at_most_one((z - m) * c - ls);
            return BF16 ? pow2(x + lg) : g * pow2(x);
        } else {
            return BF16 ? pow2(fmaf(z, c, -off)) : g * pow2(fmaf(z, c, -M) - ls);
        }
    };
    char* dv = dz + static_cast<int64_t>(s.v0 + s.lead) * ES;
    const bool whole = (reinterpret_cast<uintptr_t>(dv) & 15) == 0;
    each_vector<BF16, KEEP>(s, [&](int i, const uint4& v) {
        float o[VEC];
        uint4 w;
        if constexpr (BF16 && !FAR) {
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) unpair(pow2_pair(fma2(vec_pair<BF16>(v, e), c2, n2)), o[2 * e], o[2 * e + 1]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = f(vec_elem<BF16>(v, e));
        }
        if constexpr (BF16) w = make_uint4(pack2(o[0], o[1]) ^ sign, pack2(o[2], o[3]) ^ sign, pack2(o[4], o[5]) ^ sign, pack2(o[6], o[7]) ^ sign);
        else w = f4_bits(o[0], o[1], o[2], o[3]);
        if (whole) st16(dv + static_cast<int64_t>(i) * 16, w);
        else store_vec_anywhere<BF16>(dv + static_cast<int64_t>(i) * 16, w);
    });
    if (has_edge) {
        const float o = f(xe);
        store_elem<BF16>(dz, ve, BF16 && g < 0.0f ? -o : o);
    }
}

template <bool BF16>
__device__ __forceinline__ void write_zero(const Slice& s, char* dz) {
    constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES;
    char* dv = dz + static_cast<int64_t>(s.v0 + s.lead) * ES;
    const bool whole = (reinterpret_cast<uintptr_t>(dv) & 15) == 0;
    for (int i = threadIdx.x; i < s.nvec; i += kDistillThreads) {
        if (whole) {
            st16(dv + static_cast<int64_t>(i) * 16, make_uint4(0, 0, 0, 0));
        } else {
            for (int e = 0; e < VEC; ++e) store_elem<BF16>(dv, static_cast<int64_t>(i) * VEC + e, 0.0f);
        }
    }
    if (threadIdx.x < s.lead + s.tail) store_elem<BF16>(dz, edge<BF16>(s, threadIdx.x), 0.0f);
}

// Two values over the CTA, in every thread, with one barrier: `sh` is not used again before another.
template <class OpA, class OpB>
__device__ __forceinline__ void once_all2(float& a, float& b, float2* sh) {
    a = warp_all<OpA>(a);
    b = warp_all<OpB>(b);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 v = (threadIdx.x & 31) < kDistillThreads / 32 ? sh[threadIdx.x & 31] : make_float2(OpA::id(), OpB::id());
    a = warp_all<OpA>(v.x);
    b = warp_all<OpB>(v.y);
}

template <bool BF16, bool FWD, bool BWD>
__global__ void __launch_bounds__(kDistillThreads, 4) distill_kernel(const __grid_constant__ DistillParams a) {
    constexpr int VEC = BF16 ? 8 : 4;
    __shared__ float2 sh[2][kDistillThreads / 32];
    __shared__ float s_part[2];                      // this CTA's (m, s), read by its cluster
    __shared__ float s_loss[kDistillThreads / 32];
    __shared__ int s_idx[BWD ? kMaxTop : 1];
    __shared__ float s_p[BWD ? kMaxTop : 1];
    __shared__ int s_hash[BWD ? kHash : 1];
    __shared__ int s_twice;
    pdl_enter();
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.cluster;
    const int rank = blockIdx.x % a.cluster;
    const char* z = row_ptr<BF16>(a.z, row, a.ldz);
    // slices of whole 256-byte lines of the row's own grid
    const int per = ((a.V + a.cluster - 1) / a.cluster + 127) / 128 * 128;
    const int v0 = min(a.V, rank * per), v1 = min(a.V, v0 + per);
    const Slice s = make_slice<BF16>(z, v0, v1);

    // The teacher's entries: on their way during the pass over z, looked at after it.
    int64_t raw[kTopPerThread];
    float t[kTopPerThread];
#pragma unroll
    for (int u = 0; u < kTopPerThread; ++u) {
        const int j = tid + u * kDistillThreads;
        raw[u] = -1;
        t[u] = -INFINITY;
        if (j >= a.k) continue;
        const int64_t e = row * a.ldi + j;
        raw[u] = a.i_64 ? static_cast<const int64_t*>(a.index)[e] : static_cast<int64_t>(static_cast<const int32_t*>(a.index)[e]);
        t[u] = a.t_bf16 ? load_elem<true>(row_ptr<true>(a.teacher, row, a.ldt), j)
                        : load_elem<false>(row_ptr<false>(a.teacher, row, a.ldt), j);
    }
    const float up = BWD && a.dloss ? a.dloss[row] : 1.0f;
    const float lse_in = FWD ? 0.0f : a.lse_in[row];
    const bool has_edge = tid < s.lead + s.tail;
    const int ve = has_edge ? edge<BF16>(s, tid) : 0;
    const float xe = has_edge ? load_elem<BF16>(z, ve) : 0.0f;
    const bool hash = a.k > kScanTop;
    if constexpr (BWD) {
        if (hash)
            for (int i = tid; i < kHash; i += kDistillThreads) s_hash[i] = -1;
        if (tid == 0) s_twice = hash ? 0 : 1;
    }

    // The sum takes no maximum: fp32 holds 2^±126 about any reference near the thread's logits, and the first of its
    // vectors that is not masked (top·c > −kNear) gives one; its own top then makes the sum about 1 or more, so that
    // what the join drops, under 2^-126 of at most 1e18, is nothing beside it.  Masked vectors before it add 0:
    // the token's reference, once known, says whether they count.  A token that a thread's sum leaves that range for
    // (logits 40 nats above the reference), or whose reference is itself near the masks, is summed again with a
    // running maximum.
    float ref = -INFINITY, mc = 0.0f, part = 0.0f;      // reference (without one the largest masked logit), ref·c, sum
    bool out = false;
    if constexpr (FWD) {
        const uint64_t c2 = pair(a.c, a.c);
        uint64_t s2 = 0, n2 = 0;
        bool begun = false;
        auto begin = [&](float top) {
            if (top * a.c <= -kNear) {                   // not a NaN
                ref = fmaxf(ref, top);
                return false;
            }
            ref = fminf(top, a.top);
            mc = __fmul_rn(ref, a.c);
            n2 = pair(-mc, -mc);
            return true;
        };
        each_vector<BF16, true>(s, [&](int, const uint4& v) {
            if (!begun) {
                float top = vec_elem<BF16>(v, 0);
#pragma unroll
                for (int e = 1; e < VEC; ++e) top = max_nan(top, vec_elem<BF16>(v, e));
                begun = begin(top);                      // else n2 is 0, and 2^(z·c) as well
            }
            uint64_t v2 = pow2_pair(fma2(vec_pair<BF16>(v, 0), c2, n2));
#pragma unroll
            for (int e = 1; e < VEC / 2; ++e) v2 = add2(v2, pow2_pair(fma2(vec_pair<BF16>(v, e), c2, n2)));
            s2 = add2(s2, v2);
        });
        float s_lo, s_hi;
        unpair(s2, s_lo, s_hi);
        part = s_lo + s_hi;
        if (has_edge && (begun || (begun = begin(xe)))) part += pow2(fmaf(xe, a.c, -mc));
        out = begun && !(part > 0.5f && part < 1.0e18f);
    }

    // what the entries are, and the logits at those that this CTA writes or sums (another's slice may hold gradients)
    int idx[kTopPerThread];
    float zi[kTopPerThread];
    float tm = -INFINITY;
#pragma unroll
    for (int u = 0; u < kTopPerThread; ++u) {
        const bool in = raw[u] >= 0 && raw[u] < a.V;
        idx[u] = in ? static_cast<int>(raw[u]) : -1;
        if (!in) t[u] = -INFINITY;
        zi[u] = in && ((FWD && rank == 0) || (idx[u] >= v0 && idx[u] < v1)) ? load_elem<BF16>(z, idx[u]) : 0.0f;
        tm = max_nan(tm, t[u]);
    }

    // maxima of the logits and of the entries, then their sums
    float m = out ? INFINITY : ref;
    once_all2<MaxOp, MaxNanOp>(m, tm, sh[0]);
    bool diff = false;                                   // sums are of 2^((z − m)·c), not of 2^(z·c − M)
    if constexpr (FWD) {
        diff = m == INFINITY || (m * a.c <= kSlack - kNear && m > -INFINITY);
        if (diff) {                                      // again, with a running maximum
            Running run;
            each_vector<BF16, true>(s, [&](int, const uint4& v) {
                float top = -INFINITY;
#pragma unroll
                for (int e = 0; e < VEC; ++e) top = fmaxf(top, vec_elem<BF16>(v, e));
                run.raise(top, a.c);
#pragma unroll
                for (int e = 0; e < VEC; ++e) run.s += pow2((vec_elem<BF16>(v, e) - run.m) * a.c);
            });
            if (has_edge) {
                run.raise(xe, a.c);
                run.s += pow2((xe - run.m) * a.c);
            }
            m = run.m;
            float none = 0.0f;
            __syncthreads();
            once_all2<MaxOp, SumOp>(m, none, sh[0]);
            part = run.s * pow2((run.m - m) * a.c);
        } else {
            m = fmaxf(m, -kHuge);
            part = part == 0.0f ? 0.0f : part * pow2(mc - __fmul_rn(m, a.c));
        }
    }
    const bool some = !(tm == -INFINITY);
    float ts = 0.0f;
#pragma unroll
    for (int u = 0; u < kTopPerThread; ++u) ts += some && idx[u] >= 0 ? pow2((t[u] - tm) * a.c) : 0.0f;
    if constexpr (BWD) {                                 // repeated indices: seen where two entries meet in a slot
        if (hash) {
#pragma unroll
            for (int u = 0; u < kTopPerThread; ++u) {
                if (idx[u] < 0) continue;
                for (uint32_t h = (static_cast<uint32_t>(idx[u]) * 2654435761u) >> 21;; h = (h + 1) & (kHash - 1)) {
                    const int old = atomicCAS(&s_hash[h], -1, idx[u]);
                    if (old == idx[u]) s_twice = 1;
                    if (old == -1 || old == idx[u]) break;
                }
            }
        }
    }
    float sum = part;
    once_all2<SumOp, SumOp>(sum, ts, sh[1]);
    float M = __fmul_rn(m, a.c);
    if constexpr (FWD) {
        if (a.cluster > 1) {
            if (tid == 0) {
                s_part[0] = m;
                s_part[1] = diff || sum == 0.0f ? sum : sum * pow2(-fmaf(m, a.c, -M));
            }
            cluster_sync();
            float pm[kMaxCluster], ps[kMaxCluster];
            m = -kHuge;
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                pm[r] = r < a.cluster ? cluster_read(&s_part[0], r) : -kHuge;
                ps[r] = r < a.cluster ? cluster_read(&s_part[1], r) : 0.0f;
                m = fmaxf(m, pm[r]);
            }
            sum = 0.0f;
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) sum += ps[r] * pow2((pm[r] - m) * a.c);
            M = __fmul_rn(m, a.c);
            diff = true;
        }
    } else {
        M = lse_in * kLog2e;                             // with what the product rounds off, below
        m = fminf(fmaxf(lse_in * a.tau, -kHuge), kHuge);
    }
    // Logits far from 0 beside the temperature (a row that a finite mask leaves whole): differences first.  m is finite,
    // so that an lse of ±infinity lies in ls: q is 0 at every finite logit, and NaN at one that is infinite as it is.
    const bool far = !(fabsf(M) <= kNear);
    // q_v = 2^(z·c − M − ls), far: 2^((z − m)·c − ls); of a kept lse, ls is what rounding M or m left
    const float ls = FWD ? log2f(sum) + (diff && !far ? fmaf(m, a.c, -M) : 0.0f)
                         : far ? fmaf(lse_in, a.tau, -m) * a.c : fmaf(lse_in, kLog2e, -M) + lse_in * kLog2eLow;
    auto q2 = [&](float x) { return far ? at_most_one((x - m) * a.c - ls) : fmaf(x, a.c, -M) - ls; };
    if constexpr (FWD) {
        if (rank == 0) {
            const float lts = log2f(ts);
            float l = 0.0f;
#pragma unroll
            for (int u = 0; u < kTopPerThread; ++u) {
                const float lp = (t[u] - tm) * a.c, p = some && idx[u] >= 0 ? pow2(lp) / ts : 0.0f;
                if (p != 0.0f) l += p * (lp - lts - q2(zi[u]));
            }
            l = warp_all<SumOp>(l);
            if ((tid & 31) == 0) s_loss[tid >> 5] = l;
        }
    }
    if constexpr (BWD) {
        const float g = up * a.tau;
        char* dz = row_ptr<BF16>(a.dz, row, a.lddz);
        const bool zero = !some || g == 0.0f;
        if (zero) write_zero<BF16>(s, dz);
        else if (far) write_grad<BF16, true, !FWD>(s, dz, a.c, M, m, ls, g, has_edge, ve, xe);
        else write_grad<BF16, false, !FWD>(s, dz, a.c, M, m, ls, g, has_edge, ve, xe);
#pragma unroll
        for (int u = 0; u < kTopPerThread; ++u) {
            const int j = tid + u * kDistillThreads;
            if (j >= a.k) continue;
            s_idx[j] = idx[u];
            s_p[j] = idx[u] >= 0 ? pow2((t[u] - tm) * a.c) / ts : 0.0f;
        }
        __syncthreads();                                 // before the entries are rewritten
        if (!zero) {
            const bool twice = s_twice != 0;
#pragma unroll
            for (int u = 0; u < kTopPerThread; ++u) {
                const int j = tid + u * kDistillThreads, i = idx[u];
                if (i < v0 || i >= v1) continue;         // absent ones are negative
                float p = twice ? 0.0f : s_p[j];
                bool first = true;
                if (twice) {
                    for (int w = 0; w < a.k; ++w) {
                        if (s_idx[w] != i) continue;
                        if (w < j) first = false;
                        p += s_p[w];
                    }
                }
                if (first) store_elem<BF16>(dz, i, g * (pow2(q2(zi[u])) - p));
            }
        }
    } else {
        __syncthreads();
    }
    if constexpr (FWD) {
        if (rank == 0 && tid == 0) {
            float l = 0.0f;
#pragma unroll
            for (int w = 0; w < kDistillThreads / 32; ++w) l += s_loss[w];
            a.loss[row] = some ? l * kLn2 * a.tau * a.tau : 0.0f;
            if (a.lse) a.lse[row] = far ? m / a.tau + ls * kLn2 : (M + ls) * kLn2;
        }
        if (a.cluster > 1) cluster_sync();               // no CTA ends while another reads its part
    }
}

bool dtype_ok(int32_t t) { return t == DDP_F32 || t == DDP_BF16; }
int dsize(int32_t t) { return t == DDP_BF16 ? 2 : 4; }

template <bool BF16>
void (*pick(bool fwd, bool bwd))(DistillParams) {
    return fwd ? (bwd ? distill_kernel<BF16, true, true> : distill_kernel<BF16, true, false>) : distill_kernel<BF16, false, true>;
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
    if (k > kMaxTop || V > kMaxWidth) return DDP_ERR_UNSUPPORTED;
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
    DeviceInfo d;
    int st = current_device_info(&d);
    if (st != DDP_OK) return st;
    // one CTA per token fills the GPU from about two CTAs per SM; fewer tokens are split into slices of at least
    // 2048 logits each
    int cluster = 1;
    while (cluster < kMaxCluster && V / (2 * cluster) >= 2048 &&
           (T * cluster < 2ll * d.sm_count || (fwd && bwd && 4ll * d.sm_count / cluster * V * es > kRowsInL2)))
        cluster *= 2;
    if (T * cluster > INT32_MAX) return DDP_ERR_UNSUPPORTED;
    const DistillParams p{z, index, teacher, lse_in, dloss, loss, lse, dz, ldz, ldi, ldt, lddz, T, V, k, tau, c,
                          fminf(0.999f * kNear / c, kHuge), t_dtype == DDP_BF16, index_bits == 64, cluster};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(T * cluster));
    cfg.blockDim = dim3(kDistillThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, dtype == DDP_BF16 ? pick<true>(fwd, bwd) : pick<false>(fwd, bwd), p);
    return e == cudaSuccess ? check_launch() : cuda_fail(e);
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
