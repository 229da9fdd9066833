// Shared by the operators over a vocabulary (distillation loss, token log
// probabilities): a token's row of logits, or a slice of it, as 16-byte vectors
// and the elements at its ends, exponentials, and reads across a cluster.
#pragma once

#include <cstdint>

#include "rows.cuh"

namespace ddp {

constexpr int kVocabThreads = 256;
constexpr int kMaxCluster = 8;
constexpr float kLog2eLow = 1.9259629911e-8f;   // log2(e) − kLog2e
constexpr float kHuge = 3.4028235e38f;   // the largest finite number

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
template <bool BF16, bool KEEP, int U = 6, class F>
__device__ __forceinline__ void each_vector(const Slice& s, F body) {
    const char* zv = s.base + static_cast<int64_t>(s.v0 + s.lead) * (BF16 ? 2 : 4);
    int i = threadIdx.x;
    for (; i + (U - 1) * kVocabThreads < s.nvec; i += U * kVocabThreads) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const char* p = zv + static_cast<int64_t>(i + u * kVocabThreads) * 16;
            v[u] = KEEP ? ld16_keep(p) : ld16<false>(p);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) body(i + u * kVocabThreads, v[u]);
    }
    uint4 v[U - 1];
#pragma unroll
    for (int u = 0; u < U - 1; ++u) {
        const char* p = zv + static_cast<int64_t>(i + u * kVocabThreads) * 16;
        if (i + u * kVocabThreads < s.nvec) v[u] = KEEP ? ld16_keep(p) : ld16<false>(p);
    }
#pragma unroll
    for (int u = 0; u < U - 1; ++u)
        if (i + u * kVocabThreads < s.nvec) body(i + u * kVocabThreads, v[u]);
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

template <bool BF16>
__device__ __forceinline__ void write_zero(const Slice& s, char* dz) {
    constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES;
    char* dv = dz + static_cast<int64_t>(s.v0 + s.lead) * ES;
    const bool whole = (reinterpret_cast<uintptr_t>(dv) & 15) == 0;
    for (int i = threadIdx.x; i < s.nvec; i += kVocabThreads) {
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
    const float2 v = (threadIdx.x & 31) < kVocabThreads / 32 ? sh[threadIdx.x & 31] : make_float2(OpA::id(), OpB::id());
    a = warp_all<OpA>(v.x);
    b = warp_all<OpB>(v.y);
}

}  // namespace ddp
