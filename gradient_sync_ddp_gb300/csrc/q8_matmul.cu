// Product of 8-bit integers with a scale for each token and each channel:
//   out[m, n] = (Σ_k a[m, k]·w[n, k]) · a_scale[m] · w_scale[n]
//
// Up to kFewTokens tokens: the channels are streamed once and multiplied into
// exact 32-bit integers, with dp4a (few_kernel) or, from 3 tokens on, the
// warp-wide 8-bit tensor instruction (few_mma_kernel).  Bound by HBM (1 token,
// 8192 x 4096: 33.6 MB in 6.4 us; 16384 x 8192: 22 us, 0.91 of the copy rate;
// of 50257 x 768 8.2 us, 0.71: its 1571 groups of channels are 2.07 rounds of
// the 760 CTAs that are resident, so a third one is nearly empty), or by loads and that instruction taking turns (8
// tokens, 8192 x 4096: 9.9 us, where bytes need 5.0 and the instruction 6.0).
//
// More tokens: GB300's tensor cores run 8-bit integers far below their 16-bit
// rate, and an 8-bit integer is exact in fp16, as is a product of two in
// fp32, so the product runs as an fp16 tcgen05 contraction with fp32
// accumulators (exact while partial sums stay below 2^24, always for
// K <= 1024; beyond that each 16-wide step of K rounds once).  Computed as
// its transpose, D[n, m]: channels are the 128-row operand, tokens the wide one.
//   widen_kernel   tokens to fp16 in the workspace (channels whose rows TMA
//                  cannot address are repacked there too, still in 8 bits)
//   tile_kernel    persistent, a pair of CTAs (two SMs) per tile of 256
//                  channels x NT <= 256 tokens, roles by warp in each CTA:
//     two producers  TMA, 128 of K at a time: the CTA's half of the tokens
//                    [2 x 64][NT/2] fp16 and its 128 channels [128][128] int8
//                    (both in the 128-byte swizzle), each into its own ring
//     converters     two warpgroups, a channel row per thread, each its half
//                    of the 128: 64 bytes from shared memory, widened in
//                    registers, stored to TMEM; channels thus cost 8 bits of
//                    L2 and shared memory
//     one issuer     (of the pair's first CTA) tcgen05.mma.cta_group::2, A
//                    from TMEM, B from shared memory, fp32 accumulator in TMEM
//     epilogue       two warpgroups: TMEM -> scales -> out, 64 columns at a
//                    time; the accumulator is free before the last are stored
// 8192 x 16384 x 4096: 545-564 us in bursts, 609-622 held (the clock falls): 2.0
// and 1.8 PFLOP/s, 1.05 and 0.93 of the 16-bit rate measured with cuBLAS.  What
// that took, each by its measurement: 64-token-deep tiles of one CTA 870 us,
// held by L2 -> SM traffic (65 bytes per clock and SM); the pair halves what
// tokens cost; arrivals across the pair without release (1438 -> 1063); one
// commit per stage (845 -> 753); token scales staged for the epilogue (-> 715);
// NT = 256 with one accumulator, for a 192-wide MMA took as long as a 256-wide
// one (-> 620); the issuing warp converged, descriptors in uniform registers:
// 130 -> 45 clocks to issue an MMA (-> 562).
// Few tiles split K (the parts are fp32 in the workspace, combine_kernel adds
// them in their order).  37 x 8192 x 4096: 16.0 us, bound by the steps of the
// pipeline itself: launches and TMEM 6 us, then a stage at about 850 clocks of
// barriers (12.6 us of 16.3 were left without loads, conversions and MMAs, with
// one block of K a stage; narrow tiles take two).  1.2 us of it are the wait of
// all threads for the tokens' grid, without which channels and scales could be
// read before an earlier call's writes are visible.
// Every wait on a barrier is bounded; a tile whose wait ran out is written as NaN.
#include <cstdint>

#include <cuda.h>
#include <cuda_fp16.h>

#include "rows.cuh"

namespace ddp {
namespace {

constexpr int kMaxK = 131071;     // |Σ| < 2^31
constexpr int kFewTokens = 8;
constexpr int kCtaN = 128;        // channels per CTA; 256 per pair: the MMA's rows
constexpr int kMaxNT = 256;       // tokens per tile: an accumulator of 256 columns + 4 channel stages of 64 = 512
constexpr int kBlockK = 128;      // a block of K; a stage of the rings is one, or two for narrow tiles
constexpr int kHalfK = 64;        // a row of 128 bytes in fp16
constexpr int kWBlockBytes = kCtaN * kBlockK;
constexpr int kMaxAStages = 4;      // stages of channels in TMEM, 64 columns each; at most the rings' stages
constexpr int kMaxStages = 4;        // narrow tiles: more cost time (37 x 8192 x 4096, one block a stage: 15.9 us with 5, 16.3 with 12)
constexpr int kRingBytes = 212 * 1024;
// A tile CTA takes all of its SM's TMEM, so never two on one SM: each asks for more than half of the shared memory.
constexpr size_t kMinTileSmem = 128 * 1024;
constexpr int kTileThreads = 640;  // 4 warps of single roles, 8 of the epilogue, 8 converters
constexpr long long kWaitClocks = 2000000000ll;   // about a second (clock64: the nanosecond timer is slow to read)

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// ---- few tokens ---------------------------------------------------------

struct FewParams {
    const int8_t* a;
    const int8_t* w;
    const float* sa;
    const float* sw;
    void* out;
    int64_t lda, ldw, ldo, N;
    int32_t K, M;
    int32_t w_align, a_align;   // 16, 4 or 1: what the rows' addresses are multiples of
    int32_t split;              // mma_kernel: warps that share 16 channels, a power of two up to kFewWarps
};

// 16 bytes at p of which the first `valid` exist, the others read as 0; KEEP: the caches keep them.
template <bool KEEP>
__device__ __forceinline__ int4 load16_any(const int8_t* p, int valid, int align) {
    if (valid >= 16 && align == 16) {
        if constexpr (KEEP) return __ldg(reinterpret_cast<const int4*>(p));
        const uint4 v = ld16<true>(p);
        return make_int4(static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w));
    }
    int r[4] = {0, 0, 0, 0};
    if (valid >= 16 && align == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = __ldg(reinterpret_cast<const int*>(p) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < valid) r[i >> 2] |= static_cast<int>(static_cast<uint32_t>(static_cast<uint8_t>(p[i])) << (8 * (i & 3)));
    }
    return make_int4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ int4 load16(const int8_t* p, int valid, int align) { return load16_any<false>(p, valid, align); }
__device__ __forceinline__ int4 load16_keep(const int8_t* p, int valid, int align) { return load16_any<true>(p, valid, align); }

constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;
constexpr int kFewChunk = 4096;   // bytes of K of every token in shared memory at a time

// LPR lanes per channel row, R rows per lane group at a time, U vectors of
// each in flight: R·U·16 bytes per lane.
template <int M, int LPR, int R, int U, bool BF16>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const __grid_constant__ FewParams p) {
    extern __shared__ int4 tok[];   // [M][chunk / 16]
    pdl_enter();
    constexpr int GROUPS = kFewThreads / LPR;
    const int g = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int chunk_vec = min(kFewChunk, (p.K + 15) / 16 * 16) / 16;
    const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS * R, begin = static_cast<int64_t>(blockIdx.x) * GROUPS * R;
    for (int64_t n0 = begin; n0 < p.N; n0 += step) {
        int acc[R][M] = {};
        for (int k0 = 0; k0 < p.K; k0 += kFewChunk) {
            const int kn = min(kFewChunk, p.K - k0), nv = (kn + 15) / 16;
            auto fetch = [&](int v, int4 (&w)[R]) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int64_t n = n0 + g + static_cast<int64_t>(r) * GROUPS;
                    w[r] = n < p.N && v < nv ? load16(p.w + n * p.ldw + k0 + 16 * v, kn - 16 * v, p.w_align) : make_int4(0, 0, 0, 0);
                }
            };
            int4 w[U][R];                       // the first channels are on their way before the tokens are staged
#pragma unroll
            for (int u = 0; u < U; ++u) fetch(l + u * LPR, w[u]);
            if (p.K > kFewChunk || n0 == begin) {
                __syncthreads();
                for (int i = threadIdx.x; i < M * nv; i += kFewThreads) {
                    const int m = i / nv, v = i - m * nv;
                    tok[m * chunk_vec + v] = load16(p.a + m * p.lda + k0 + 16 * v, kn - 16 * v, p.a_align);
                }
                __syncthreads();
            }
            for (int v0 = l;; ) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int v = v0 + u * LPR;
                    if (v >= nv) break;
#pragma unroll
                    for (int m = 0; m < M; ++m) {
                        const int4 t = tok[m * chunk_vec + v];
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            acc[r][m] = __dp4a(w[u][r].x, t.x, acc[r][m]);
                            acc[r][m] = __dp4a(w[u][r].y, t.y, acc[r][m]);
                            acc[r][m] = __dp4a(w[u][r].z, t.z, acc[r][m]);
                            acc[r][m] = __dp4a(w[u][r].w, t.w, acc[r][m]);
                        }
                    }
                }
                v0 += U * LPR;
                if (v0 >= nv) break;
#pragma unroll
                for (int u = 0; u < U; ++u) fetch(v0 + u * LPR, w[u]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t n = n0 + g + static_cast<int64_t>(r) * GROUPS;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                int s = acc[r][m];
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (l == m % LPR && n < p.N)
                    store_elem<BF16>(p.out, m * p.ldo + n, static_cast<float>(s) * p.sa[m] * p.sw[n]);
            }
        }
    }
}

__device__ __forceinline__ void mma_s8(int (&c)[4], int a0, int a1, int a2, int a3, int b0, int b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp takes 16 channels and every SK-th block of 64 of K, up to 8 tokens, U
// blocks in flight.  The sum over k does not care in which order k goes as long
// as both operands agree, so a lane's 16 bytes of a row are the words of two
// MMAs as they come from memory: no shared memory, no shuffles.
template <bool BF16>
__global__ void __launch_bounds__(kFewThreads) few_mma_kernel(const __grid_constant__ FewParams p) {
    constexpr int U = 3;
    __shared__ int part[kFewWarps][4][32];
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int sk = p.split, s = warp % sk;
    const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * (kFewWarps / sk) + warp / sk) * 16;
    const int64_t na = n0 + g, nb = na + 8;
    const int8_t* wa = p.w + na * p.ldw + 16 * q;
    const int8_t* wb = p.w + nb * p.ldw + 16 * q;
    const int8_t* ta = p.a + g * p.lda + 16 * q;
    int acc[4] = {};
    const int blocks = (p.K + 63) / 64;
    const int4 zero = make_int4(0, 0, 0, 0);
    for (int b0 = s; b0 < blocks; b0 += U * sk) {
        int4 a[U], b[U], t[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (b0 + u * sk) * 64, valid = p.K - k - 16 * q;
            a[u] = na < p.N && valid > 0 ? load16(wa + k, valid, p.w_align) : zero;
            b[u] = nb < p.N && valid > 0 ? load16(wb + k, valid, p.w_align) : zero;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (b0 + u * sk) * 64, valid = p.K - k - 16 * q;
            t[u] = g < p.M && valid > 0 ? load16_keep(ta + k, valid, p.a_align) : zero;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mma_s8(acc, a[u].x, b[u].x, a[u].y, b[u].y, t[u].x, t[u].y);
            mma_s8(acc, a[u].z, b[u].z, a[u].w, b[u].w, t[u].z, t[u].w);
        }
    }
    if (sk > 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) part[warp][j][lane] = acc[j];
        __syncthreads();
        if (s != 0) return;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            for (int w = 1; w < sk; ++w) acc[j] += part[warp + w][j][lane];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int m = 2 * q + (j & 1);
        const int64_t n = j < 2 ? na : nb;
        if (m < p.M && n < p.N) store_elem<BF16>(p.out, m * p.ldo + n, static_cast<float>(acc[j]) * p.sa[m] * p.sw[n]);
    }
}

// ---- tokens to fp16, unaligned channels to a 16-byte pitch ---------------

struct WidenParams {
    const int8_t* a;
    __half* x;         // [M][xp]
    const int8_t* w;
    int8_t* wr;        // [N][wp] or NULL
    int64_t lda, ldw, M, N, xp, wp;
    int32_t K, a_align;
};

__device__ __forceinline__ void widen4(uint32_t v, uint32_t& lo, uint32_t& hi) {
    // byte b + 128 behind the exponent of 1024 is fp16 1152 + b; 1152 is exact, so the difference is b
    const uint32_t u = v ^ 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t l = __byte_perm(u, 0x64646464u, 0x4140), h = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&l), off), y = __hsub2(*reinterpret_cast<__half2*>(&h), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

// Lets the tile kernel begin once everything before this kernel is done: its
// CTAs set up their barriers and TMEM while tokens are widened.
__global__ void __launch_bounds__(kThreads) widen_kernel(const __grid_constant__ WidenParams p) {
    pdl_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t av = (p.xp + 15) / 16;
    for (int64_t i = first; i < p.M * av; i += stride) {
        const int64_t m = i / av, v = i - m * av;
        const int4 t = load16(p.a + m * p.lda + 16 * v, static_cast<int>(p.K - 16 * v), p.a_align);
        uint4 q[2];
        widen4(t.x, q[0].x, q[0].y);
        widen4(t.y, q[0].z, q[0].w);
        widen4(t.z, q[1].x, q[1].y);
        widen4(t.w, q[1].z, q[1].w);
        uint4* d = reinterpret_cast<uint4*>(p.x + m * p.xp + 16 * v);
        d[0] = q[0];
        if (16 * v + 8 < p.xp) d[1] = q[1];
    }
    if (p.wr == nullptr) return;
    const int64_t wv = p.wp / 16;
    for (int64_t i = first; i < p.N * wv; i += stride) {
        const int64_t n = i / wv, v = i - n * wv;
        *reinterpret_cast<int4*>(p.wr + n * p.wp + 16 * v) = load16(p.w + n * p.ldw + 16 * v, static_cast<int>(p.K - 16 * v), 1);
    }
}

// ---- tensor core tiles ---------------------------------------------------

struct TileParams {
    CUtensorMap tx, tw;
    const float* sa;
    const float* sw;
    void* out;       // or the parts, float [splits][M][N]
    int64_t ldo;
    int32_t M, N, halves, nt, m_tiles, n_tiles, group, splits, stages_per_split, stages, a_stages, d_stages, subs;   // subs: blocks per stage
};

struct TileShared {
    uint64_t w_full[kMaxStages], w_empty[kMaxStages];
    uint64_t ready[kMaxStages];  // of the first CTA: both CTAs' tokens are in shared memory, their channels in TMEM
    uint64_t done[kMaxStages];   // a stage's MMAs: its tokens and its channels in TMEM may be overwritten
    uint64_t d_full[2], d_empty[2], idle;
    alignas(16) float sa[8][kMaxNT / 2];     // token scales of each epilogue warp's columns
    uint32_t tmem;
    volatile int failed;
};

__device__ __forceinline__ void bar_init(uint64_t* b, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
// The barrier of the pair's first CTA at the place of this CTA's.
__device__ __forceinline__ uint32_t first_of_pair(uint64_t* b) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(b)));
    return r;
}
// Arrive on it.  Relaxed, so only for reads and writes of TMEM, which the tcgen05 fences about the arrival order.
__device__ __forceinline__ void bar_arrive_first(uint64_t* b) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(first_of_pair(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_poll(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
// For what the other CTA of the pair announces.
__device__ __forceinline__ bool bar_poll_pair(uint64_t* b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool bar_wait_pair(uint64_t* b, uint32_t parity, TileShared& s) {
    const long long t0 = clock64();
    while (!bar_poll_pair(b, parity)) {
        if (s.failed) return false;
        if (clock64() - t0 > kWaitClocks) {
            s.failed = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool bar_test_pair(uint64_t* b, uint32_t parity) {   // does not wait
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Wait for the phase of `parity`; false once a wait of this CTA has run out.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, TileShared& s) {
    if (bar_poll(b, parity)) return true;
    const long long t0 = clock64();
    while (!bar_poll(b, parity)) {
        if (s.failed) return false;
        if (clock64() - t0 > kWaitClocks) {
            s.failed = 1;
            return false;
        }
    }
    return true;
}
// The same for work of this CTA that is still in flight when it ends, whether or not a wait has run out before.
__device__ __forceinline__ void bar_drain(uint64_t* b, uint32_t parity, TileShared& s) {
    const long long t0 = clock64();
    while (!bar_poll(b, parity)) {
        if (clock64() - t0 > kWaitClocks) {
            s.failed = 1;
            return;
        }
    }
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// Into this CTA's shared memory, told to a barrier of either CTA of the pair: the copy itself orders its bytes before
// the arrival.  A thread that waits for the copy and arrives with a release takes 8192 x 16384 x 4096 from 553 to 729 us.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Shared-memory operand, K-major rows of 128 bytes in the 128-byte swizzle: 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
}
// The barrier arrives when the MMAs issued so far are done: that of the first CTA, and with BOTH that of the second at
// the same place.  An arrival is under way until a thread of its CTA has seen it, so each is waited for there.
template <bool BOTH = true>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(BOTH ? 3 : 1))
        : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Position of a ring: index and phase parity.
struct Ring {
    int i = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) {
            i = 0;
            ph ^= 1;
        }
    }
    __device__ __forceinline__ void back(int n) {
        if (i == 0) {
            i = n;
            ph ^= 1;
        }
        --i;
    }
};

// The u-th piece of work: a tile and a range of K blocks.  Tiles go in groups
// of `group` token tiles, channels outer within a group, so that the pairs
// running at a time share both operands in L2.
struct Piece {
    int m0, n0, split, h0, h1;   // tokens, channels, part of K, halves of 64 of K
};
__device__ __forceinline__ Piece piece(const TileParams& p, int u) {
    Piece w;
    w.split = u % p.splits;
    const int t = u / p.splits, per_group = p.group * p.n_tiles, g = t / per_group, r = t - g * per_group;
    const int wide = min(p.group, p.m_tiles - g * p.group);
    w.n0 = r / wide * 2 * kCtaN;
    w.m0 = (g * p.group + r % wide) * p.nt;
    w.h0 = w.split * p.stages_per_split * 2 * p.subs;
    w.h1 = min(p.halves, w.h0 + p.stages_per_split * 2 * p.subs);
    return w;
}

enum { kTileF32 = 0, kTileBf16 = 1, kTilePart = 2 };

template <int OUT>
__global__ void __launch_bounds__(kTileThreads, 1) tile_kernel(const __grid_constant__ TileParams p) {
    extern __shared__ unsigned char raw[];
    __shared__ TileShared s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x & 1;
    const int nth = p.nt / 2, x_half = nth * 128, x_stage = 2 * p.subs * x_half, w_stage = p.subs * kWBlockBytes, hstep = 2 * p.subs;
    const uint32_t pad = (1024u - (smem_u32(raw) & 1023u)) & 1023u;
    unsigned char* xs = raw + pad;                                   // [stages][subs][2][nt / 2][128]
    unsigned char* wsm = xs + p.stages * x_stage;                    // [stages][subs][128][128]
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            bar_init(&s.ready[i], 17);                               // eight warps of either CTA, and the bytes of both's tokens
            bar_init(&s.done[i], 1);
            bar_init(&s.w_full[i], 1);
            bar_init(&s.w_empty[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&s.d_full[i], 1);
            bar_init(&s.d_empty[i], 16);
        }
        bar_init(&s.idle, 1);
        s.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    pair_sync();
    fence_after();
    // all 512 columns are this pair's, from address 0 on
    const uint32_t a_col0 = (p.d_stages * p.nt + 31) / 32 * 32, xs_addr = smem_u32(xs);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Every thread waits for the tokens' grid itself, those that read none of its output too: what the calls before it
    // wrote (scales, channels) is visible to a thread that has waited, and to no other.  No bounded wait begins before.
    pdl_wait();
    const int pieces = p.m_tiles * p.n_tiles * p.splits, first = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (warp == 0 && lane == 0) {                       // token producer
        Ring r;
        int issued = 0;
        bool ok = true;
        for (int u = first; u < pieces && ok; u += pairs) {
            const Piece w = piece(p, u);
            for (int h = w.h0; h < w.h1; h += hstep) {
                if (!(ok = bar_wait(&s.done[r.i], r.ph ^ 1, s))) break;
                const int n = min(hstep, w.h1 - h);
                if (rank == 0) bar_expect(&s.ready[r.i], 2 * n * x_half);
                const uint32_t bar = first_of_pair(&s.ready[r.i]);
                unsigned char* d = xs + r.i * x_stage;
                for (int i = 0; i < n; ++i) tma_load_pair(d + i * x_half, &p.tx, (h + i) * kHalfK, w.m0 + rank * nth, bar);
                r.next(p.stages);
                ++issued;
            }
        }
        // Every copy has landed before the CTA gives its shared memory back: what has been multiplied has, and where a
        // wait ran out, this one's limit is far longer than a copy takes.
        for (int j = 0; j < p.stages && j < issued; ++j) {
            r.back(p.stages);
            bar_drain(&s.done[r.i], r.ph, s);
        }
    } else if (warp == 2 && lane == 0) {                // channel producer
        Ring r;
        int issued = 0;
        bool ok = true;
        for (int u = first; u < pieces && ok; u += pairs) {
            const Piece w = piece(p, u);
            for (int h = w.h0; h < w.h1; h += hstep) {
                if (!(ok = bar_wait(&s.w_empty[r.i], r.ph ^ 1, s))) break;
                const int n = (min(hstep, w.h1 - h) + 1) / 2;
                bar_expect(&s.w_full[r.i], n * kWBlockBytes);
                for (int i = 0; i < n; ++i)
                    tma_load(wsm + r.i * w_stage + i * kWBlockBytes, &p.tw, (h + 2 * i) * kHalfK, w.n0 + rank * kCtaN, &s.w_full[r.i]);
                r.next(p.stages);
                ++issued;
            }
        }
        for (int j = 0; j < p.stages && j < issued; ++j) {
            r.back(p.stages);
            bar_drain(&s.w_full[r.i], r.ph, s);
        }
    } else if (warp == 1 && rank == 0) {                // issuer: the whole warp, so that descriptors stay in uniform registers
        Ring x, d;
        int a = 0;
        const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(p.nt / 8) << 17) | ((2 * kCtaN / 16u) << 24);
        const bool one = elect();
        bool ok = true, there = false;
        for (int u = first; u < pieces && ok; u += pairs) {
            const Piece w = piece(p, u);
            if (!(ok = __all_sync(0xffffffffu, bar_wait(&s.d_empty[d.i], d.ph ^ 1, s)))) break;
            const uint32_t acc = d.i * p.nt;
            for (int h = w.h0; h < w.h1; h += hstep) {
                if (!there && !(ok = __all_sync(0xffffffffu, bar_wait_pair(&s.ready[x.i], x.ph, s)))) break;
                fence_after();
                const uint32_t bs = xs_addr + x.i * x_stage, at = a_col0 + a * 64 * p.subs;
                const int n = min(hstep, w.h1 - h);
                if (one) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_ts(acc, at + 8 * k, smem_desc(bs) + 2 * k, idesc, h > w.h0 || k > 0);
                }
                // A look at the next stage while these four run: a barrier costs 120 to 300 clocks to look at even
                // where it is ready, in which the tensor cores would run dry.
                Ring y = x;
                y.next(p.stages);
                there = __all_sync(0xffffffffu, bar_test_pair(&s.ready[y.i], y.ph));
                if (one) {
                    for (int i = 1; i < n; ++i) {
                        const uint64_t desc = smem_desc(bs + i * x_half);
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_ts(acc, at + 32 * i + 8 * k, desc + 2 * k, idesc, true);
                    }
                    mma_commit(&s.done[x.i]);
                }
                __syncwarp();
                x = y;
                a = a + 1 == p.a_stages ? 0 : a + 1;
            }
            if (ok && one) mma_commit(&s.d_full[d.i]);
            d.next(p.d_stages);
        }
        if (one) {
            mma_commit<false>(&s.idle);                 // no one in the second CTA waits for it
            bar_drain(&s.idle, 0, s);
        }
    } else if (warp >= 4 && warp < 12) {                // epilogue: warp's channels, half of the tokens
        Ring d;
        const int q = warp & 3, c0 = warp < 8 ? 0 : (p.nt / 2 + 15) / 16 * 16, c1 = warp < 8 ? (p.nt / 2 + 15) / 16 * 16 : p.nt;
        float* sa = s.sa[warp - 4];
        const int64_t ld = OUT == kTilePart ? p.N : p.ldo;
        constexpr int ES = OUT == kTileBf16 ? 2 : 4;
        constexpr int BATCH = OUT == kTileBf16 ? 4 : 2;   // chunks of 16 columns held at a time: 32 registers (64 spill)
        for (int u = first; u < pieces; u += pairs) {
            const Piece w = piece(p, u);
            const int64_t n = w.n0 + rank * kCtaN + q * 32 + lane;
            const int cols = min(c1, p.M - w.m0);
            const bool in = n < p.N;
            float swn = 1.0f;
            __syncwarp();
            if constexpr (OUT != kTilePart) {           // fetched while the tile is still being summed
                if (in) swn = p.sw[n];
                for (int c = c0 + lane; c < cols; c += 32) sa[c - c0] = p.sa[w.m0 + c];
            }
            const bool ok = bar_wait(&s.d_full[d.i], d.ph, s) && !s.failed;
            fence_after();
            if (!ok) swn = __int_as_float(0x7fffffff);
            const uint64_t sw2 = pair(swn, swn);
            __syncwarp();
            char* o = static_cast<char*>(p.out) + ((OUT == kTilePart ? static_cast<int64_t>(w.split) * p.M * p.N : 0) + (w.m0 + c0) * ld + n) * ES;
            const uint32_t acc = d.i * p.nt + (static_cast<uint32_t>(q * 32) << 16);
            if (c0 >= c1 && lane == 0) bar_arrive_first(&s.d_empty[d.i]);   // a tile of 16 tokens
            // The accumulator is given back before the last columns are stored: the next tile waits for it.
            for (int b = c0; b < c1; b += 16 * BATCH) {
                uint32_t r[BATCH][ES == 2 ? 8 : 16];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int c = b + 16 * i;
                    if (c >= c1) break;
                    float v[16];
                    tmem_ld16(acc + c, v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint64_t lo = pair(v[4 * j], v[4 * j + 1]), hi = pair(v[4 * j + 2], v[4 * j + 3]);
                        if constexpr (OUT != kTilePart) {
                            const float4 f = *reinterpret_cast<const float4*>(sa + (c - c0) + 4 * j);
                            lo = mul2(lo, pair(f.x, f.y));
                            hi = mul2(hi, pair(f.z, f.w));
                        }
                        lo = mul2(lo, sw2);
                        hi = mul2(hi, sw2);
                        float o0, o1, o2, o3;
                        unpair(lo, o0, o1);
                        unpair(hi, o2, o3);
                        if constexpr (ES == 2) {
                            r[i][2 * j] = pack2(o0, o1);
                            r[i][2 * j + 1] = pack2(o2, o3);
                        } else {
                            r[i][4 * j] = __float_as_uint(o0);
                            r[i][4 * j + 1] = __float_as_uint(o1);
                            r[i][4 * j + 2] = __float_as_uint(o2);
                            r[i][4 * j + 3] = __float_as_uint(o3);
                        }
                    }
                }
                if (b + 16 * BATCH >= c1) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive_first(&s.d_empty[d.i]);
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int c = b + 16 * i;
                    if (c >= cols) break;
#pragma unroll
                    for (int j = 0; j < 16; ++j, o += ld * ES) {
                        if (!in || c + j >= cols) continue;
                        if constexpr (ES == 2) *reinterpret_cast<unsigned short*>(o) = static_cast<unsigned short>(r[i][j / 2] >> (16 * (j & 1)));
                        else *reinterpret_cast<uint32_t*>(o) = r[i][j];
                    }
                }
            }
            d.next(p.d_stages);
        }
    } else if (warp >= 12) {                            // converters
        const int half = (warp - 12) >> 2, q = warp & 3, row = q * 32 + lane;
        Ring w, e;                                       // e: the stage that last held this one's columns of TMEM
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        int block = 0, a = 0;
        bool ok = true;
        for (int u = first; u < pieces && ok; u += pairs) {
            const Piece pc = piece(p, u);
            for (int h = pc.h0; h < pc.h1; h += hstep, ++block) {
                if (!(ok = __all_sync(0xffffffffu, bar_wait(&s.w_full[w.i], w.ph, s)))) break;
                const unsigned char* src = wsm + w.i * w_stage + row * kBlockK;
                uint32_t r[32];
                for (int b = 0; b < p.subs; ++b, src += kWBlockBytes) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int4 v = *reinterpret_cast<const int4*>(src + (((4 * half + c) ^ (row & 7)) << 4));
                        widen4(v.x, r[8 * c], r[8 * c + 1]);
                        widen4(v.y, r[8 * c + 2], r[8 * c + 3]);
                        widen4(v.z, r[8 * c + 4], r[8 * c + 5]);
                        widen4(v.w, r[8 * c + 6], r[8 * c + 7]);
                    }
                    if (b == 0 && block >= p.a_stages) {
                        if (!(ok = __all_sync(0xffffffffu, bar_wait(&s.done[e.i], e.ph, s)))) break;
                        e.next(p.stages);
                    }
                    fence_after();
                    tmem_st32(a_col0 + (a * p.subs + b) * 64 + half * 32 + lane_base, r);
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) bar_arrive(&s.w_empty[w.i]);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive_first(&s.ready[w.i]);
                w.next(p.stages);
                a = a + 1 == p.a_stages ? 0 : a + 1;
            }
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    pair_sync();                                        // nothing of the pair's is in flight any more
    fence_after();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(s.tmem) : "memory");
}

struct CombineParams {
    const float* part;
    const float* sa;
    const float* sw;
    void* out;
    int64_t ldo, M, N;
    int32_t splits;
};

// out = (Σ over the parts, in their order)·scales.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ CombineParams p) {
    pdl_enter();
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, m = blockIdx.y;
    if (n >= p.N) return;
    float v = 0.0f;
#pragma unroll 4
    for (int i = 0; i < p.splits; ++i) v += p.part[(i * p.M + m) * p.N + n];
    store_elem<BF16>(p.out, m * p.ldo + n, v * p.sa[m] * p.sw[n]);
}

// ---- host ----------------------------------------------------------------

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

int encode(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t cols, int64_t rows,
           int64_t pitch_bytes, int box_cols, int box_rows, CUtensorMapSwizzle swizzle) {
    EncodeFn fn = encode_fn();
    if (fn == nullptr) return DDP_ERR_UNSUPPORTED;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch_bytes)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)}, one[2] = {1, 1};
    const CUresult r = fn(map, type, 2, const_cast<void*>(base), dims, strides, box, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? DDP_OK : cuda_fail(cudaErrorInvalidValue);
}

// dp4a for up to kDotTokens.  Lanes per row, rows at a time and vectors in flight by K (us): 50257 x 768 at 8.3 with
// (16, 2, 3), 13.2 with (32, 1, 8); 8192 x 4096 at 8.0 and 6.2.  From 3 tokens on the 8-bit tensor instruction is ahead:
// 8 tokens of 8192 x 4096 17.7 by dp4a, 9.9; of 50257 x 768 19.3, 12.0 (1 token there 11.7).
constexpr int kDotTokens = 2;
struct DotPlan {
    void (*kernel)(FewParams);
    int rows;   // per CTA
};
template <bool BF16>
DotPlan dot_plan(int M, int32_t K) {
    if (K <= 1024) return {M == 1 ? few_kernel<1, 16, 2, 3, BF16> : few_kernel<2, 16, 2, 3, BF16>, kFewThreads / 16 * 2};
    return {M == 1 ? few_kernel<1, 32, 1, 8, BF16> : few_kernel<2, 32, 1, 8, BF16>, kFewThreads / 32};
}

int row_align(const void* p, int64_t ld, int64_t rows) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p) | (rows > 1 ? static_cast<uintptr_t>(ld) : 0);
    return a % 16 == 0 ? 16 : a % 4 == 0 ? 4 : 1;
}

// Channels whose rows are not on 16-byte boundaries are repacked for TMA; the
// workspace keeps room for that, so that it depends on the sizes alone.
int64_t token_pitch(int32_t K) { return round_up(K, 8); }
int64_t channel_pitch(int32_t K) { return round_up(K, 16); }
size_t token_bytes(int64_t M, int32_t K) { return static_cast<size_t>(round_up(M * token_pitch(K) * 2, 256)); }
size_t channel_bytes(int64_t N, int32_t K) { return static_cast<size_t>(round_up(N * channel_pitch(K), 256)); }

// Tiles of more than kFewTokens tokens, and the parts of K where the tiles
// alone leave pairs of SMs without work (at least kMinBlocks stages each).
constexpr int kMinBlocks = 4;
constexpr int kMaxSplits = 16;
constexpr int kPairs = 76;        // of a full GB300: what tiles and splits are made for
constexpr int kTileCost = 24;     // in token columns
struct Tiles {
    int nt, m_tiles, n_tiles, subs, splits, per_split;   // blocks of K per stage, stages per split
};
Tiles plan_tiles(int64_t M, int64_t N, int32_t K) {
    Tiles t{};
    t.n_tiles = static_cast<int>((N + 2 * kCtaN - 1) / (2 * kCtaN));
    // The width of a tile: the least of waves times the time of a tile (its width, and kTileCost for its ends):
    // 4096 x 4096 x 4096 86 us with 224 tokens, 94 with 256.
    const int64_t mt0 = (M + kMaxNT - 1) / kMaxNT;
    int64_t best = INT64_MAX;
    const int64_t mt1 = mt0 * t.n_tiles > kPairs ? 2 * mt0 : mt0;       // what one wave holds is not cut further
    for (int64_t mt = mt0; mt <= mt1 && mt < mt0 + 64; ++mt) {
        const int64_t nt = round_up((M + mt - 1) / mt, 16), m_tiles = (M + nt - 1) / nt;
        const int64_t cost = (m_tiles * t.n_tiles + kPairs - 1) / kPairs * (nt + kTileCost);
        if (cost >= best) continue;
        best = cost;
        t.nt = static_cast<int>(nt);
        t.m_tiles = static_cast<int>(m_tiles);
    }
    // the barriers of a stage take as long as the MMAs of a narrow one: two blocks a stage
    t.subs = t.nt <= kMaxNT / 2 && K > kBlockK ? 2 : 1;
    const int stages = (K + t.subs * kBlockK - 1) / (t.subs * kBlockK);
    int64_t s = kPairs / (static_cast<int64_t>(t.m_tiles) * t.n_tiles);
    if (s > stages / (kMinBlocks / t.subs)) s = stages / (kMinBlocks / t.subs);
    if (s > kMaxSplits) s = kMaxSplits;
    if (s < 1) s = 1;
    t.per_split = static_cast<int>((stages + s - 1) / s);
    t.splits = (stages + t.per_split - 1) / t.per_split;
    return t;
}

}  // namespace
}  // namespace ddp

using namespace ddp;

extern "C" size_t q8_matmul_workspace_bytes(int64_t M, int64_t N, int32_t K) {
    if (M < 0 || N < 0 || K < 0 || K > kMaxK || M > kMaxWidth || N > kMaxWidth) return 0;
    if (M <= kFewTokens || N == 0 || K == 0) return 16;
    const Tiles t = plan_tiles(M, N, K);
    return token_bytes(M, K) + channel_bytes(N, K) + (t.splits > 1 ? static_cast<size_t>(t.splits) * M * N * 4 : 0);
}

extern "C" int q8_matmul(const int8_t* a, int64_t lda, const float* a_scale, const int8_t* w, int64_t ldw,
                         const float* w_scale, int64_t M, int64_t N, int32_t K, void* out, int64_t ldo,
                         int32_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if ((out_dtype != DDP_F32 && out_dtype != DDP_BF16) || M < 0 || N < 0 || K < 0) return DDP_ERR_INVALID_ARG;
    if (K > kMaxK || M > kMaxWidth || N > kMaxWidth) return DDP_ERR_UNSUPPORTED;
    const Mat ma{a, M, K, lda, 1}, mw{w, N, K, ldw, 1}, mo{out, M, N, ldo, out_dtype == DDP_BF16 ? 2 : 4},
        msa{a_scale, 1, M, M, 4}, msw{w_scale, 1, N, N, 4};
    if (!mat_valid(ma) || !mat_valid(mw) || !mat_valid(mo)) return DDP_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && (out == nullptr || a_scale == nullptr || w_scale == nullptr || workspace == nullptr ||
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
    if (!aligned16(workspace)) return DDP_ERR_ALIGNMENT;
    if (workspace_bytes < need) return DDP_ERR_CAPACITY;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = out_dtype == DDP_BF16;
    DeviceInfo d;
    int st = current_device_info(&d);
    if (st != DDP_OK) return st;

    if (K == 0) {                                       // a sum of no parts
        for (int64_t m = 0; m < M; m += 65535) {
            const int64_t rows = M - m < 65535 ? M - m : 65535;
            const CombineParams q{nullptr, a_scale + m, w_scale, static_cast<char*>(out) + m * ldo * (bf16 ? 2 : 4), ldo, rows, N, 0};
            st = launch_pdl(bf16 ? combine_kernel<true> : combine_kernel<false>,
                            dim3(static_cast<unsigned>((N + kThreads - 1) / kThreads), static_cast<unsigned>(rows)), kThreads, s, q);
            if (st != DDP_OK) return st;
        }
        return DDP_OK;
    }
    if (M <= kFewTokens) {
        const int32_t rows = static_cast<int32_t>(M);
        FewParams p{a, w, a_scale, w_scale, out, lda, ldw, ldo, N, K, rows, row_align(w, ldw, N), row_align(a, lda, M), 1};
        if (rows <= kDotTokens) {
            const DotPlan plan = bf16 ? dot_plan<true>(rows, K) : dot_plan<false>(rows, K);
            const int64_t need_ctas = (N + plan.rows - 1) / plan.rows, cap = 8ll * d.sm_count;
            const int64_t kc = K < kFewChunk ? round_up(K, 16) : kFewChunk;
            return launch_smem(plan.kernel, static_cast<unsigned>(need_ctas < cap ? need_ctas : cap), kFewThreads,
                               static_cast<size_t>(rows * kc), s, p);
        }
        // enough warps to fill the SMs, each with four blocks of K at least
        const int64_t groups = (N + 15) / 16, blocks = (K + 63) / 64;
        while (p.split < kFewWarps && groups * p.split < 16ll * d.sm_count && blocks >= 4 * p.split) p.split *= 2;
        const int64_t per_cta = kFewWarps / p.split;
        return launch_pdl(bf16 ? few_mma_kernel<true> : few_mma_kernel<false>,
                          dim3(static_cast<unsigned>((groups + per_cta - 1) / per_cta)), kFewThreads, s, p);
    }

    __half* x = static_cast<__half*>(workspace);
    int8_t* wr = static_cast<int8_t*>(workspace) + token_bytes(M, K);
    const bool repack = row_align(w, ldw, N) != 16 || (N > 1 && ldw >= (1ll << 40)) || (N == 1 && (ldw % 16 != 0 || ldw < K));
    const int64_t xp = token_pitch(K), wp = channel_pitch(K);
    const WidenParams wp_{a, x, w, repack ? wr : nullptr, lda, ldw, M, N, xp, wp, K, row_align(a, lda, M)};
    int64_t vecs = M * ((xp + 15) / 16);
    if (repack && N * (wp / 16) > vecs) vecs = N * (wp / 16);
    const int64_t wide = (vecs + kThreads - 1) / kThreads, cap = 16ll * d.sm_count;
    st = launch_pdl(widen_kernel, dim3(static_cast<unsigned>(wide < cap ? wide : cap)), kThreads, s, wp_);
    if (st != DDP_OK) return st;

    const Tiles t = plan_tiles(M, N, K);
    const int64_t pieces = static_cast<int64_t>(t.m_tiles) * t.n_tiles * t.splits;
    if (pieces > INT32_MAX / 2) return DDP_ERR_UNSUPPORTED;
    float* parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + token_bytes(M, K) + channel_bytes(N, K));
    TileParams p{};
    p.nt = t.nt;
    p.m_tiles = t.m_tiles;
    p.n_tiles = t.n_tiles;
    p.splits = t.splits;
    p.stages_per_split = t.per_split;
    p.halves = (K + kHalfK - 1) / kHalfK;
    p.group = 8;
    p.subs = t.subs;
    const int stage = t.subs * (p.nt * 128 + kWBlockBytes);
    p.stages = kRingBytes / stage < kMaxStages ? kRingBytes / stage : kMaxStages;
    // TMEM: accumulators (two of up to 64 columns), then stages of channels
    p.d_stages = p.nt <= kMaxNT / 4 ? 2 : 1;
    const int a_room = (512 - (p.d_stages * p.nt + 31) / 32 * 32) / (64 * t.subs);
    p.a_stages = a_room < kMaxAStages ? a_room : kMaxAStages;
    if (p.a_stages > p.stages) p.a_stages = p.stages;
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.sa = a_scale;
    p.sw = w_scale;
    p.out = t.splits > 1 ? parts : out;
    p.ldo = ldo;
    if ((st = encode(&p.tx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x, K, M, xp * 2, kHalfK, p.nt / 2,
                     CU_TENSOR_MAP_SWIZZLE_128B)) != DDP_OK)
        return st;
    if ((st = encode(&p.tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, repack ? wr : w, K, N, repack ? wp : ldw, kBlockK, kCtaN,
                     CU_TENSOR_MAP_SWIZZLE_128B)) != DDP_OK)
        return st;
    const int64_t pairs = pieces < d.sm_count / 2 ? pieces : d.sm_count / 2;
    size_t smem = static_cast<size_t>(p.stages) * stage + 1024;
    if (smem < kMinTileSmem) smem = kMinTileSmem;
    st = launch_smem(t.splits > 1 ? tile_kernel<kTilePart> : bf16 ? tile_kernel<kTileBf16> : tile_kernel<kTileF32>,
                     static_cast<unsigned>(2 * pairs), kTileThreads, smem, s, p, 2);
    if (st != DDP_OK || t.splits == 1) return st;
    const CombineParams q{parts, a_scale, w_scale, out, ldo, M, N, t.splits};
    return launch_pdl(bf16 ? combine_kernel<true> : combine_kernel<false>,
                      dim3(static_cast<unsigned>((N + kThreads - 1) / kThreads), static_cast<unsigned>(M)), kThreads, s, q);
}
