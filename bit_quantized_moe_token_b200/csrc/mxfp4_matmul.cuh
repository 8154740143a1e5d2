// mxfp4_matmul.cuh — out = A B^T with both operands in MXFP4 rows (mxfp4.cuh):
//   out[m, n] = sum_b 2^(sa[m,b] + sb[n,b] - 254) sum_{k in block b} A[m,k] B[n,k]
#pragma once
#include "mxfp4.cuh"
#include "route.cuh"
#include "tc_pipe.cuh"

namespace moe {

// ---- M <= 16 and one wave: mma.sync ----------------------------------------------------------------------------
//
// A few tokens' product is the reading of B.  A CTA takes 16 rows of B (the MMA's M = 16; tokens are its N = 8
// columns, in one or two blocks) and its eight warps 512 columns at a time each; a warp asks for all of its codes
// and scales at once and for the next 512 columns' before it multiplies, so B streams in with one latency, and the
// warps' sums meet in shared memory in a fixed order.  Word t of a 16-byte block goes to lane t of a row's four, so an
// MMA pair covers one block; E2M1 is exact in f16.  A block's sum is a multiple of 1/4 below 2^11: multiplied first by
// the smaller of its two scales it neither overflows (unless the result does) nor loses bits, and a scale of 255 (NaN,
// the largest as bits too) stays what it is.
// Measured (bf16 out, M = 1, 4096 x 4096 weights, 8.9 MB): 6.9 us with weights that come from HBM (20 % of its measured rate,
// a chain of latencies), 6.1 with the same weights, then in L2, in every call.  It serves one wave of CTAs, two an SM for up
// to eight tokens and one beyond; more rows of B, and M > 16, go to the tensor-memory kernel, which reads 128 rows of A
// whatever M is.  This kernel against that one, in us, weights from HBM (in L2):
//            2048 x 4096              4096 x 4096               8192 x 4096                14336 x 4096
//   M =  1   4.3 (3.6)  9.2 (8.7)     6.9 (6.1)  10.6 (10.1)    11.5 (10.2)  11.6 (10.7)   18.3 (16.6)  14.5 (13.3)
//   M =  8   5.3 (4.5)  9.2 (8.7)     8.0 (7.2)  10.7 (10.1)    13.7 (13.1)  12.2 (11.6)   21.9 (20.1)  14.3 (13.1)
//   M = 16   6.8 (5.9)  9.2 (8.8)    12.1 (11.0) 10.4 ( 9.6)    22.7 (20.8)  12.0 (11.3)   38.2 (35.2)  13.8 (13.0)
// (The rule gives away up to half a microsecond at M = 1 and 8192 rows, where the two meet.)
namespace mxmm {

// Sixteen scales (blocks b .. b + 15) of a row of `blocks`; 0 past its end.  One 16-byte load where the row allows it:
// loads of many rows cost their sectors, and this halves or quarters them.
__device__ __forceinline__ uint4 scales16(const uint8_t* row, int b, int blocks) {
    uint32_t v[4] = {0u, 0u, 0u, 0u};
    if (row != nullptr && b < blocks) {
        const uint8_t* at = row + b;
        const int n = blocks - b;   // scales left in the row
        const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at));
        if (n >= 16 && (low & 15u) == 0) return __ldg(reinterpret_cast<const uint4*>(at));
        if (n >= 16 && (low & 3u) == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __ldg(reinterpret_cast<const uint32_t*>(at) + i);
        } else if (n >= 20) {   // five whole words around them, all in this row and those before it
            const uint32_t* words = reinterpret_cast<const uint32_t*>(at - (low & 3u));
            uint32_t u[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) u[i] = __ldg(words + i);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(u[i], u[i + 1], 8 * (low & 3u));
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i >> 2] |= (i < n ? static_cast<uint32_t>(__ldg(at + i)) : 0u) << (8 * (i & 3));
        }
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

template <int NT, int kType>
__global__ void __launch_bounds__(256) k_few(const uint8_t* __restrict__ a, const uint8_t* __restrict__ as,
                                             const uint8_t* __restrict__ b, const uint8_t* __restrict__ bs, int M, int64_t N, int K,
                                             void* __restrict__ out) {
    __shared__ float red[8][NT * 4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int blocks = K / kMxBlock;
    const uint8_t* rows[2] = {n0 + g < N ? b + (n0 + g) * (K / 2) : nullptr, n0 + g + 8 < N ? b + (n0 + g + 8) * (K / 2) : nullptr};
    float acc[NT][4] = {};
    for (int b0 = warp * 16; b0 < blocks; b0 += 8 * 16) {
        uint32_t w[2][16], x[NT][16];
        uint4 sw[2], sx[NT][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                w[i][j] = rows[i] && b0 + j < blocks ? __ldg(reinterpret_cast<const uint32_t*>(rows[i] + (b0 + j) * 16) + t) : 0u;
            sw[i] = scales16(rows[i] ? bs + (n0 + g + 8 * i) * blocks : nullptr, b0, blocks);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int m = 8 * n + g;
#pragma unroll
            for (int j = 0; j < 16; ++j)
                x[n][j] = m < M && b0 + j < blocks ? __ldg(reinterpret_cast<const uint32_t*>(a + (int64_t)m * (K / 2) + (b0 + j) * 16) + t) : 0u;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int mc = 8 * n + 2 * t + c;
                sx[n][c] = scales16(mc < M ? as + (int64_t)mc * blocks : nullptr, b0, blocks);
            }
        }
        auto word = [](const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; };
#pragma unroll
        for (int j4 = 0; j4 < 4; ++j4) {
            float fw[2][4], fx[NT][2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) e8m0x4_to_f32(word(sw[i], j4), fw[i]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) e8m0x4_to_f32(word(sx[n][c], j4), fx[n][c]);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                const int j = 4 * j4 + jj;
                uint32_t r0[4], r1[4];
                e2m1x8_to_f16(w[0][j], r0);
                e2m1x8_to_f16(w[1][j], r1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint32_t c[4];
                    e2m1x8_to_f16(x[n][j], c);
                    float p[4];
                    mma_f16(p, r0[0], r1[0], r0[1], r1[1], c[0], c[1], 0.0f, 0.0f, 0.0f, 0.0f);
                    mma_f16(p, r0[2], r1[2], r0[3], r1[3], c[2], c[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t u = __float_as_uint(fw[i >> 1][jj]), v = __float_as_uint(fx[n][i & 1][jj]);
                        acc[n][i] = fmaf(p[i] * __uint_as_float(min(u, v)), __uint_as_float(max(u, v)), acc[n][i]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp][n * 4 + i][lane] = acc[n][i];
    __syncthreads();
    for (int s = threadIdx.x; s < NT * 128; s += 256) {
        const int i = s >> 5, m = (i >> 2) * 8 + 2 * t + (i & 1);
        const int64_t n = n0 + g + 8 * ((i >> 1) & 1);
        if (m >= M || n >= N) continue;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) sum += red[w][i][lane];
        if constexpr (kType == MOE_F32) static_cast<float*>(out)[m * N + n] = sum;
        else static_cast<uint16_t*>(out)[m * N + n] = f32_to_bf16_bits(sum);
    }
}

}  // namespace mxmm

// ---- else: tcgen05 -------------------------------------------------------------------------------
//
// kind::mxf4.block_scale takes both operands as they are stored: K in stages of 256 codes (128-byte rows, TMA in the
// 128-byte swizzle), four MMAs of K = 64 a stage into one fp32 accumulator in TMEM, each block's two scales applied by the
// tensor core (products exact, fp32 sums).  A tile is 128 x BN outputs of a CTA, or 256 x 256 of a pair of CTAs
// (cta_group::2): each has 128 rows of A and of the accumulator and half of B's rows, the first issues the MMAs.
//
// Roles: kDrain warps drain the accumulator, four bring the scales, one thread issues the TMA loads, one the MMAs.
//
// Scales.  The tensor core wants 128 rows' four scales of 128 codes as four TMEM columns: row 32 c + l in lane l of
// column c, the same in all four lane quadrants; each scale warp stores its quadrant's with tcgen05.st.  (tcgen05.cp from
// shared memory, issued ahead of the stage's MMAs, held those up: 16384 x 4096 x 4096 in 173 us against 156.)  They come
// as TMA boxes of 16 bytes (two stages) of every row; where K, the pointers or M do not suit those, the warps load the
// same 16 bytes a row two such pairs ahead and exchange them through shared memory.  With these loads everywhere the
// product takes 135 us against 115: a load of 32 rows is 32 passes of the shared memory's data path, which is what the
// kernel is short of (a stage's codes are written once and read once, 512 cycles of it; by loads and exchange the
// scales took 335 more, now 120).
//
// The issuing thread.  What it does a stage has to take less than the stage's 512 cycles of MMA: one barrier for the bytes
// and the scales, and a thread chosen by elect.sync, whose operands the compiler keeps in uniform registers (with two
// barriers and lane 0 a stage took it 980 cycles, 530 of them to issue; 147 us against 144).
//
// The accumulator's 256 columns and the scales leave no room in TMEM for a second one, so the draining warps first take it
// into registers (rounded to the output type), free it, and store while the next tile's MMAs run: sixteen warps of 64
// columns (eight of 128: 144 us against 136), which leaves 80 registers a thread; 4 bytes a thread are spilled for bf16
// outputs and 40 for fp32.
//
// Measured (bf16 out): 16384 x 4096 x 4096 111 to 115 us in runs of six products, 4,800 to 4,970 TFLOP/s, some 2.9 times the
// measured bf16 peak (FP4's nominal rate is four times bf16's); one call after another for longer, under the power limit,
// 136 to 140 us = 3,900 to 4,040 TFLOP/s.  2048 x 4096 x 4096 19.9 us: two waves for 1.73 waves of tiles.
namespace mxmm {

constexpr int kStageK = 256;

template <int BN, bool kPair>
struct Cfg {
    static_assert(kPair ? BN == 256 : BN <= 128);
    static constexpr int kStages = BN >= 128 ? 6 : 8;
    static constexpr int kDrain = BN == 256 ? 16 : 8;                // warps that drain the accumulator
    static constexpr int kThreads = (kDrain + 6) * 32;
    static constexpr int kBRows = kPair ? BN / 2 : BN;               // of B in this CTA's shared memory
    static constexpr int kA = 128 * 128, kB = kBRows * 128;
    static constexpr int kHalves = BN > 128 ? 2 : 1;                 // 128-row blocks of B's scales
    static constexpr int kStage = kA + kB;
    static constexpr int kCols = 4 * (2 + 2 * kHalves);              // TMEM columns of a stage's scales: A's 2 x 4, B's 2 x 4 kHalves
    static constexpr int kSmem = 1024 + kStages * kStage + kDrain * 1024 + 12 * 1024;   // and the draining and the scale warps' buffers
};
constexpr uint32_t kScaleCol = 256;                                  // the first of them

// One lane of the warp, in a form that lets the compiler keep what that lane issues in uniform registers.
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ uint32_t idesc(int m, int n, int sf) {
    return (static_cast<uint32_t>(sf) << 4)       // which of a column's four scales: B
           | (1u << 7) | (1u << 10)               // A, B = E2M1
           | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23)   // N / 8, scales UE8M0
           | (static_cast<uint32_t>(m >> 4) << 24) | (static_cast<uint32_t>(sf) << 29);      // M / 16, A's scales
}
template <bool kPair>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sa, uint32_t sb, uint32_t accumulate) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}
// Four TMEM columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint4& v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// A barrier of the four scale warps that also tells whether all of them are well: they leave together or not at all.
__device__ __forceinline__ bool all_well(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(static_cast<uint32_t>(ok)) : "memory");
    return r != 0;
}

// Arrives on `bar` (of both CTAs of a pair) once every MMA issued so far by this thread has completed.
template <bool kPair>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (kPair)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(tc::smem_u32(bar)),
                     "h"(static_cast<uint16_t>(3))
                     : "memory");
    else
        tc::mma_commit(bar);
}
template <bool kPair>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot) {
    if constexpr (kPair)
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(tc::smem_u32(slot)) : "memory");
    else
        tc::tmem_alloc(slot, 512);
}
template <bool kPair>
__device__ __forceinline__ void tmem_free(uint32_t taddr) {
    if constexpr (kPair) {
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
    } else {
        tc::tmem_relinquish();
        tc::tmem_dealloc(taddr, 512);
    }
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `bar`'s place in the first CTA of the pair.
__device__ __forceinline__ uint32_t in_first(uint64_t* bar) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(tc::smem_u32(bar)));
    return a;
}
// What a warp of the second CTA hands to the thread that issues the MMAs for both lies in TMEM (its scales stored there, its
// part of the accumulator read): tcgen05.wait and the tcgen05 fences around arrival and wait order it.  The arrival
// therefore needs the cluster's scope but no release of memory (with release.cluster, which waits for the warp's stores,
// 16384 x 4096 x 4096 takes 214 us against 112).  That thread waits at the same scope, from which the bytes of the other
// CTA's TMA loads come too.
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_first(bar)) : "memory");
}
// A TMA load into this CTA's shared memory whose bytes count on the first CTA's barrier.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(tc::smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(in_first(bar))
        : "memory");
}

template <int BN, int kType, bool kPair>
__global__ void __launch_bounds__(Cfg<BN, kPair>::kThreads, 1) k_gemm(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                                                      const __grid_constant__ CUtensorMap map_as, const __grid_constant__ CUtensorMap map_bs, bool boxes,
                                                      const uint8_t* __restrict__ as, const uint8_t* __restrict__ bs, int M, int N, int K,
                                                      void* __restrict__ out) {
    using C = Cfg<BN, kPair>;
    constexpr int kRows = kPair ? 256 : 128;   // of A in a tile
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ uint64_t full[C::kStages], empty[C::kStages], sc_full[2], sc_empty[2], acc_full, acc_empty;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort;
    const uint32_t base = (tc::smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tn = (N + BN - 1) / BN, tiles = (M + kRows - 1) / kRows * tn, stages = (K + kStageK - 1) / kStageK, blocks = K / kMxBlock;

    // A pair of CTAs computes one tile: each has its 128 rows of A and of the accumulator and half of B; the first
    // issues the MMAs, and what it waits for arrives on its barriers.
    const int rank = kPair ? static_cast<int>(cluster_rank()) : 0;
    const int tile0 = kPair ? blockIdx.x / 2 : blockIdx.x, tile_step = kPair ? gridDim.x / 2 : gridDim.x;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            tc::mbar_init(&full[i], 1 + (kPair ? 8 : 4));   // the bytes, and the scale warps
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sc_full[i], 1);
            tc::mbar_init(&sc_empty[i], 4);
        }
        tc::mbar_init(&acc_full, 1);
        tc::mbar_init(&acc_empty, (kPair ? 2 : 1) * C::kDrain);
        tc::fence_mbar_init();
        abort = 0;
    }
    if (warp == 0) tmem_alloc<kPair>(&tmem_slot);
    if (warp == C::kDrain + 4 && lane == 0) {
        ws::prefetch_map(&map_a);
        ws::prefetch_map(&map_b);
        if (boxes) {
            ws::prefetch_map(&map_as);
            ws::prefetch_map(&map_bs);
        }
    }
    tc::tc_fence_before();
    if constexpr (kPair) cluster_sync();
    else __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    bool ok = true;

    if (warp == C::kDrain + 4) {
        if (elected()) {
            uint32_t pair = 0;
            ws::Ring<C::kStages> r;
            for (int tile = tile0; ok && tile < tiles; tile += tile_step) {
                const int m0 = tile / tn * kRows + rank * 128, n0 = tile % tn * BN + rank * C::kBRows;
                for (int s = 0; s < stages; ++s, r.next()) {
                    if (boxes && (s & 1) == 0) {   // the scales of this stage and the next
                        if (!(ok = ws::wait(&sc_empty[pair & 1u], ((pair >> 1) & 1u) ^ 1u, &abort))) break;
                        uint64_t* bar = &sc_full[pair & 1u];
                        uint8_t* to = raw + (base - tc::smem_u32(raw)) + C::kStages * C::kStage + C::kDrain * 1024 + (pair & 1u) * 6144;
                        tc::mbar_arrive_expect_tx(bar, 2048 * (1 + C::kHalves));
                        ws::tma_load_2d(to, &map_as, s * 8, m0, bar);
                        ws::tma_load_2d(to + 2048, &map_bs, s * 8, tile % tn * BN, bar);
                        ++pair;
                    }
                    if (!(ok = ws::wait(&empty[r.idx], r.phase ^ 1u, &abort))) break;
                    if (rank == 0) tc::mbar_arrive_expect_tx(&full[r.idx], (kPair ? 2 : 1) * C::kStage);
                    uint8_t* dst = raw + (base - tc::smem_u32(raw)) + r.idx * C::kStage;
                    if constexpr (kPair) {
                        tma_load_pair(dst, &map_a, s * 128, m0, &full[r.idx]);
                        tma_load_pair(dst + C::kA, &map_b, s * 128, n0, &full[r.idx]);
                    } else {
                        ws::tma_load_2d(dst, &map_a, s * 128, m0, &full[r.idx]);
                        ws::tma_load_2d(dst + C::kA, &map_b, s * 128, n0, &full[r.idx]);
                    }
                }
            }
        }
    } else if (warp == C::kDrain + 5) {
        if (rank == 0 && elected()) {
            ws::Ring<C::kStages> r;
            uint32_t phase = 0;
            for (int tile = tile0; ok && tile < tiles; tile += tile_step, phase ^= 1u) {
                ok = ws::wait<kPair>(&acc_empty, phase ^ 1u, &abort);
                tc::tc_fence_after();
                for (int s = 0; ok && s < stages; ++s, r.next()) {
                    ok = ws::wait<kPair>(&full[r.idx], r.phase, &abort);
                    if (!ok) break;
                    tc::tc_fence_after();
                    const uint32_t a = base + r.idx * C::kStage, sf = tmem + kScaleCol + r.idx * C::kCols;
                    const uint64_t da = tc::sdesc_sw128(a), db = tc::sdesc_sw128(a + C::kA);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (s * kStageK + 64 * j >= K) break;
                        mma<kPair>(tmem, da + 2 * j, db + 2 * j, idesc(kRows, BN, 2 * (j & 1)), sf + 4 * (j >> 1),
                            sf + 8 + 4 * C::kHalves * (j >> 1), s > 0 || j > 0);
                    }
                    commit<kPair>(&empty[r.idx]);
                }
                if (ok) commit<kPair>(&acc_full);
            }
        }
    } else if (warp >= C::kDrain) {
        const int w = warp - C::kDrain;
        uint8_t* buf = raw + (base - tc::smem_u32(raw)) + C::kStages * C::kStage + C::kDrain * 1024;   // two pairs of stages
        ws::Ring<C::kStages> r;
        auto put = [&](uint32_t column, const uint4& v) {   // four columns of the stage's
            tmem_st4(tmem + (static_cast<uint32_t>(w * 32) << 16) + kScaleCol + r.idx * C::kCols + column, v);
        };
        auto stored = [&] {
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (kPair) arrive_first(&full[r.idx]);
                else tc::mbar_arrive(&full[r.idx]);
            }
            r.next();
        };
        if (boxes) {
            uint32_t pair = 0;
            for (int tile = tile0; ok && tile < tiles; tile += tile_step)
                for (int s = 0; ok && s < stages; s += 2, ++pair) {
                    if (!(ok = __all_sync(~0u, ws::wait(&sc_full[pair & 1u], (pair >> 1) & 1u, &abort)))) break;
                    const uint8_t* from = buf + (pair & 1u) * 6144 + lane * 16;
                    uint4 v[4 * (1 + C::kHalves)];           // rows lane, 32 + lane ..: the two stages' words
#pragma unroll
                    for (int i = 0; i < 4 * (1 + C::kHalves); ++i) v[i] = *reinterpret_cast<const uint4*>(from + 512 * i);
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sc_empty[pair & 1u]);
#pragma unroll
                    for (int d = 0; d < 2; ++d) {
                        if (!(ok = __all_sync(~0u, ws::wait(&empty[r.idx], r.phase ^ 1u, &abort)))) break;
                        tc::tc_fence_after();
#pragma unroll
                        for (int i = 0; i < 1 + C::kHalves; ++i) {
                            const uint4 *q = v + 4 * i;
                            put(i ? 8 + 4 * (i - 1) : 0, d ? make_uint4(q[0].z, q[1].z, q[2].z, q[3].z) : make_uint4(q[0].x, q[1].x, q[2].x, q[3].x));
                            put(i ? 8 + 4 * (C::kHalves + i - 1) : 4,
                                d ? make_uint4(q[0].w, q[1].w, q[2].w, q[3].w) : make_uint4(q[0].y, q[1].y, q[2].y, q[3].y));
                        }
                        stored();
                    }
                }
        }
        bool well = !boxes;   // (all four warps')
        uint32_t turn = 0;
        for (int tile = tile0; well && tile < tiles; tile += tile_step) {
            const int m = tile / tn * kRows + rank * 128 + 32 * w + lane, n = tile % tn * BN + 32 * w + lane;
            const uint8_t* rows[1 + C::kHalves];
            rows[0] = m < M ? as + (int64_t)m * blocks : nullptr;
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h) rows[1 + h] = n + 128 * h < N ? bs + (int64_t)(n + 128 * h) * blocks : nullptr;
            constexpr int kAhead = 2;   // pairs of stages whose scales are on their way
            uint4 v[kAhead][1 + C::kHalves];
            auto load = [&](int pair, uint4 (&to)[1 + C::kHalves]) {
#pragma unroll
                for (int i = 0; i < 1 + C::kHalves; ++i) to[i] = scales16(rows[i], pair * 16, blocks);
            };
#pragma unroll
            for (int d = 0; d < kAhead; ++d) load(d, v[d]);
            for (int s0 = 0; well && s0 < stages; s0 += 2 * kAhead) {
#pragma unroll
                for (int d = 0; d < kAhead; ++d) {
                    if (!well || s0 + 2 * d >= stages) break;
                    uint8_t* of = buf + (turn & 1u) * 6144 + lane * 16;
                    ++turn;
#pragma unroll
                    for (int i = 0; i < 1 + C::kHalves; ++i) {
                        uint8_t* to = of + w * 4 + 2048 * i;
                        *reinterpret_cast<uint32_t*>(to) = v[d][i].x;
                        *reinterpret_cast<uint32_t*>(to + 512) = v[d][i].y;
                        *reinterpret_cast<uint32_t*>(to + 1024) = v[d][i].z;
                        *reinterpret_cast<uint32_t*>(to + 1536) = v[d][i].w;
                    }
                    if (!(well = all_well(ok))) break;
                    load(s0 / 2 + d + kAhead, v[d]);
                    for (int s = s0 + 2 * d; ok && s < min(s0 + 2 * d + 2, stages); ++s) {
                        if (!(ok = __all_sync(~0u, ws::wait(&empty[r.idx], r.phase ^ 1u, &abort)))) break;
                        tc::tc_fence_after();
                        const uint8_t* from = of + (s & 1) * 1024;
#pragma unroll
                        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                            for (int i = 0; i < 1 + C::kHalves; ++i)
                                put(i ? 8 + 4 * (kb * C::kHalves + i - 1) : 4 * kb, *reinterpret_cast<const uint4*>(from + 2048 * i + 512 * kb));
                        stored();
                    }
                }
            }
        }
    } else {
        constexpr int kCols = BN / (C::kDrain / 4);
        const int q = warp & 3, c0 = (warp >> 2) * kCols;
        uint32_t phase = 0;
        for (int tile = tile0; ok && tile < tiles; tile += tile_step, phase ^= 1u) {
            if (!(ok = __all_sync(~0u, ws::wait(&acc_full, phase, &abort)))) break;
            tc::tc_fence_after();
            uint32_t v[kType == MOE_F32 ? kCols : kCols / 2];
#pragma unroll
            for (int c = 0; c < kCols; c += 32) {
                uint32_t t[32];
                tc::tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c0 + c, t);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if constexpr (kType == MOE_F32) v[c + i] = t[i];
                    else if (i & 1)
                        v[(c + i) >> 1] = static_cast<uint32_t>(f32_to_bf16_bits(__uint_as_float(t[i - 1]))) |
                                          (static_cast<uint32_t>(f32_to_bf16_bits(__uint_as_float(t[i]))) << 16);
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (kPair) arrive_first(&acc_empty);
                else tc::mbar_arrive(&acc_empty);
            }
            const int m0 = tile / tn * kRows + rank * 128 + q * 32, n0 = tile % tn * BN + c0;
            constexpr int kElem = kType == MOE_F32 ? 4 : 2, kVec = 16 / kElem;
            if (N % kVec == 0) {
                // 64 bytes of each of the 32 rows at a time through shared memory, so that a store writes whole rows'
                // segments (chunk c of row l at c ^ (l / 2) % 4: no bank conflicts either way)
                uint8_t* buf = raw + (base - tc::smem_u32(raw)) + C::kStages * C::kStage + warp * 1024;
#pragma unroll
                for (int c = 0; c < kCols * kElem / 64; ++c) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // 16 rows at a time
                        __syncwarp();
                        if (lane >> 4 == h) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                *reinterpret_cast<uint4*>(buf + (lane & 15) * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
                                    make_uint4(v[16 * c + 4 * i], v[16 * c + 4 * i + 1], v[16 * c + 4 * i + 2], v[16 * c + 4 * i + 3]);
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int row = i * 8 + (lane >> 2), m = m0 + 16 * h + row, n = n0 + (64 / kElem) * c + (lane & 3) * kVec;
                            const uint4 x = *reinterpret_cast<const uint4*>(buf + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
                            if (m < M && n < N) *reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + ((int64_t)m * N + n) * kElem) = x;
                        }
                    }
                }
            } else if (m0 + lane < M) {
                uint8_t* o = static_cast<uint8_t*>(out) + ((int64_t)(m0 + lane) * N + n0) * kElem;
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    if (n0 + c < N) {
                        if constexpr (kType == MOE_F32) reinterpret_cast<uint32_t*>(o)[c] = v[c];
                        else reinterpret_cast<uint16_t*>(o)[c] = static_cast<uint16_t>(v[c >> 1] >> (16 * (c & 1)));
                    }
            }
        }
    }
    if (!ok) atomicOr(&g_device_status, kStatusTimeout);
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    if (abort) {   // copies and MMAs in flight (microseconds) end before the CTA does
        const uint64_t t0 = tc::globaltimer_ns();
        while (tc::globaltimer_ns() - t0 < 10000000ull) __nanosleep(100000);
    }
    if constexpr (kPair) cluster_sync();   // neither leaves while the other may still use its barriers or memory
    tc::tc_fence_after();
    if (warp == 0) tmem_free<kPair>(tmem);
}

template <int BN, int kType, bool kPair = false>
inline int launch(const uint8_t* a, const uint8_t* as, const uint8_t* b, const uint8_t* bs, int M, int N, int K, void* out, int sms,
                  cudaStream_t stream) {
    using C = Cfg<BN, kPair>;
    CUtensorMap ma, mb, mas = {}, mbs = {};
    // scales by TMA: rows of whole 16-byte pieces.  (Few tokens: rows outside the tensor cost the boxes more than loads
    // that skip them; 16 x 14336 x 4096 took 16.4 us against 14.6, 64 x 4096 x 4096 8.5 against 9.3.)
    const bool boxes = K % 512 == 0 && aligned(as, 16) && aligned(bs, 16) && M >= 64;
    if (!make_map_u8(&ma, a, K / 2, M, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_u8(&mb, b, K / 2, N, 128, C::kBRows, CU_TENSOR_MAP_SWIZZLE_128B) ||
        (boxes && (!make_map_u8(&mas, as, K / kMxBlock, M, 16, 128, CU_TENSOR_MAP_SWIZZLE_NONE) ||
                   !make_map_u8(&mbs, bs, K / kMxBlock, N, 16, 128 * C::kHalves, CU_TENSOR_MAP_SWIZZLE_NONE))))
        return MOE_ERR_CUDA;
    const void* fn = reinterpret_cast<const void*>(k_gemm<BN, kType, kPair>);
    if (set_smem(fn, C::kSmem)) return MOE_ERR_CUDA;
    constexpr int kRows = kPair ? 256 : 128;
    const int64_t tiles = (int64_t)((M + kRows - 1) / kRows) * ((N + BN - 1) / BN);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(kPair ? 2 * std::min<int64_t>(tiles, sms / 2) : std::min<int64_t>(tiles, sms)));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kPair ? 2 : 1;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_gemm<BN, kType, kPair>, ma, mb, mas, mbs, boxes, as, bs, M, N, K, out) == cudaSuccess) return MOE_OK;
    (void)cudaGetLastError();   // a rejected launch leaves no error behind for later calls
    return MOE_ERR_CUDA;
}

}  // namespace mxmm

}  // namespace moe

extern "C" int mxfp4_matmul(const uint8_t* a, const uint8_t* a_scales, const uint8_t* b, const uint8_t* b_scales,
                            int64_t M, int64_t N, int64_t K, void* out, int out_type, moe_stream_t stream) {
    using namespace moe;
    if (M < 0 || N < 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (out_type != MOE_BF16 && out_type != MOE_F32) return MOE_ERR_INVALID_ARG;
    if (K % kMxBlock != 0 || K > 65536 || M > (1 << 22) || N > (1 << 22)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return MOE_OK;
    if (!a || !a_scales || !b || !b_scales || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scales, 4) || !aligned(b_scales, 4) || !aligned(out, 16))
        return MOE_ERR_MISALIGNED;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return MOE_ERR_CUDA;
    const int64_t few = (N + 15) / 16;   // CTAs
    if (M > 16 || few > (M <= 8 ? 2 : 1) * sms) {
        const int m = (int)M, n = (int)N, k = (int)K;
        // 64 columns a CTA while that is one wave (256 x 4096 x 4096: 8.8 us against 9.7 for 128).  Else 128, or 256 x 256
        // for a pair of CTAs: a wave of the latter takes 1.6 times as long (8.3 us against 5.2 at K = 4096) for up to twice
        // the outputs (512 rows x 4096: 10.4 us against 12.9; 1024: 15.5 against 13.9; 2048: 25.8 against 21.2).
        const int64_t rows = (M + 127) / 128, t128 = rows * ((N + 127) / 128), t256 = (M + 255) / 256 * ((N + 255) / 256);
        const bool narrow = rows * ((N + 63) / 64) <= sms;
        if (!narrow && 3 * ((t256 + sms / 2 - 1) / (sms / 2)) <= 2 * ((t128 + sms - 1) / sms))
            return out_type == MOE_F32 ? mxmm::launch<256, MOE_F32, true>(a, a_scales, b, b_scales, m, n, k, out, sms, stream)
                                       : mxmm::launch<256, MOE_BF16, true>(a, a_scales, b, b_scales, m, n, k, out, sms, stream);
#define MOE_MM(BN, TYPE) mxmm::launch<BN, TYPE>(a, a_scales, b, b_scales, m, n, k, out, sms, stream)
        if (out_type == MOE_F32) return narrow ? MOE_MM(64, MOE_F32) : MOE_MM(128, MOE_F32);
        return narrow ? MOE_MM(64, MOE_BF16) : MOE_MM(128, MOE_BF16);
#undef MOE_MM
    }
    const unsigned grid = static_cast<unsigned>(few);
#define MOE_MF(NT, TYPE) mxmm::k_few<NT, TYPE><<<grid, 256, 0, stream>>>(a, a_scales, b, b_scales, (int)M, N, (int)K, out)
    if (out_type == MOE_F32) { if (M <= 8) MOE_MF(1, MOE_F32); else MOE_MF(2, MOE_F32); }
    else { if (M <= 8) MOE_MF(1, MOE_BF16); else MOE_MF(2, MOE_BF16); }
#undef MOE_MF
    return launch_status();
}
