// decode.cuh — the whole routed MoE layer for a few tokens (T <= 16), on W4A8 or MXFP4 experts, in
// one kernel.
//
// The arithmetic of moe_w4a8_forward: S1 (FP8 of the tokens), S2 (top-k, gates), S4 (gate, up,
// SwiGLU), S5 (FP8 of h for each routed pair), S6 (down), S7 (the gated sum) and S8 (shared
// experts), with the experts' weights in pack-quantized INT4 or in MXFP4.
//
// What bounds it: a few tokens use each weight once or twice, so the time is the reading of the
// touched experts' weights (13 MB an expert at H = 4096, N = 2048) and, at one token, of launches.
// So one persistent cooperative grid (one CTA an SM) streams every weight byte once through a ring
// of shared-memory stages, and the stream does not stop at the layer's two inner dependencies: the
// weights of the down projections do not depend on h, so the producer warp fills the whole ring
// with them while the grid finishes h (barrier), quantizes it (barrier) and comes back to read.
//
//   prologue  every CTA ranks the logits itself (one warp a token), lists the touched experts and
//             starts streaming; meanwhile the consumer warps quantize the tokens into shared memory
//   phase A   unit = 8 gate rows and the same 8 up rows of one touched expert, all of K; the
//             units are split evenly over the CTAs; h (fp32) goes to the workspace
//   barrier, S5 (one CTA a routed pair), barrier
//   phase B   unit = 16 down rows of one touched expert; units run tile by tile (16 outputs of every
//             token), so a tile's experts add up in registers, in a fixed order; the two CTAs that
//             share a tile at the border of their ranges leave partial sums, and the one that comes
//             last adds them, again in a fixed order
//
// A stage is 16 rows x 2 KB (32 KB): 16 pieces of 16 rows x 128 bytes, one for each consumer warp
// (a row longer than 2 KB takes several stages, shorter rows put several units into one).  It is
// loaded by one TMA box for each of its row sets, in the 128-byte swizzle, so a warp reads 16 bytes
// of eight rows without bank conflicts.
//
// The products run on mma.sync m16n8k16 (f16, fp32 sums): the rows are the M = 16, up to eight
// tokens the N = 8.  tcgen05 would put 128 rows a tile and the widened weights through TMEM for the
// same eight columns; here its rate is not needed (the stream leaves an SM 1,400 cycles a stage),
// and a warp's registers hold the whole tile.  E4M3 values are exact in f16, and so are the weights:
//   INT4:  a nibble n = code + 8 left where it lies in a 16-bit half is the f16 subnormal n 2^-24
//          (bits 0..3) or n 2^-20 (bits 4..7, whose tokens' values carry 2^-4), so widening a packed
//          word costs four ANDs and a shift; the accumulator starts at -8 2^-24 sum q, which takes
//          the offset off again.
//   MXFP4: cvt.rn.f16x2.e2m1x2.
// (mma.sync on E4M3 is no way round the conversion: it took 400 warp instructions a stage and warp
// against 190, and the layer at T = 8 took 213 us.)
// A group's (block's) partial sum is scaled in fp32 by its weight scale: one promotion every 128
// (32) weights.  Shared experts run on the bf16 MMA, their activation as bf16 hi + lo halves.
#pragma once
#include <cooperative_groups.h>
#include <type_traits>
#include "forward.cuh"
#include "mxfp4.cuh"

namespace moe {

constexpr int kDecodeMaxT = 16;
constexpr int kDecodeWarps = 8;                          // consumer warps; one more streams the weights
constexpr int kDecodeThreads = 32 * (kDecodeWarps + 1);
constexpr int kDecodeStage = 32 * 1024;                  // weight bytes of a stage
constexpr int kDecodeMaxPairs = kDecodeMaxT * kMaxK;
constexpr int kDecodeMaxSlots = 8;
constexpr int kDecodeMaxGrid = 256;                      // CTAs the workspace's partial sums provide for
constexpr int kDecodeBatch = 4;                          // phase A: most stages between two sums over the warps
constexpr int kDecodePiece = 2048;                       // B-fragment bytes of 256 columns of eight tokens

struct DecodeLayer {
    int E, H, N;
    const uint8_t *w[3];          // gate, up [E, N, H/2], down [E, H, N/2]
    const void *s[3];             // INT4: bf16 [.., K/128]; MXFP4: E8M0 [.., K/32]
    int n_shared, shared_N;
    const uint16_t *sw[3];        // shared experts' gate, up, down (bf16)
};

// How rows of one weight matrix fill stages: `pieces` of 128 bytes a row.  A unit takes 1 << log of a
// stage's 16 pieces in each of `chunks` stages, and 1 << wlog of the 8 consumer warps, two pieces a
// warp (one where a row has no more); 8 >> wlog units share a stage.
struct DecodeRows {
    int pieces, log, wlog, chunks;
};

struct alignas(64) DecodeParams {
    CUtensorMap map[6];           // gate, up, down, shared gate, up, down
    const uint8_t* scale[3];
    const uint16_t *x, *wr;
    const float* logits;
    uint16_t* out;
    float *h, *gs, *hsum, *part, *ws_logits;
    uint8_t* hq;
    uint16_t *act_hi, *act_lo;
    unsigned* count;
    DecodeRows ra, rs, rb;        // gate/up, shared gate/up, down (routed; its log serves the shared rows too)
    int shared_chunks;            // stages' worth of a shared down row
    int E, H, N, k, T, n_shared, Ns;
    int slots, slot_bytes, batch, flat;   // flat: bit i set, map i is 2-D (rows are not whole pieces)
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ float lds_bf16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return bf16_bits_to_f32(v);
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Two E8M0 bytes (the low half of b) -> two floats.
__device__ __forceinline__ float2 e8m0x2_to_f32(uint32_t b) {
    const __nv_bfloat162_raw r = __nv_cvt_e8m0x2_to_bf162raw(static_cast<__nv_fp8x2_storage_t>(b & 0xFFFFu));
    return make_float2(bf16_bits_to_f32(r.x), bf16_bits_to_f32(r.y));
}

// Where the FP8 codes of columns 8 c8 .. 8 c8 + 7 lie in a token's row of B fragments: pieces of
// 256 columns; lane (token, t) reads its 64 bytes of a piece as four 16-byte words i = 2 h + j / 2, each
// the codes of weight words j and j + 1 of half h.  Word j of lane t covers columns 32 t + 8 j (INT4:
// a lane's 16 bytes of a weight row) or 32 j + 8 t (MXFP4: one block a word of the lanes) of the half.
template <bool kMx>
__device__ __forceinline__ void frag_place(int c8, int& piece, int& i, int& t, int& odd) {
    const int idx = c8 & 15, h = (c8 >> 4) & 1;
    const int j = kMx ? idx >> 2 : idx & 3;
    t = kMx ? idx & 3 : idx >> 2;
    piece = c8 >> 5;
    i = 2 * h + (j >> 1);
    odd = j & 1;
}
// Eight codes in column order -> the order in which the weights' widening pairs them: for INT4 the
// nibbles of a word come out as (0,4) (1,5) (2,6) (3,7), for MXFP4 as they are.
template <bool kMx>
__device__ __forceinline__ uint2 frag_order(uint2 c) {
    return kMx ? c : make_uint2(__byte_perm(c.x, c.y, 0x5140), __byte_perm(c.x, c.y, 0x7362));
}
// Four codes in that order -> the two B registers of one MMA.
template <bool kMx>
__device__ __forceinline__ void frag_f16(uint32_t c, uint32_t& b0, uint32_t& b1) {
    const __half2_raw l = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c & 0xFFFFu), __NV_E4M3);
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c >> 16), __NV_E4M3);
    b0 = *reinterpret_cast<const uint32_t*>(&l);
    b1 = *reinterpret_cast<const uint32_t*>(&h);
    if constexpr (!kMx) {   // the nibbles in bits 4..7 stand for 16 n
        const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x2C00)));   // 2^-4
        b1 = *reinterpret_cast<const uint32_t*>(&v);
    }
}
constexpr float kNibbleOffset = -8.0f / 16777216.0f;   // -8 2^-24

// A warp's B fragments of one block of eight tokens: the 512 columns of its two pieces as f16 (four
// halves of 128 columns), from the FP8 codes.
template <bool kMx>
__device__ __forceinline__ void frags_f16(const uint4 (&q)[8], uint32_t (&f)[64]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) frag_f16<kMx>(word(q[i >> 2], i & 3), f[2 * i], f[2 * i + 1]);
}
// INT4: where the accumulators start, off[h] = -8 2^-24 sum_q over half h, for the lane's two
// token columns.
__device__ __forceinline__ void nibble_offsets(const uint32_t (&f)[64], float2 (&off)[4]) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        float p[4] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i)   // -8 2^-24, -8 2^-20
            mma_f16(p, 0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u, f[16 * h + 2 * i], f[16 * h + 2 * i + 1]);
        off[h] = make_float2(p[0], p[1]);
    }
}

// Two E2M1 codes (the low byte of c) -> f16x2, the low nibble first.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t c) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(c & 0xFFu), __NV_E2M1);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// acc += the products of 16 rows x 512 weights (two pieces, `step` bytes apart in the stage) with the
// B fragments of one block of tokens.  row_a / row_b: the lane's rows g and g + 8; sa / sb: those
// rows' scales at the first piece; halves: how many of the four 128-column halves lie inside the row
// (a missing one has fragments and offsets of zero, and its scale is taken as nothing).  Nothing
// branches, so the halves' loads and MMA chains overlap.
template <bool kMx>
__device__ __forceinline__ void pieces_mma(uint32_t row_a, uint32_t row_b, uint32_t step, uint32_t sa, uint32_t sb,
                                           int halves, const uint32_t (&f)[64], const float2 (&off)[4], float (&acc)[4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if constexpr (!kMx) {
        const uint32_t at0 = (t ^ g) << 4;
        float s0[4], s1[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            s0[h] = h < halves ? lds_bf16(sa + 2 * h) : 0.0f;
            s1[h] = h < halves ? lds_bf16(sb + 2 * h) : 0.0f;
        }
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
            uint4 wa[2], wb[2];
            float p[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                wa[h] = lds128(row_a + pc * step + (at0 ^ (h * 64)));
                wb[h] = lds128(row_b + pc * step + (at0 ^ (h * 64)));
                p[h][0] = p[h][2] = off[2 * pc + h].x;
                p[h][1] = p[h][3] = off[2 * pc + h].y;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a = word(wa[h], j) >> (8 * s), c = word(wb[h], j) >> (8 * s);
                        const int i = 16 * (2 * pc + h) + 4 * j + 2 * s;
                        mma_f16(p[h], a & 0x000F000Fu, c & 0x000F000Fu, a & 0x00F000F0u, c & 0x00F000F0u, f[i], f[i + 1]);
                    }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                acc[0] = fmaf(s0[2 * pc + h], p[h][0], acc[0]);
                acc[1] = fmaf(s0[2 * pc + h], p[h][1], acc[1]);
                acc[2] = fmaf(s1[2 * pc + h], p[h][2], acc[2]);
                acc[3] = fmaf(s1[2 * pc + h], p[h][3], acc[3]);
            }
        }
    } else {
        uint32_t ea[4], eb[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            ea[h] = h < halves ? lds32(sa + 4 * h) : 0u;
            eb[h] = h < halves ? lds32(sb + 4 * h) : 0u;
        }
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t at = (h >> 1) * step + ((((h & 1) * 4 + j) ^ g) << 4) + 4 * t;
                const uint32_t a = lds32(row_a + at), c = lds32(row_b + at);
                const float2 e0 = e8m0x2_to_f32(ea[h] >> (16 * (j >> 1))), e1 = e8m0x2_to_f32(eb[h] >> (16 * (j >> 1)));
                const float f0 = j & 1 ? e0.y : e0.x, f1 = j & 1 ? e1.y : e1.x;
                float p[4] = {};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int i = 16 * h + 4 * j + 2 * s;
                    mma_f16(p, e2m1x2_to_f16x2(a >> (16 * s)), e2m1x2_to_f16x2(c >> (16 * s)),
                            e2m1x2_to_f16x2(a >> (16 * s + 8)), e2m1x2_to_f16x2(c >> (16 * s + 8)), f[i], f[i + 1]);
                }
                acc[0] = fmaf(f0, p[0], acc[0]);
                acc[1] = fmaf(f0, p[1], acc[1]);
                acc[2] = fmaf(f1, p[2], acc[2]);
                acc[3] = fmaf(f1, p[3], acc[3]);
            }
    }
}
// The power of two that pieces_mma's sums lack.
template <bool kMx>
constexpr float kDecodeLadder = kMx ? 1.0f : 16777216.0f;

// The same for 16 rows x 64 bf16 weights of one piece and one block of tokens; b: the lane's eight
// values of each half (32 columns).
__device__ __forceinline__ void piece_mma_bf16(uint32_t row_a, uint32_t row_b, const uint4 (&b)[2], float (&acc)[4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t at = ((h * 4 + t) ^ g) << 4;
        const uint4 wa = lds128(row_a + at), wb = lds128(row_b + at);
        mma_bf16(acc, wa.x, wb.x, wa.y, wb.y, b[h].x, b[h].y);
        mma_bf16(acc, wa.z, wb.z, wa.w, wb.w, b[h].z, b[h].w);
    }
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_load_2d_at(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(x), "r"(y)
        : "memory");
}
// `bytes` contiguous bytes (both addresses and the size multiples of 16).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kDecodeWarps) : "memory"); }

// The first unit of CTA c's even share of n units.
__device__ __forceinline__ int share(int n, int c, int G) { return static_cast<int>((int64_t)n * c / G); }

// S2 of one token by one warp, as topk_row (ranked by logit descending, index ascending; NaN as
// -inf), with the warp's maximum and the lowest index that has it in two redux instructions: the
// stream waits for this.  A logit's key is its bits in the order of the values, 0 once taken.
template <int EPL>
__device__ __forceinline__ void rank_row(const float* l, int E, int k, int* ids, float* gates, int lane) {
    uint32_t key[EPL];
#pragma unroll
    for (int s = 0; s < EPL; ++s) {
        const int e = lane + 32 * s;
        float x = e < E ? __ldcg(l + e) : 0.0f;
        x = isnan(x) ? -INFINITY : x + 0.0f;   // -0 ties with +0
        const uint32_t u = __float_as_uint(x);
        key[s] = e < E ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
    }
    float first = 0.0f, sum = 0.0f, mine = 0.0f;
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0u;
#pragma unroll
        for (int s = 0; s < EPL; ++s) best = max(best, key[s]);
        best = __reduce_max_sync(0xffffffffu, best);
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int s = EPL - 1; s >= 0; --s) at = key[s] == best ? lane + 32 * s : at;
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int s = 0; s < EPL; ++s) key[s] = at == lane + 32 * s ? 0u : key[s];
        const float v = __uint_as_float(best & 0x80000000u ? best & 0x7FFFFFFFu : ~best);
        if (j == 0) first = v;
        const float e = expf(v - first);
        sum = __fadd_rn(sum, e);
        if (lane == j) { ids[j] = at; mine = e; }
    }
    if (lane < k) gates[lane] = __fdiv_rn(mine, sum);
}

// A wait ran out: the status word is set, and the warp stays until its CTA's copies in flight (microseconds) have landed.
__device__ __forceinline__ void give_up() {
    if ((threadIdx.x & 31) == 0) atomicOr(&g_device_status, kStatusTimeout);
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 10000000ull) __nanosleep(100000);
}

struct DecodeShared {
    uint64_t full[kDecodeMaxSlots], empty[kDecodeMaxSlots];
    int ids[kDecodeMaxPairs];
    float gates[kDecodeMaxPairs], gs[kDecodeMaxPairs];
    int expert[kDecodeMaxPairs];                     // the touched experts, ascending
    uint32_t tokens[kDecodeMaxPairs];                // bit t: token t is routed to it
    int8_t pick[kDecodeMaxPairs][kDecodeMaxT];       // as its which selection
    uint32_t bitmap[kMaxE / 32];
    unsigned amax[kDecodeMaxT];
    float red[32];
    int n_experts, last;
    volatile int abort;
};

// A stage ring's position, as the producer and the consumers count it.
struct DecodeRing {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int slots) {
        if (++slot == slots) { slot = 0; phase ^= 1u; }
    }
};

template <bool kMx, int NT>
__global__ void __launch_bounds__(kDecodeThreads, 1) k_decode(const __grid_constant__ DecodeParams p) {
    namespace cg = cooperative_groups;
    extern __shared__ uint8_t smem_raw[];
    __shared__ DecodeShared S;
    const uint32_t ring = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t frags = ring + p.slots * p.slot_bytes;               // B fragments of the tokens
    const uint32_t frag_bytes = ((p.H + 255) / 256) * NT * kDecodePiece;
    float* red = reinterpret_cast<float*>(smem_raw + (frags + frag_bytes - tc::smem_u32(smem_raw)));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int G = gridDim.x, cta = blockIdx.x;
    const int T = p.T, k = p.k, P = T * k;
    const bool producer = warp == kDecodeWarps;

    // ---- prologue ----
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.slots; ++i) {
            tc::mbar_init(&S.full[i], 1);
            tc::mbar_init(&S.empty[i], kDecodeWarps);
        }
        tc::fence_mbar_init();
        S.abort = 0;
    }
    if (producer && lane < (p.n_shared ? 6 : 3)) ws::prefetch_map(&p.map[lane]);
    for (int i = threadIdx.x; i < kMaxE / 32; i += kDecodeThreads) S.bitmap[i] = 0u;
    for (int i = threadIdx.x; i < kDecodeMaxPairs; i += kDecodeThreads) S.tokens[i] = 0u;
    if (threadIdx.x < kDecodeMaxT) S.amax[threadIdx.x] = 0u;
    const int tiles = p.H / 16;
    for (int i = cta * kDecodeThreads + threadIdx.x; i < tiles; i += G * kDecodeThreads) p.count[i] = 0u;
    __syncthreads();

    // max |x| of the tokens: 8 / (T rounded up to a power of two) warps a token
    const int twarps = kDecodeWarps >> (T > 4 ? 3 : T > 2 ? 2 : T > 1 ? 1 : 0);
    const int tok0 = warp / twarps, tpart = warp % twarps;
    if (!producer) {
        for (int tok = tok0; tok < T; tok += kDecodeWarps / twarps) {
            const uint4* xrow = reinterpret_cast<const uint4*>(p.x + (int64_t)tok * p.H);
            float a = 0.0f;
            for (int c = tpart * 32 + lane; c < p.H / 8; c += twarps * 32) a = fmaxf(a, amax8(__ldg(xrow + c)));
            a = warp_max(a);
            if (lane == 0) atomicMax(&S.amax[tok], __float_as_uint(a));
        }
    }

    const float* logits = p.logits;
    if (p.wr) {   // logits of experts 2 c and 2 c + 1, then of those 2 G further: four warps an expert
        logits = p.ws_logits;
        const int half = warp >> 2, part = warp & 3, HC = p.H / 8;
        for (int e0 = 2 * cta; e0 < p.E; e0 += 2 * G) {
            const int e = e0 + half;
            float acc[8 * NT];
#pragma unroll
            for (int j = 0; j < 8 * NT; ++j) acc[j] = 0.0f;
            if (!producer && e < p.E) {
                const uint4* w4 = reinterpret_cast<const uint4*>(p.wr + (int64_t)e * p.H);
                for (int c = part * 32 + lane; c < HC; c += 128) {
                    float wf[8];
                    bf16x8_to_f32(__ldg(w4 + c), wf);
#pragma unroll
                    for (int j = 0; j < 8 * NT; ++j) {
                        if (j < T) {
                            float xf[8];
                            bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(p.x) + (int64_t)j * HC + c), xf);
#pragma unroll
                            for (int q = 0; q < 8; ++q) acc[j] = fmaf(xf[q], wf[q], acc[j]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 8 * NT; ++j) {
                    const float s = warp_sum(acc[j]);
                    if (lane == 0) red[warp * 8 * NT + j] = s;
                }
            }
            __syncthreads();
            if (threadIdx.x < 2 * T) {
                const int hh = threadIdx.x / T, j = threadIdx.x % T;
                if (e0 + hh < p.E) {
                    float s = 0.0f;
#pragma unroll
                    for (int w = 0; w < 4; ++w) s += red[(hh * 4 + w) * 8 * NT + j];
                    p.ws_logits[(int64_t)j * p.E + e0 + hh] = s;
                }
            }
            __syncthreads();
        }
        cg::this_grid().sync();
    }

    // S2: a warp a token, the streaming warp (which has nothing else to do yet) first
    for (int tt = kDecodeWarps - warp; tt < T; tt += kDecodeWarps + 1) {
        const float* l = logits + (int64_t)tt * p.E;
        int* ids = S.ids + tt * k;
        float* gates = S.gates + tt * k;
        if (p.E <= 256) rank_row<8>(l, p.E, k, ids, gates, lane);
        else rank_row<kMaxE / 32>(l, p.E, k, ids, gates, lane);
        __syncwarp();
        if (lane < k) atomicOr(&S.bitmap[ids[lane] >> 5], 1u << (ids[lane] & 31));
    }
    __syncthreads();
    if (threadIdx.x < P) {   // the pair's expert's place among the touched ones
        const int e = S.ids[threadIdx.x], tt = threadIdx.x / k;
        int r = __popc(S.bitmap[e >> 5] & ((1u << (e & 31)) - 1u));
        for (int i = 0; i < (e >> 5); ++i) r += __popc(S.bitmap[i]);
        S.expert[r] = e;
        S.pick[r][tt] = static_cast<int8_t>(threadIdx.x - tt * k);
        atomicOr(&S.tokens[r], 1u << tt);
    }
    if (threadIdx.x == kDecodeThreads - 1) {
        int n = 0;
        for (int i = 0; i < (p.E + 31) / 32; ++i) n += __popc(S.bitmap[i]);
        S.n_experts = n;
    }
    __syncthreads();
    const int n_ex = S.n_experts;

    // ranges of this CTA
    const int nb = p.N / 8, nbs = p.Ns / 8;
    const int a0 = share(n_ex * nb, cta, G), a1 = share(n_ex * nb, cta + 1, G);
    const int s0 = share(p.n_shared * nbs, cta, G), s1 = share(p.n_shared * nbs, cta + 1, G);
    const int Vr = n_ex * p.rb.chunks, V = Vr + p.n_shared * p.shared_chunks;   // units of a tile
    const int v0 = share(tiles * V, cta, G), v1 = share(tiles * V, cta + 1, G);
    const int row_scale_a = kMx ? p.H / 32 : p.H / 64, row_scale_b = kMx ? p.N / 32 : p.N / 64;   // bytes

    if (producer) {
        // ---- the weight stream ----
        DecodeRing r;
        // One stage: waits for its slot, announces `bytes` and lets each lane issue copies.
        auto begin = [&](uint32_t bytes) {
            if (!ws::wait(&S.empty[r.slot], r.phase ^ 1u, &S.abort)) return false;
            if (lane == 0) tc::mbar_arrive_expect_tx(&S.full[r.slot], bytes);
            __syncwarp();
            return true;
        };
        // `1 << log` pieces of `rows` rows from piece `z` on, at dst.
        auto box = [&](int m, uint32_t dst, int rows, int row, int z, int log) {
            if (!((p.flat >> m) & 1)) {
                tma_load_3d(dst, &p.map[m], 0, row, z, &S.full[r.slot]);
            } else {
                for (int i = 0; i < (1 << log); ++i)
                    tma_load_2d_at(dst + i * rows * 128, &p.map[m], (z + i) * 128, row, &S.full[r.slot]);
            }
        };
        bool ok = true;
        for (int pass = 0; pass < 2; ++pass) {   // phase A: routed units, then the shared experts'
            const DecodeRows& R = pass ? p.rs : p.ra;
            const int u0 = pass ? s0 : a0, u1 = pass ? s1 : a1, per = pass ? nbs : nb, rows = pass ? p.Ns : p.N;
            const int upu = kDecodeWarps >> R.wlog;
            for (int u = u0; ok && u < u1; u += upu) {
                const int n = min(upu, u1 - u);
                for (int c = 0; ok && c < R.chunks; ++c) {
                    const uint32_t unit = 2048u << R.log, sc = pass ? 0u : 16u * row_scale_a;
                    if (!(ok = begin(n * (unit + sc)))) break;
                    const uint32_t base = ring + r.slot * p.slot_bytes;
                    for (int i = lane; i < 4 * n; i += 32) {
                        const int q = i >> 2, what = i & 3, ei = (u + q) / per, b = (u + q) % per;
                        const int row = (pass ? ei : S.expert[ei]) * rows + b * 8;
                        if (what < 2)
                            box((pass ? 3 : 0) + what, base + q * unit + what * (unit / 2), 8, row, c * 16, R.log);
                        else if (!pass)
                            bulk_load(base + kDecodeStage + q * sc + (what - 2) * (sc / 2),
                                      p.scale[what - 2] + (int64_t)row * row_scale_a, sc / 2, &S.full[r.slot]);
                    }
                    __syncwarp();
                    r.next(p.slots);
                }
            }
        }
        // phase B: as many stages as there are slots before the barriers, the rest after them
        int issued = 0, synced = 0;
        const int upu = kDecodeWarps >> p.rb.wlog;
        for (int v = v0; ok && v < v1;) {
            const int tile = v / V, lo = v - tile * V, hi = min(V, lo + v1 - v);
            for (int q = lo; ok && q < hi; q += upu) {
                if (issued == p.slots && !synced) {
                    cg::this_grid().sync();
                    cg::this_grid().sync();
                    synced = 1;
                }
                const int n = min(upu, hi - q), nr = max(0, min(n, Vr - q));   // routed units among them
                const uint32_t unit = 2048u << p.rb.log, sc = 16u * row_scale_b;
                if (!(ok = begin(n * unit + nr * sc))) break;
                const uint32_t base = ring + r.slot * p.slot_bytes;
                for (int i = lane; i < 2 * n; i += 32) {
                    const int j = i >> 1, what = i & 1, id = q + j;
                    const bool routed = id < Vr;
                    const int per = routed ? p.rb.chunks : p.shared_chunks, o = routed ? id : id - Vr;
                    const int row = (routed ? S.expert[o / per] : o / per) * p.H + tile * 16;
                    if (!what)
                        box(routed ? 2 : 5, base + j * unit, 16, row, (o % per) << p.rb.log, p.rb.log);
                    else if (routed)
                        bulk_load(base + kDecodeStage + j * sc, p.scale[2] + (int64_t)row * row_scale_b, sc, &S.full[r.slot]);
                }
                __syncwarp();
                r.next(p.slots);
                ++issued;
            }
            v += hi - lo;
        }
        if (!synced) {
            cg::this_grid().sync();
            cg::this_grid().sync();
        }
        if (!ok) give_up();
        return;
    }

    // ---- the consumer warps ----
    // S1: the tokens' FP8 codes as B fragments
    for (int tok = tok0; tok < T; tok += kDecodeWarps / twarps) {
        const uint4* xrow = reinterpret_cast<const uint4*>(p.x + (int64_t)tok * p.H);
        const float s = __fdiv_rn(__uint_as_float(S.amax[tok]), kFp8Max);
        for (int c = tpart * 32 + lane; c < p.H / 8; c += twarps * 32) {
            const uint2 q = frag_order<kMx>(quant8(__ldg(xrow + c), s));
            int piece, i, tt, odd;
            frag_place<kMx>(c, piece, i, tt, odd);
            const uint32_t at = frags + ((piece * NT + (tok >> 3)) * 4 + i) * 512 + ((tok & 7) * 4 + tt) * 16 + odd * 8;
            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at), "r"(q.x), "r"(q.y) : "memory");
        }
    }
    consumers_sync();

    DecodeRing r;
    bool ok = true;
    auto wait_full = [&]() { ok = ok && ws::wait(&S.full[r.slot], r.phase, &S.abort); };
    auto release = [&]() {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.empty[r.slot]);
        r.next(p.slots);
    };
    // This warp's sums into set `s` of `red` (one float a lane and register: no bank conflicts).
    auto put_sums = [&](int s, const float (&acc)[NT][4]) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[((s * kDecodeWarps + warp) * NT * 4 + n * 4 + i) * 32 + lane] = acc[n][i];
    };
    // The gate and up sums of output s (unit, token column, row g) of a set of stages.
    auto get_sums = [&](int s, int wlog, int& unit, int& col, float& gate, float& up) {
        const int c1 = (s >> 5) & 1, n = (s >> 6) % NT, per = 1 << wlog;
        unit = s / (64 * NT);
        col = n * 8 + t * 2 + c1;
        gate = up = 0.0f;
        const float* f = red + ((unit << wlog) * NT * 4 + n * 4 + c1) * 32 + lane;
        for (int w = 0; w < per; ++w) {
            gate += f[w * NT * 128];
            up += f[w * NT * 128 + 64];
        }
    };
    const int batch = p.batch;

    // phase A, routed units: h = silu(G) U.  A batch of stages, then their sums over the warps.
    {
        const int upu = kDecodeWarps >> p.ra.wlog, slot_unit = warp >> p.ra.wlog;
        const int pair0 = warp & ((1 << p.ra.wlog) - 1);          // which two pieces of a chunk
        const uint32_t row_off = slot_unit * (2048 << p.ra.log) + 2 * pair0 * 1024 + g * 128, row_b = 1024 << p.ra.log;
        const uint32_t sc_off = kDecodeStage + (slot_unit * 16 + g) * row_scale_a;
        uint32_t f[64];
        float2 off[4];
        int held = -1;   // what f holds: two pieces of one block of tokens
        int ei = a0 / nb, left = nb - a0 % nb;   // the expert of unit u and how many of its units are left
        for (int u = a0; u < a1; u += upu * batch) {
#pragma unroll 1
            for (int s = 0; s < batch && u + s * upu < a1; ++s) {
                int e = ei;                      // this warp's expert
                for (int ahead = s * upu + slot_unit - left; ahead >= 0; ahead -= nb) ++e;
                const bool mine = u + s * upu + slot_unit < a1;
                const uint32_t toks = NT > 1 && mine ? S.tokens[e] : 0xFFu;
                float acc[NT][4] = {};
                for (int c = 0; c < p.ra.chunks; ++c) {
                    const int pair = c * 8 + pair0, halves = p.H / 128 - 4 * pair;
                    wait_full();
                    if (ok && mine && halves > 0) {
                        const uint32_t base = ring + r.slot * p.slot_bytes;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (NT > 1 && !((toks >> (8 * n)) & 0xFFu)) continue;
                            if (held != pair * NT + n) {
                                held = pair * NT + n;
                                uint4 q[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    q[i] = i < 2 * halves ? lds128(frags + (((2 * pair + (i >> 2)) * NT + n) * 4 + (i & 3)) * 512 + lane * 16)
                                                          : make_uint4(0u, 0u, 0u, 0u);
                                frags_f16<kMx>(q, f);
                                if constexpr (!kMx) nibble_offsets(f, off);
                            }
                            pieces_mma<kMx>(base + row_off, base + row_off + row_b, 1024, base + sc_off + pair * (kMx ? 16 : 8),
                                            base + sc_off + 8 * row_scale_a + pair * (kMx ? 16 : 8), halves, f, off, acc[n]);
                        }
                    }
                    release();
                }
                put_sums(s, acc);
            }
            consumers_sync();
            const int n_out = min(batch * upu, a1 - u) * 64 * NT;
            for (int s = threadIdx.x; s < n_out; s += 32 * kDecodeWarps) {
                int unit, col;
                float gt, up;
                get_sums(s, p.ra.wlog, unit, col, gt, up);
                int e = ei, b = unit + nb - left;
                for (; b >= nb; b -= nb) ++e;
                if (col >= T || !((S.tokens[e] >> col) & 1u)) continue;
                const float sx = __fdiv_rn(__uint_as_float(S.amax[col]), kFp8Max) * kDecodeLadder<kMx>;
                p.h[(int64_t)(col * k + S.pick[e][col]) * p.N + b * 8 + g] = silu(gt * sx) * (up * sx);
            }
            consumers_sync();
            for (left -= upu * batch; left <= 0; left += nb) ++ei;
        }
    }
    // phase A, shared experts: the same on bf16 weights and tokens
    {
        const int upu = kDecodeWarps >> p.rs.wlog, slot_unit = warp >> p.rs.wlog;
        const int pair0 = warp & ((1 << p.rs.wlog) - 1);
        const uint32_t row_off = slot_unit * (2048 << p.rs.log) + 2 * pair0 * 1024 + g * 128, row_b = 1024 << p.rs.log;
        for (int u = s0; u < s1; u += upu) {
            float acc[NT][4] = {};
            for (int c = 0; c < p.rs.chunks; ++c) {
                const int piece = 2 * (c * 8 + pair0);
                const bool mine = u + slot_unit < s1 && piece < p.rs.pieces;   // pieces: even, 2 H bytes
                uint4 b[NT][2][2] = {};
                if (mine) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (n * 8 + g < T)
                                b[n][i >> 1][i & 1] = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(n * 8 + g) * p.H) + piece * 8 + i * 4 + t);
                }
                wait_full();
                if (ok && mine) {
                    const uint32_t row = ring + r.slot * p.slot_bytes + row_off;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int pc = 0; pc < 2; ++pc) piece_mma_bf16(row + pc * 1024, row + row_b + pc * 1024, b[n][pc], acc[n]);
                }
                release();
            }
            put_sums(0, acc);
            consumers_sync();
            const int n_out = min(upu, s1 - u) * 64 * NT;
            for (int s = threadIdx.x; s < n_out; s += 32 * kDecodeWarps) {
                int unit, col;
                float gt, up;
                get_sums(s, p.rs.wlog, unit, col, gt, up);
                if (col >= T) continue;
                const float a = silu(gt) * up;
                const uint16_t hi = f32_to_bf16_bits(a);   // hi + lo: 16 bits of the activation
                const int64_t at = (int64_t)col * p.n_shared * p.Ns + (u + unit) * 8 + g;
                p.act_hi[at] = hi;
                p.act_lo[at] = f32_to_bf16_bits(a - bf16_bits_to_f32(hi));
            }
            consumers_sync();
        }
    }

    cg::this_grid().sync();
    // S5: pair q's codes as B fragments, by CTA q
    const int hq_row = ((p.N + 255) / 256) * 256;
    for (int q = cta; q < P; q += G) {
        const float4* src = reinterpret_cast<const float4*>(p.h + (int64_t)q * p.N);
        float a = 0.0f;
        for (int c = threadIdx.x; c < p.N / 4; c += 32 * kDecodeWarps) {
            const float4 v = __ldcg(src + c);
            a = fmaxf(fmaxf(a, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
        }
        a = warp_max(a);
        consumers_sync();
        if (lane == 0) S.red[warp] = a;
        consumers_sync();
        a = warp_max(S.red[lane & (kDecodeWarps - 1)]);
        const float s = __fdiv_rn(a, kFp8Max);
        for (int c = threadIdx.x; c < p.N / 8; c += 32 * kDecodeWarps) {   // whole half-warps: N is a multiple of 128
            uint2 codes = make_uint2(0u, 0u);
            if (s != 0.0f) {
                const float4 v = __ldcg(src + 2 * c), w = __ldcg(src + 2 * c + 1);
                codes.x = static_cast<uint32_t>(f32x2_to_e4m3x2(__fdiv_rn(v.x, s), __fdiv_rn(v.y, s))) |
                          (static_cast<uint32_t>(f32x2_to_e4m3x2(__fdiv_rn(v.z, s), __fdiv_rn(v.w, s))) << 16);
                codes.y = static_cast<uint32_t>(f32x2_to_e4m3x2(__fdiv_rn(w.x, s), __fdiv_rn(w.y, s))) |
                          (static_cast<uint32_t>(f32x2_to_e4m3x2(__fdiv_rn(w.z, s), __fdiv_rn(w.w, s))) << 16);
            }
            int piece, i, tt, odd;
            frag_place<kMx>(c, piece, i, tt, odd);
            *reinterpret_cast<uint2*>(p.hq + (int64_t)q * hq_row + piece * 256 + i * 64 + tt * 16 + odd * 8) =
                frag_order<kMx>(codes);
            if constexpr (!kMx) {   // the sums of the 128-column groups, for the nibbles' offset
                float sum = e4m3x8_sum(codes);
                const uint32_t half = 0xFFFFu << (lane & 16);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(half, sum, o);
                if ((c & 15) == 0) p.hsum[(int64_t)q * (hq_row / 128) + (c >> 4)] = sum * kNibbleOffset;
            }
        }
        if (threadIdx.x == 0) p.gs[q] = S.gates[q] * s * kDecodeLadder<kMx>;
    }
    cg::this_grid().sync();
    if (threadIdx.x < P) S.gs[threadIdx.x] = __ldcg(p.gs + threadIdx.x);
    consumers_sync();

    // phase B.  The FP8 activations of a warp's next stage (its first block of tokens) are fetched
    // while it works on this one.
    const int upu = kDecodeWarps >> p.rb.wlog, slot_unit = warp >> p.rb.wlog;
    const int pair0 = warp & ((1 << p.rb.wlog) - 1), pairs = 1 << p.rb.wlog;   // of a unit
    const uint32_t row_off = slot_unit * (2048 << p.rb.log) + 2 * pair0 * 2048 + g * 128;
    const uint32_t sc_off = kDecodeStage + (slot_unit * 16 + g) * row_scale_b;
    uint4 q[8] = {};
    float2 off[4] = {};
    // Block n of routed expert ei's activations at columns 512 pair ..
    auto fetch = [&](int ei, int pair, int n) {
        const int halves = p.N / 128 - 4 * pair, col = n * 8 + g;
        const uint32_t toks = S.tokens[ei];
        const bool on = (toks >> col) & 1u;
        const uint4* src = reinterpret_cast<const uint4*>(p.hq + (int64_t)(on ? col * k + S.pick[ei][col] : 0) * hq_row + pair * 512) + t;
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = on && i < 2 * halves ? __ldcg(src + (i >> 2) * 16 + (i & 3) * 4) : make_uint4(0u, 0u, 0u, 0u);
        if constexpr (!kMx) {
            float f[2][4] = {};
#pragma unroll
            for (int c1 = 0; c1 < 2; ++c1) {
                const int c2 = n * 8 + t * 2 + c1;
                if ((toks >> c2) & 1u) {
                    const float* hs = p.hsum + (int64_t)(c2 * k + S.pick[ei][c2]) * (hq_row / 128) + 4 * pair;
#pragma unroll
                    for (int h = 0; h < 4; ++h) f[c1][h] = h < halves ? __ldcg(hs + h) : 0.0f;
                }
            }
#pragma unroll
            for (int h = 0; h < 4; ++h) off[h] = make_float2(f[0][h], f[1][h]);
        }
    };
    auto first_block = [&](int ei) { return NT > 1 && !(S.tokens[ei] & 0xFFu) ? 1 : 0; };
    // The next stage's first block, where the warp's unit there is a routed expert's.
    auto prefetch = [&](int id, int hi) {
        if (id < hi && id < Vr) fetch(id / p.rb.chunks, (id % p.rb.chunks) * pairs + pair0, first_block(id / p.rb.chunks));
    };
    for (int v = v0; v < v1;) {
        const int tile = v / V, lo = v - tile * V, hi = min(V, lo + v1 - v);
        float acc[NT][4] = {};
        prefetch(lo + slot_unit, hi);
        for (int u = lo; u < hi; u += upu) {
            const int id = u + slot_unit;
            const uint32_t base = ring + r.slot * p.slot_bytes;
            if (id < Vr && id < hi) {
                const int ei = id / p.rb.chunks, pair = (id % p.rb.chunks) * pairs + pair0, halves = p.N / 128 - 4 * pair;
                const uint32_t toks = S.tokens[ei];
                uint32_t f[64];
                float2 o[4];
                frags_f16<kMx>(q, f);
#pragma unroll
                for (int h = 0; h < 4; ++h) o[h] = off[h];
                prefetch(id + upu, hi);
                wait_full();
                if (ok && halves > 0) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (NT > 1 && !((toks >> (8 * n)) & 0xFFu)) continue;
                        if (NT > 1 && n != first_block(ei)) {      // a second block: fetched now, the next stage's again after it
                            fetch(ei, pair, n);
                            frags_f16<kMx>(q, f);
#pragma unroll
                            for (int h = 0; h < 4; ++h) o[h] = off[h];
                            prefetch(id + upu, hi);
                        }
                        float y[4] = {};
                        pieces_mma<kMx>(base + row_off, base + row_off + 1024, 2048, base + sc_off + pair * (kMx ? 16 : 8),
                                        base + sc_off + 8 * row_scale_b + pair * (kMx ? 16 : 8), halves, f, o, y);
#pragma unroll
                        for (int c1 = 0; c1 < 2; ++c1) {
                            const int col = n * 8 + t * 2 + c1;
                            if ((toks >> col) & 1u) {   // the other columns hold nothing of this expert's
                                const float fac = S.gs[col * k + S.pick[ei][col]];
                                acc[n][c1] = fmaf(fac, y[c1], acc[n][c1]);
                                acc[n][c1 + 2] = fmaf(fac, y[c1 + 2], acc[n][c1 + 2]);
                            }
                        }
                    }
                }
            } else {
                const int o = id - Vr, e = o / max(1, p.shared_chunks), piece = ((o % max(1, p.shared_chunks)) << p.rb.log) + 2 * pair0;
                const bool mine = id < hi && piece < p.Ns / 64;
                uint4 b[NT][2][2][2] = {};   // hi and lo
                if (mine) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (n * 8 + g < T && (i < 2 || p.rb.log > 0)) {
                                const int64_t at = ((int64_t)(n * 8 + g) * p.n_shared + e) * (p.Ns / 8) + piece * 8 + i * 4 + t;
                                b[n][0][i >> 1][i & 1] = __ldcg(reinterpret_cast<const uint4*>(p.act_hi) + at);
                                b[n][1][i >> 1][i & 1] = __ldcg(reinterpret_cast<const uint4*>(p.act_lo) + at);
                            }
                }
                wait_full();
                if (ok && mine) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int pc = 0; pc < 2; ++pc) {
                            if (pc && p.rb.log == 0) break;   // the unit has one piece
#pragma unroll
                            for (int part = 0; part < 2; ++part)
                                piece_mma_bf16(base + row_off + pc * 2048, base + row_off + 1024 + pc * 2048, b[n][part][pc], acc[n]);
                        }
                }
            }
            release();
        }
        put_sums(0, acc);
        consumers_sync();
        const bool whole = hi - lo == V;
        float* part = p.part + (int64_t)(tile + cta) * (128 * NT);   // tile + cta: its own for each (tile, CTA)
        float sum = 0.0f;
        const int s = threadIdx.x;
        if (s < 128 * NT)
            for (int w = 0; w < kDecodeWarps; ++w) sum += red[w * NT * 128 + s];
        if (!whole) {
            if (s < 128 * NT) part[s] = sum;
            __threadfence();
            consumers_sync();
            // the CTAs that hold a piece of this tile: first .. last (those with an empty share hold none)
            const int U = tiles * V, f0 = tile * V, f1 = f0 + V - 1;
            const int first = static_cast<int>(((int64_t)(f0 + 1) * G - 1) / U), last = static_cast<int>(((int64_t)(f1 + 1) * G - 1) / U);
            const int parts = U >= G ? last - first + 1 : V;
            if (threadIdx.x == 0) S.last = atomicAdd(p.count + tile, 1u) == (unsigned)(parts - 1);
            consumers_sync();
            if (S.last) {
                __threadfence();
                sum = 0.0f;
                if (s < 128 * NT)
                    for (int c = first; c <= last; ++c)
                        if (share(U, c, G) < share(U, c + 1, G)) sum += __ldcg(p.part + (int64_t)(tile + c) * (128 * NT) + s);
            }
        }
        if (s < 128 * NT && (whole || S.last)) {
            const int i = s >> 5, col = (i >> 2) * 8 + t * 2 + (i & 1), m = tile * 16 + g + 8 * ((i >> 1) & 1);
            if (col < T) p.out[(int64_t)col * p.H + m] = f32_to_bf16_bits(sum);
        }
        consumers_sync();   // red is free for the next tile
        v += hi - lo;
    }
    if (!ok) give_up();
}

// ---- host ---------------------------------------------------------------------------------------

struct DecodePlan {
    size_t logits, h, hq, gs, hsum, act, part, count, total;
};

inline DecodePlan plan_decode(const DecodeLayer& L, int64_t T, int k) {
    DecodePlan p{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + (bytes ? bytes : 1), 256);
        return at;
    };
    const size_t P = (size_t)T * k, nt = (T + 7) / 8;
    p.logits = take((size_t)T * L.E * 4);
    p.h = take(P * L.N * 4);
    p.hq = take(P * align_up(L.N, 256));
    p.gs = take(P * 4);
    p.hsum = take(P * (align_up(L.N, 256) / 128) * 4);
    p.act = take((size_t)T * L.n_shared * L.shared_N * 4);     // hi, then lo
    p.part = take((size_t)(L.H / 16 + kDecodeMaxGrid) * 128 * nt * 4);
    p.count = take((size_t)(L.H / 16) * 4);
    p.total = off;
    return p;
}

inline int decode_args_ok(const DecodeLayer& L, int64_t T, int k) {
    if (T < 0 || L.E < 1 || L.H <= 0 || L.N <= 0 || k < 1 || L.n_shared < 0) return MOE_ERR_INVALID_ARG;
    if (T > kDecodeMaxT || L.H % 128 || L.N % 128 || L.H > 16384 || L.N > 8192) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (L.H * ((T + 7) / 8) > 16384) return MOE_ERR_UNSUPPORTED_SHAPE;
    const int st = route_args_ok(T, L.E, k);
    if (st != MOE_OK) return st;
    if (L.n_shared > 0 && (L.shared_N <= 0 || L.shared_N % 128 || L.shared_N > 8192 || L.n_shared > 64))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

inline DecodeRows decode_rows(int64_t row_bytes, int log = -1) {
    DecodeRows r{};
    r.pieces = static_cast<int>((row_bytes + 127) / 128);
    while (r.log < 4 && (1 << r.log) < r.pieces) ++r.log;
    if (log >= 0) r.log = log;
    r.wlog = r.log > 0 ? r.log - 1 : 0;
    r.chunks = (r.pieces + (1 << r.log) - 1) >> r.log;
    return r;
}

// Weight rows as [piece][row][128 bytes]: a 3-D view where rows are whole pieces, else a 2-D one.
inline bool decode_map(CUtensorMap* m, const void* w, uint64_t row_bytes, uint64_t rows, uint32_t box_rows, int log, bool* flat) {
    *flat = row_bytes % 128 != 0;
    if (*flat) return make_map_u8(m, w, row_bytes, rows, 128, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
    const cuuint64_t dims[3] = {128, rows, row_bytes / 128};
    const cuuint64_t strides[2] = {row_bytes, 128};
    const cuuint32_t box[3] = {128, box_rows, 1u << log};
    return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, w, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <bool kMx, int NT>
inline int launch_decode(DecodeParams& q, cudaStream_t stream) {
    const size_t scale_a = (size_t)(kDecodeWarps >> q.ra.wlog) * 16 * (kMx ? q.H / 32 : q.H / 64);
    const size_t scale_b = (size_t)(kDecodeWarps >> q.rb.wlog) * 16 * (kMx ? q.N / 32 : q.N / 64);
    q.slot_bytes = static_cast<int>(align_up(kDecodeStage + std::max(scale_a, scale_b), 1024));
    const size_t frag = (size_t)((q.H + 255) / 256) * NT * kDecodePiece;
    const size_t room = 227 * 1024 - sizeof(DecodeShared) - 1024 - 256 - frag;   // of a CTA's 227 KB
    size_t red = 0;
    for (q.batch = kDecodeBatch; q.batch > 0; q.batch >>= 1) {   // fewer stages a sum where slots are short
        red = (size_t)q.batch * kDecodeWarps * NT * 128 * 4;
        q.slots = static_cast<int>(std::min<size_t>(kDecodeMaxSlots, (room - red) / q.slot_bytes));
        if (q.slots >= 4 || q.batch == 1) break;
    }
    if (q.slots < 2) return MOE_ERR_UNSUPPORTED_SHAPE;
    const size_t smem = 1024 + (size_t)q.slots * q.slot_bytes + frag + red;
    const void* fn = reinterpret_cast<const void*>(k_decode<kMx, NT>);
    if (set_smem(fn, smem)) return MOE_ERR_CUDA;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return MOE_ERR_CUDA;
    void* args[] = {&q};
    if (cudaLaunchCooperativeKernel(fn, dim3(std::min(sms, kDecodeMaxGrid)), dim3(kDecodeThreads), args, smem, stream) != cudaSuccess) {
        (void)cudaGetLastError();   // a rejected launch leaves no error behind for later calls
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

// With `router` non-null the logits are computed from it and `logits` is ignored.
template <bool kMx>
inline int decode_impl(const DecodeLayer& L, const uint16_t* x, const float* logits, const uint16_t* router, int64_t T,
                       int k, uint16_t* out, void* ws, size_t ws_bytes, cudaStream_t stream) {
    int st = decode_args_ok(L, T, k);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!x || !(router ? (const void*)router : logits) || !out) return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) {
        if (!L.w[i] || !L.s[i] || (L.n_shared > 0 && !L.sw[i])) return MOE_ERR_INVALID_ARG;
        if (!aligned(L.w[i], 16) || !aligned(L.s[i], 16) || (L.n_shared > 0 && !aligned(L.sw[i], 16)))
            return MOE_ERR_MISALIGNED;
    }
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(router ? (const void*)router : logits, router ? 16 : 4))
        return MOE_ERR_MISALIGNED;
    const DecodePlan p = plan_decode(L, T, k);
    if (!ws || ws_bytes < p.total) return MOE_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return MOE_ERR_MISALIGNED;
    uint8_t* b = static_cast<uint8_t*>(ws);
    DecodeParams q{};
    q.ra = decode_rows(L.H / 2);
    q.rb = decode_rows(L.N / 2);
    if (L.n_shared > 0) {
        q.rs = decode_rows((int64_t)L.H * 2);
        q.shared_chunks = decode_rows((int64_t)L.shared_N * 2, q.rb.log).chunks;
    }
    for (int i = 0; i < (L.n_shared > 0 ? 6 : 3); ++i) {
        const bool sh = i >= 3, down = i % 3 == 2;
        const uint64_t cols = down ? (sh ? L.shared_N : L.N) : L.H, rows = down ? L.H : (sh ? L.shared_N : L.N);
        bool flat;
        if (!decode_map(&q.map[i], sh ? static_cast<const void*>(L.sw[i - 3]) : L.w[i], sh ? cols * 2 : cols / 2,
                        rows * (sh ? L.n_shared : L.E), down ? 16 : 8, down ? q.rb.log : sh ? q.rs.log : q.ra.log, &flat))
            return MOE_ERR_CUDA;
        q.flat |= flat ? 1 << i : 0;
    }
    for (int i = 0; i < 3; ++i) q.scale[i] = static_cast<const uint8_t*>(L.s[i]);
    q.x = x;
    q.wr = router;
    q.logits = logits;
    q.out = out;
    q.ws_logits = reinterpret_cast<float*>(b + p.logits);
    q.h = reinterpret_cast<float*>(b + p.h);
    q.hq = b + p.hq;
    q.gs = reinterpret_cast<float*>(b + p.gs);
    q.hsum = reinterpret_cast<float*>(b + p.hsum);
    q.act_hi = reinterpret_cast<uint16_t*>(b + p.act);
    q.act_lo = q.act_hi + (size_t)T * L.n_shared * L.shared_N;
    q.part = reinterpret_cast<float*>(b + p.part);
    q.count = reinterpret_cast<unsigned*>(b + p.count);
    q.E = L.E; q.H = L.H; q.N = L.N; q.k = k; q.T = static_cast<int>(T);
    q.n_shared = L.n_shared;
    q.Ns = L.n_shared > 0 ? L.shared_N : 0;
    return T <= 8 ? launch_decode<kMx, 1>(q, stream) : launch_decode<kMx, 2>(q, stream);
}

inline DecodeLayer decode_layer(const moe_w4a8_layer& L) {
    return DecodeLayer{L.E, L.H, L.N,
                       {reinterpret_cast<const uint8_t*>(L.gate_packed), reinterpret_cast<const uint8_t*>(L.up_packed),
                        reinterpret_cast<const uint8_t*>(L.down_packed)},
                       {L.gate_scales, L.up_scales, L.down_scales},
                       L.n_shared, L.shared_N, {L.sh_gate, L.sh_up, L.sh_down}};
}
inline DecodeLayer decode_layer(const moe_mxfp4_layer& L) {
    return DecodeLayer{L.E, L.H, L.N, {L.gate_f4, L.up_f4, L.down_f4}, {L.gate_e8, L.up_e8, L.down_e8},
                       L.n_shared, L.shared_N, {L.sh_gate, L.sh_up, L.sh_down}};
}

}  // namespace moe

extern "C" size_t moe_w4a8_decode_workspace_bytes(const moe_w4a8_layer* layer, int64_t T, int k) {
    if (!layer || layer->group != moe::kGroup) return 0;
    const moe::DecodeLayer L = moe::decode_layer(*layer);
    return moe::decode_args_ok(L, T, k) == MOE_OK ? moe::plan_decode(L, T, k).total : 0;
}
extern "C" int moe_w4a8_decode(const moe_w4a8_layer* layer, const uint16_t* x_bf16, const float* router_logits, int64_t T,
                               int k, uint16_t* out_bf16, void* ws, size_t ws_bytes, moe_stream_t stream) {
    if (!layer) return MOE_ERR_INVALID_ARG;
    if (layer->group != moe::kGroup) return MOE_ERR_UNSUPPORTED_SHAPE;
    return moe::decode_impl<false>(moe::decode_layer(*layer), x_bf16, router_logits, nullptr, T, k, out_bf16, ws, ws_bytes, stream);
}
extern "C" int moe_w4a8_decode_router(const moe_w4a8_layer* layer, const uint16_t* x_bf16, const uint16_t* wr_bf16, int64_t T,
                                      int k, uint16_t* out_bf16, void* ws, size_t ws_bytes, moe_stream_t stream) {
    if (!layer || (T > 0 && !wr_bf16)) return MOE_ERR_INVALID_ARG;
    if (layer->group != moe::kGroup) return MOE_ERR_UNSUPPORTED_SHAPE;
    return moe::decode_impl<false>(moe::decode_layer(*layer), x_bf16, nullptr, wr_bf16, T, k, out_bf16, ws, ws_bytes, stream);
}
extern "C" size_t moe_mxfp4_decode_workspace_bytes(const moe_mxfp4_layer* layer, int64_t T, int k) {
    if (!layer) return 0;
    const moe::DecodeLayer L = moe::decode_layer(*layer);
    return moe::decode_args_ok(L, T, k) == MOE_OK ? moe::plan_decode(L, T, k).total : 0;
}
extern "C" int moe_mxfp4_decode(const moe_mxfp4_layer* layer, const uint16_t* x_bf16, const float* router_logits, int64_t T,
                                int k, uint16_t* out_bf16, void* ws, size_t ws_bytes, moe_stream_t stream) {
    if (!layer) return MOE_ERR_INVALID_ARG;
    return moe::decode_impl<true>(moe::decode_layer(*layer), x_bf16, router_logits, nullptr, T, k, out_bf16, ws, ws_bytes, stream);
}
extern "C" int moe_mxfp4_decode_router(const moe_mxfp4_layer* layer, const uint16_t* x_bf16, const uint16_t* wr_bf16, int64_t T,
                                       int k, uint16_t* out_bf16, void* ws, size_t ws_bytes, moe_stream_t stream) {
    if (!layer || (T > 0 && !wr_bf16)) return MOE_ERR_INVALID_ARG;
    return moe::decode_impl<true>(moe::decode_layer(*layer), x_bf16, nullptr, wr_bf16, T, k, out_bf16, ws, ws_bytes, stream);
}
