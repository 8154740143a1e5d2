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
// The products run on mma.sync m16n8k32 (E4M3): the rows are the M = 16, up to eight tokens the
// N = 8.  tcgen05 would put 128 rows a tile and the widened weights through TMEM for the same
// eight columns; here its rate is not needed (16 x 256 weights cost a warp about 150 instructions,
// a third of the issue slots at the full HBM rate), and a warp's registers hold the whole tile.
//   INT4:  the stored nibble n = code + 8 is the E4M3 encoding of n 2^-9 (the header of
//          tc_tiles.cuh); a second MMA with the constant -8 2^-9 takes the offset off, so the
//          fp32 accumulator holds 2^-9 sum q code exactly as signed codes would.
//   MXFP4: the nibble s e e m, shifted to s 00ee m00, is the E4M3 encoding of its value 2^-6.
// A group's (block's) partial sum is scaled in fp32 by its weight scale: one promotion every 128
// (32) weights.  Shared experts run on the bf16 MMA, their activation as bf16 hi + lo halves.
#pragma once
#include <cooperative_groups.h>
#include "forward.cuh"
#include "mxfp4.cuh"

namespace moe {

constexpr int kDecodeMaxT = 16;
constexpr int kDecodeWarps = 16;                         // consumer warps; one more streams the weights
constexpr int kDecodeThreads = 32 * (kDecodeWarps + 1);
constexpr int kDecodeStage = 32 * 1024;                  // weight bytes of a stage
constexpr int kDecodeMaxPairs = kDecodeMaxT * kMaxK;
constexpr int kDecodeMaxSlots = 8;
constexpr int kDecodeMaxGrid = 256;                      // CTAs the workspace's partial sums provide for
constexpr int kDecodePiece = 2048;                       // B-fragment bytes of 256 columns of eight tokens

struct DecodeLayer {
    int E, H, N;
    const uint8_t *w[3];          // gate, up [E, N, H/2], down [E, H, N/2]
    const void *s[3];             // INT4: bf16 [.., K/128]; MXFP4: E8M0 [.., K/32]
    int n_shared, shared_N;
    const uint16_t *sw[3];        // shared experts' gate, up, down (bf16)
};

// How rows of one weight matrix fill stages: `pieces` of 128 bytes a row; a unit takes 1 << log of
// a stage's 16 pieces in each of `chunks` stages, 16 >> log units share a stage.
struct DecodeRows {
    int pieces, log, chunks;
};

struct alignas(64) DecodeParams {
    CUtensorMap map[6];           // gate, up, down, shared gate, up, down
    const uint8_t* scale[3];
    const uint16_t *x, *wr;
    const float* logits;
    uint16_t* out;
    float *h, *gs, *part, *ws_logits;
    uint8_t* hq;
    uint16_t *act_hi, *act_lo;
    unsigned* count;
    DecodeRows ra, rs, rb;        // gate/up, shared gate/up, down (routed; its log serves the shared rows too)
    int shared_chunks;            // stages' worth of a shared down row
    int E, H, N, k, T, n_shared, Ns;
    int slots, slot_bytes, red_bufs, flat;   // flat: bit i set, map i is 2-D (rows are not whole pieces)
};

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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

// Where a lane's eight FP8 codes of columns 8 c8 .. 8 c8 + 7 of token column `col` (0..7) lie in a
// row of B fragments: pieces of 256 columns; a lane (col, t) reads its 64 bytes of a piece as four
// 16-byte words i = 2 half + j / 2, each the codes of MMAs j and j + 1 of that half.  MMA j of half
// h covers columns 32 t + 8 j (INT4: a lane's 16 bytes of a weight row) or 32 j + 8 t (MXFP4: one
// block an MMA) of the half, t = 0..3.  Returns {piece, byte in the 64-byte rows of a token}.
template <bool kMx>
__device__ __forceinline__ void frag_place(int c8, int& piece, int& i, int& t, int& odd) {
    const int idx = c8 & 15, h = (c8 >> 4) & 1;
    const int j = kMx ? idx >> 2 : idx & 3;
    t = kMx ? idx & 3 : idx >> 2;
    piece = c8 >> 5;
    i = 2 * h + (j >> 1);
    odd = j & 1;
}

// acc += the products of one piece (16 rows x 256 weights at row_a / row_b, rows g and g + 8 of the
// lane's group g) with the B fragments of NT blocks of eight tokens.  sa / sb: the rows' scales at
// this piece; halves: 128-weight halves of the piece inside the row; live: bit n set, block n has a
// routed token.
template <bool kMx, int NT>
__device__ __forceinline__ void piece_mma(uint32_t row_a, uint32_t row_b, uint32_t sa, uint32_t sb, int halves,
                                          const uint4 (&b)[NT][4], uint32_t live, float (&acc)[NT][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h >= halves) break;
        if constexpr (!kMx) {
            const uint32_t at = ((h * 4 + t) ^ g) << 4;
            const uint4 wa = lds128(row_a + at), wb = lds128(row_b + at);
            const float s0 = lds_bf16(sa + 2 * h), s1 = lds_bf16(sb + 2 * h);
            float p[NT][4] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a = word(wa, j), c = word(wb, j);
                const uint32_t a0 = a & 0x0F0F0F0Fu, a2 = (a >> 4) & 0x0F0F0F0Fu;
                const uint32_t a1 = c & 0x0F0F0F0Fu, a3 = (c >> 4) & 0x0F0F0F0Fu;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (NT > 1 && !((live >> n) & 1)) continue;
                    const uint4& q = b[n][2 * h + (j >> 1)];
                    const uint32_t b0 = j & 1 ? q.z : q.x, b1 = j & 1 ? q.w : q.y;
                    mma_e4m3(p[n], a0, a1, a2, a3, b0, b1);
                    mma_e4m3(p[n], 0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u, b0, b1);   // -8 2^-9
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(s0, p[n][0], acc[n][0]);
                acc[n][1] = fmaf(s0, p[n][1], acc[n][1]);
                acc[n][2] = fmaf(s1, p[n][2], acc[n][2]);
                acc[n][3] = fmaf(s1, p[n][3], acc[n][3]);
            }
        } else {
            const uint32_t ea = lds32(sa + 4 * h), eb = lds32(sb + 4 * h);
#pragma unroll
            for (int j2 = 0; j2 < 2; ++j2) {
                const float2 s0 = e8m0x2_to_f32(ea >> (16 * j2)), s1 = e8m0x2_to_f32(eb >> (16 * j2));
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const int j = 2 * j2 + jj;
                    const uint32_t at = (((h * 4 + j) ^ g) << 4) + 4 * t;
                    const uint32_t a = lds32(row_a + at), c = lds32(row_b + at);
                    const uint32_t a0 = ((a << 4) & 0x80808080u) | ((a << 2) & 0x1C1C1C1Cu);
                    const uint32_t a2 = (a & 0x80808080u) | ((a >> 2) & 0x1C1C1C1Cu);
                    const uint32_t a1 = ((c << 4) & 0x80808080u) | ((c << 2) & 0x1C1C1C1Cu);
                    const uint32_t a3 = (c & 0x80808080u) | ((c >> 2) & 0x1C1C1C1Cu);
                    const float f0 = jj ? s0.y : s0.x, f1 = jj ? s1.y : s1.x;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (NT > 1 && !((live >> n) & 1)) continue;
                        const uint4& q = b[n][2 * h + (j >> 1)];
                        float p[4] = {};
                        mma_e4m3(p, a0, a1, a2, a3, jj ? q.z : q.x, jj ? q.w : q.y);
                        acc[n][0] = fmaf(f0, p[0], acc[n][0]);
                        acc[n][1] = fmaf(f0, p[1], acc[n][1]);
                        acc[n][2] = fmaf(f1, p[2], acc[n][2]);
                        acc[n][3] = fmaf(f1, p[3], acc[n][3]);
                    }
                }
            }
        }
    }
}
// The power of two that piece_mma's sums lack (the E4M3 encodings of the weights).
template <bool kMx>
constexpr float kDecodeLadder = kMx ? 64.0f : 512.0f;

// The same for 16 rows x 64 bf16 weights; b: the lane's eight values of each half (32 columns).
template <int NT>
__device__ __forceinline__ void piece_mma_bf16(uint32_t row_a, uint32_t row_b, const uint4 (&b)[NT][2], float (&acc)[NT][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t at = ((h * 4 + t) ^ g) << 4;
        const uint4 wa = lds128(row_a + at), wb = lds128(row_b + at);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            mma_bf16(acc[n], wa.x, wb.x, wa.y, wb.y, b[n][h].x, b[n][h].y);
            mma_bf16(acc[n], wa.z, wb.z, wa.w, wb.w, b[n][h].z, b[n][h].w);
        }
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

    // max |x| of the tokens: 16 / (T rounded up to a power of two) warps a token
    const int twarps = kDecodeWarps >> (T > 8 ? 4 : T > 4 ? 3 : T > 2 ? 2 : T > 1 ? 1 : 0);
    const int tok = warp / twarps, tpart = warp % twarps;
    const uint4* xrow = reinterpret_cast<const uint4*>(p.x + (int64_t)tok * p.H);
    if (!producer && tok < T) {
        float a = 0.0f;
        for (int c = tpart * 32 + lane; c < p.H / 8; c += twarps * 32) a = fmaxf(a, amax8(__ldg(xrow + c)));
        a = warp_max(a);
        if (lane == 0) atomicMax(&S.amax[tok], __float_as_uint(a));
    }

    const float* logits = p.logits;
    if (p.wr) {   // logits of experts 2 c and 2 c + 1, then of those 2 G further: eight warps an expert
        logits = p.ws_logits;
        const int half = warp >> 3, part = warp & 7, HC = p.H / 8;
        for (int e0 = 2 * cta; e0 < p.E; e0 += 2 * G) {
            const int e = e0 + half;
            float acc[8 * NT];
#pragma unroll
            for (int j = 0; j < 8 * NT; ++j) acc[j] = 0.0f;
            if (!producer && e < p.E) {
                const uint4* w4 = reinterpret_cast<const uint4*>(p.wr + (int64_t)e * p.H);
                for (int c = part * 32 + lane; c < HC; c += 256) {
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
                    for (int w = 0; w < 8; ++w) s += red[(hh * 8 + w) * 8 * NT + j];
                    p.ws_logits[(int64_t)j * p.E + e0 + hh] = s;
                }
            }
            __syncthreads();
        }
        cg::this_grid().sync();
    }

    // S2: token t by warp 16 - t (the streaming warp has nothing else to do yet)
    {
        const int tt = kDecodeWarps - warp;
        if (tt < T) {
            const float* l = logits + (int64_t)tt * p.E;
            int* ids = S.ids + tt * k;
            float* gates = S.gates + tt * k;
            if (p.E <= 256) topk_row<8, true>(l, p.E, k, ids, gates, lane);
            else topk_row<32, true>(l, p.E, k, ids, gates, lane);
            __syncwarp();
            if (lane < k) atomicOr(&S.bitmap[ids[lane] >> 5], 1u << (ids[lane] & 31));
        }
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
            const int upu = 16 >> R.log;
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
        const int upu = 16 >> p.rb.log;
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
    if (tok < T) {
        const float s = __fdiv_rn(__uint_as_float(S.amax[tok]), kFp8Max);
        for (int c = tpart * 32 + lane; c < p.H / 8; c += twarps * 32) {
            const uint2 q = perm8(quant8(__ldg(xrow + c), s));
            int piece, i, tt, odd;
            frag_place<kMx>(c, piece, i, tt, odd);
            const uint32_t at = frags + ((piece * NT + (tok >> 3)) * 4 + i) * 512 + ((tok & 7) * 4 + tt) * 16 + odd * 8;
            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at), "r"(q.x), "r"(q.y) : "memory");
        }
    }
    consumers_sync();

    DecodeRing r;
    bool ok = true;
    int buf = 0;
    const int red_words = kDecodeWarps * NT * 128;
    auto wait_full = [&]() { ok = ok && ws::wait(&S.full[r.slot], r.phase, &S.abort); };
    auto release = [&]() {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.empty[r.slot]);
        r.next(p.slots);
    };
    // Leaves every warp's sums in `red` and returns the buffer; the caller reads it before the next call.
    auto share_sums = [&](const float (&acc)[NT][4]) {
        float* dst = red + buf * red_words;
        if (p.red_bufs > 1) buf ^= 1;
        else consumers_sync();                        // the last readers of the one buffer are done
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[(warp * NT * 4 + n * 4 + i) * 32 + lane] = acc[n][i];
        consumers_sync();
        return dst;
    };

    // phase A, routed units: h = silu(G) U
    for (int u = a0; u < a1; u += 16 >> p.ra.log) {
        const int slot_unit = warp >> p.ra.log, piece0 = warp & ((1 << p.ra.log) - 1);
        const int uu = u + slot_unit, ei = uu / nb;
        float acc[NT][4] = {};
        uint32_t live = 0;
        if (uu < a1) {
            const uint32_t toks = S.tokens[ei];
#pragma unroll
            for (int n = 0; n < NT; ++n) live |= (toks >> (8 * n) & 0xFFu) ? 1u << n : 0u;
        }
        for (int c = 0; c < p.ra.chunks; ++c) {
            wait_full();
            const int piece = c * 16 + piece0, halves = min(2, p.H / 128 - 2 * piece);
            if (ok && uu < a1 && halves > 0) {
                const uint32_t base = ring + r.slot * p.slot_bytes;
                const uint32_t row = base + slot_unit * (2048 << p.ra.log) + piece0 * 1024 + g * 128;
                const uint32_t sc = base + kDecodeStage + (slot_unit * 16 + g) * row_scale_a + piece * (kMx ? 8 : 4);
                uint4 b[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) b[n][i] = lds128(frags + ((piece * NT + n) * 4 + i) * 512 + lane * 16);
                piece_mma<kMx, NT>(row, row + (1024 << p.ra.log), sc, sc + 8 * row_scale_a, halves, b, live, acc);
            }
            release();
        }
        const float* sums = share_sums(acc);
        const int per = 1 << p.ra.log, n_out = (16 >> p.ra.log) * 64 * NT;
        for (int s = threadIdx.x; s < n_out; s += 32 * kDecodeWarps) {
            const int c1 = (s >> 5) & 1, n = (s >> 6) % NT, q = s / (64 * NT);
            const int col = n * 8 + t * 2 + c1, unit = u + q;
            if (col >= T || unit >= a1) continue;
            const int e = unit / nb;
            if (!((S.tokens[e] >> col) & 1u)) continue;
            float gt = 0.0f, up = 0.0f;
            for (int w = 0; w < per; ++w) {
                const float* f = sums + ((q * per + w) * NT * 4 + n * 4 + c1) * 32 + lane;
                gt += f[0];
                up += f[64];
            }
            const float sx = __fdiv_rn(__uint_as_float(S.amax[col]), kFp8Max) * kDecodeLadder<kMx>;
            p.h[(int64_t)(col * k + S.pick[e][col]) * p.N + (unit % nb) * 8 + g] = silu(gt * sx) * (up * sx);
        }
    }
    // phase A, shared experts: the same on bf16 weights and tokens
    for (int u = s0; u < s1; u += 16 >> p.rs.log) {
        const int slot_unit = warp >> p.rs.log, piece0 = warp & ((1 << p.rs.log) - 1);
        float acc[NT][4] = {};
        for (int c = 0; c < p.rs.chunks; ++c) {
            const int piece = c * 16 + piece0;
            const bool mine = u + slot_unit < s1 && piece < p.rs.pieces;
            uint4 b[NT][2] = {};
            if (mine) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (n * 8 + g < T)
                            b[n][h] = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(n * 8 + g) * p.H) + piece * 8 + h * 4 + t);
            }
            wait_full();
            if (ok && mine) {
                const uint32_t row = ring + r.slot * p.slot_bytes + slot_unit * (2048 << p.rs.log) + piece0 * 1024 + g * 128;
                piece_mma_bf16<NT>(row, row + (1024 << p.rs.log), b, acc);
            }
            release();
        }
        const float* sums = share_sums(acc);
        const int per = 1 << p.rs.log, n_out = (16 >> p.rs.log) * 64 * NT;
        for (int s = threadIdx.x; s < n_out; s += 32 * kDecodeWarps) {
            const int c1 = (s >> 5) & 1, n = (s >> 6) % NT, q = s / (64 * NT);
            const int col = n * 8 + t * 2 + c1, unit = u + q;
            if (col >= T || unit >= s1) continue;
            float gt = 0.0f, up = 0.0f;
            for (int w = 0; w < per; ++w) {
                const float* f = sums + ((q * per + w) * NT * 4 + n * 4 + c1) * 32 + lane;
                gt += f[0];
                up += f[64];
            }
            const float a = silu(gt) * up;
            const uint16_t hi = f32_to_bf16_bits(a);   // hi + lo: 16 bits of the activation
            const int64_t at = (int64_t)col * p.n_shared * p.Ns + unit * 8 + g;
            p.act_hi[at] = hi;
            p.act_lo[at] = f32_to_bf16_bits(a - bf16_bits_to_f32(hi));
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
        for (int c = threadIdx.x; c < p.N / 8; c += 32 * kDecodeWarps) {
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
            *reinterpret_cast<uint2*>(p.hq + (int64_t)q * hq_row + piece * 256 + i * 64 + tt * 16 + odd * 8) = perm8(codes);
        }
        if (threadIdx.x == 0) p.gs[q] = S.gates[q] * s * kDecodeLadder<kMx>;
    }
    cg::this_grid().sync();
    if (threadIdx.x < P) S.gs[threadIdx.x] = __ldcg(p.gs + threadIdx.x);
    consumers_sync();

    // phase B
    const int upu = 16 >> p.rb.log, slot_unit = warp >> p.rb.log, piece0 = warp & ((1 << p.rb.log) - 1);
    for (int v = v0; v < v1;) {
        const int tile = v / V, lo = v - tile * V, hi = min(V, lo + v1 - v);
        float acc[NT][4] = {};
        for (int q = lo; q < hi; q += upu) {
            const int id = q + slot_unit;
            const bool mine = id < hi, routed = id < Vr;
            const int per = routed ? p.rb.chunks : p.shared_chunks, o = routed ? id : id - Vr;
            const int ei = o / per, piece = ((o % per) << p.rb.log) + piece0;
            const uint32_t base = ring + r.slot * p.slot_bytes;
            const uint32_t row = base + slot_unit * (2048 << p.rb.log) + piece0 * 2048 + g * 128;
            if (mine && routed) {
                const int halves = min(2, p.N / 128 - 2 * piece);
                const uint32_t toks = S.tokens[ei];
                uint4 b[NT][4] = {};
                uint32_t live = 0;
                if (halves > 0) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        live |= (toks >> (8 * n) & 0xFFu) ? 1u << n : 0u;
                        const int col = n * 8 + g;
                        if ((toks >> col) & 1u) {
                            const uint4* src = reinterpret_cast<const uint4*>(
                                p.hq + (int64_t)(col * k + S.pick[ei][col]) * hq_row + piece * 256) + t;
#pragma unroll
                            for (int i = 0; i < 4; ++i) b[n][i] = __ldcg(src + i * 4);
                        }
                    }
                }
                wait_full();
                if (ok && halves > 0) {
                    float y[NT][4] = {};
                    const uint32_t sc = base + kDecodeStage + (slot_unit * 16 + g) * row_scale_b + piece * (kMx ? 8 : 4);
                    piece_mma<kMx, NT>(row, row + 1024, sc, sc + 8 * row_scale_b, halves, b, live, y);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c1 = 0; c1 < 2; ++c1) {
                            const int col = n * 8 + t * 2 + c1;
                            if ((toks >> col) & 1u) {   // the other columns hold nothing of this expert's
                                const float f = S.gs[col * k + S.pick[ei][col]];
                                acc[n][c1] = fmaf(f, y[n][c1], acc[n][c1]);
                                acc[n][c1 + 2] = fmaf(f, y[n][c1 + 2], acc[n][c1 + 2]);
                            }
                        }
                }
            } else {
                uint4 bh[NT][2] = {}, bl[NT][2] = {};
                const bool live = mine && piece < p.Ns / 64;
                if (live) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (n * 8 + g < T) {
                                const int64_t at = ((int64_t)(n * 8 + g) * p.n_shared + ei) * (p.Ns / 8) + piece * 8 + h * 4 + t;
                                bh[n][h] = __ldcg(reinterpret_cast<const uint4*>(p.act_hi) + at);
                                bl[n][h] = __ldcg(reinterpret_cast<const uint4*>(p.act_lo) + at);
                            }
                }
                wait_full();
                if (ok && live) {
                    piece_mma_bf16<NT>(row, row + 1024, bh, acc);
                    piece_mma_bf16<NT>(row, row + 1024, bl, acc);
                }
            }
            release();
        }
        const float* sums = share_sums(acc);
        const bool whole = hi - lo == V;
        float* part = p.part + (int64_t)(tile + cta) * (128 * NT);   // tile + cta: its own for each (tile, CTA)
        float sum = 0.0f;
        const int s = threadIdx.x;
        if (s < 128 * NT)
            for (int w = 0; w < kDecodeWarps; ++w) sum += sums[w * NT * 128 + s];
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
        v += hi - lo;
    }
    if (!ok) give_up();
}

// ---- host ---------------------------------------------------------------------------------------

struct DecodePlan {
    size_t logits, h, hq, gs, act, part, count, total;
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
    const size_t red = (size_t)kDecodeWarps * NT * 128 * 4;
    const size_t scale_a = (size_t)(16 >> q.ra.log) * 16 * (kMx ? q.H / 32 : q.H / 64);
    const size_t scale_b = (size_t)(16 >> q.rb.log) * 16 * (kMx ? q.N / 32 : q.N / 64);
    q.slot_bytes = static_cast<int>(align_up(kDecodeStage + std::max(scale_a, scale_b), 1024));
    const size_t frag = (size_t)((q.H + 255) / 256) * NT * kDecodePiece;
    // 227 KB a CTA; long rows of two token blocks take one sum buffer so that two slots still fit
    const size_t room = 227 * 1024 - sizeof(DecodeShared) - 1024 - 256 - frag;
    q.red_bufs = room >= 2 * red + 3 * (size_t)q.slot_bytes ? 2 : 1;
    q.slots = static_cast<int>(std::min<size_t>(kDecodeMaxSlots, (room - q.red_bufs * red) / q.slot_bytes));
    if (q.slots < 2) return MOE_ERR_UNSUPPORTED_SHAPE;
    const size_t smem = 1024 + (size_t)q.slots * q.slot_bytes + frag + q.red_bufs * red;
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
