// decode.cuh — the whole routed MoE layer for a few tokens (T <= 16), on W4A8 or MXFP4 experts, in
// one kernel.
//
// The arithmetic of moe_w4a8_forward: S1 (FP8 of the tokens), S2 (top-k, gates), S4 (gate, up,
// SwiGLU), S5 (FP8 of h for each routed pair), S6 (down), S7 (the gated sum) and S8 (shared
// experts), with the experts' weights in pack-quantized INT4 or in MXFP4.
//
// What bounds it: a few tokens use each weight once or twice, so the time is the reading of the touched experts' weights
// (13 MB an expert at H = 4096, N = 2048) and, at one token, a chain of latencies.  One persistent cooperative grid (one
// CTA an SM) therefore reads every weight byte once, and the stream does not stop at the layer's inner dependency: the
// weights of the down projections do not depend on h, so the rings fill with them while the grid finishes h.
//
//   prologue  (router form: the logits, a barrier.)  Every CTA ranks the logits itself, a warp a token, lists the touched
//             experts and starts streaming; meanwhile the multiplying warps quantize the tokens that its experts need into
//             B fragments in shared memory: f16 for up to six tokens, FP8 (widened at each use) beyond, since a CTA's
//             share of the experts (one to four of them) seldom has more
//   gate/up   unit = 8 gate rows and the same 8 up rows of one touched expert, all of K; a phase's units are split evenly
//             over the CTAs; h (fp32) goes to the workspace.  Then the shared experts' (bf16)
//   barrier   each CTA quantizes the rows of h that its down units read into its own shared memory; where some CTA's rows
//             do not fit, CTA r quantizes row r into the workspace and a second barrier follows
//   down      unit = 16 rows of one touched expert (then of a shared expert); gated rows to the workspace
//   barrier   the rows are added in selection order
//
// Eight warps multiply and four stream for them.  A warp has rings of its own (two to four slots of 8 KB, chunks of 4
// pieces of 16 rows x 128 bytes in the 128-byte swizzle, one TMA box a row set), so that no warp waits for another's data;
// a streaming warp has a lane for each ring it feeds.  Issued by the multiplying warps themselves a chunk's copies cost
// them some 1,000 cycles.  A row's scales come beside its unit's first chunk where the buffers fit, else they are read in
// place.  Measured against each other on one build, in us for W4A8 (T = 1, 8 and 16) and MXFP4 (T = 1 and 8) at the sizes
// below, the same inputs over and over:
//   8 + 4 warps                          37.8  137  285   41  138
//   12 + 4 (chunks of two pieces)        36.9  146  336   40  146
//   9 + 3                                40.3  143  333   44  154
//   10 + 2                               39.6  145  339   44  163
//   rows of h always by the workspace    40.9  148  314   44  150
//   scales always in place               41.7  151  313   46  158
//   fragments always FP8                 39.3  146  304   43  148
//   pieces unrolled twice                40.1  144  300   43  142   (rolled, the loop stays in the instruction cache)
//
// The products run on mma.sync m16n8k16 (f16, fp32 sums): a unit's 16 rows are the M, up to eight tokens the N.  tcgen05
// would put 128 rows a tile, and the widened weights through TMEM, for the same eight columns.  E4M3 values are exact in
// f16, and so are the weights:
//   INT4:  a nibble n = code + 8 left where it lies in a 16-bit half is the f16 subnormal n 2^-24 (bits 0..3) or n 2^-20
//          (bits 4..7, whose tokens' values carry 2^-4), so widening a packed word costs four ANDs and a shift; the
//          accumulator starts at -8 2^-24 sum q, which takes the offset off again.  A group's fp32 sum thus runs over
//          numbers of up to 23 sum |q|, where the result has 8 sum |q| at most: it is exact while 23 sum |q| < 2^15 (codes
//          are multiples of 2^-9), and beyond that loses the last bits of the group's smallest codes.
//   MXFP4: cvt.rn.f16x2.e2m1x2.
// (mma.sync on E4M3 is no way round the conversion: with it the layer at T = 8 took 213 us.)  A group's (block's) partial
// sum is scaled in fp32 by its weight scale: one promotion every 128 (32) weights.  Shared experts run on the bf16 MMA,
// their activation as bf16 hi + lo halves (16 bits of it).
//
// Measured, E = 256, top 6, H = 4096, N = 2048, each call with other tokens and experts (16 calls or more touch all 3.3 GB):
// W4A8 from logits
//   T                                 1     2     4     8    12    16
//   us                             38.3  53.4  83.0   136   183   227      (78 MB at T = 1: 31 % of HBM's measured 6.56 TB/s;
//   moe_w4a8_forward               46.5  64.9  92.9   147   194   238       578 MB at T = 8: 65 %)
//   with two shared experts        64.3  79.3   107   160   242   286
//   moe_w4a8_forward                143   160   193   244   293   314
// and MXFP4 38.6, 55.2, 83.6, 138, 185 and 257.  The router form takes 2 to 5 us more.  With the same six experts in every
// call, which L2 then holds, T = 1 takes 34 to 36 us.  The gain over the forward shrinks with T, hence 16.
// At T = 1 the chain is: lists 4.6 us, tokens quantized 9.5, gate/up 22, barrier 24, h quantized 26, down 32, sums 34.  At
// T = 8 the same grid reads the bytes in 104 us when nothing is multiplied, and the multiplying warps find their chunks
// there (they wait 5 % of the gate/up phase).  A piece is some 200 warp instructions (80 of them the widening's half-rate
// logic) in 640 cycles, two warps a scheduler; no unit is saturated (issue slots 42 % and ALU 41 % of the whole kernel), so
// what is left are the fixed latencies of the widening and the MMAs, which two warps do not cover.  Loading half a piece
// ahead of the MMAs (147 us), or addresses that run from piece to piece (145), hide latency but add instructions.
#pragma once
#include <cooperative_groups.h>
#include <type_traits>
#include "forward.cuh"
#include "mxfp4.cuh"

namespace moe {

constexpr int kDecodeMaxT = 16;
constexpr int kDecodeWarps = 8;                          // that multiply
constexpr int kDecodeStreams = 4;                        // that stream the weights for them
constexpr int kDecodeThreads = 32 * (kDecodeWarps + kDecodeStreams);
constexpr int kDecodeMaxPairs = kDecodeMaxT * kMaxK;
constexpr int kDecodeMaxSlots = 4;

struct DecodeLayer {
    int E, H, N;
    const uint8_t *w[3];          // gate, up [E, N, H/2], down [E, H, N/2]
    const void *s[3];             // INT4: bf16 [.., K/128]; MXFP4: E8M0 [.., K/32]
    int n_shared, shared_N;
    const uint16_t *sw[3];        // shared experts' gate, up, down (bf16)
};

// Rows of one weight matrix: `pieces` of 128 bytes a row; a chunk is `cp` of them for the 16 rows of a
// unit, a unit `chunks` chunks.
struct DecodeRows {
    int pieces, cp, chunks;
};

struct alignas(64) DecodeParams {
    CUtensorMap map[6];           // gate, up, down, shared gate, up, down
    const uint8_t* scale[3];
    const uint16_t *x, *wr;
    const float* logits;
    uint16_t* out;
    float *h, *gs, *y, *hsum, *ws_logits;
    uint8_t* hq;
    uint16_t *act_hi, *act_lo;
    DecodeRows rows[4];           // gate/up, shared gate/up, down, shared down
    int E, H, N, k, T, n_shared, Ns;
    int slots, slot_bytes, scale_bytes;   // scale_bytes: of one of a warp's `slots` scale buffers, 0: read in place
    int frag_bytes, max_tokens, max_rows;   // of the fragments in shared memory; f16 rows of x and of h that fit there
    int flat;                     // bit i set: map i is 2-D (rows are not whole pieces)
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Shared memory by its offset in the dynamic array (plain loads: the compiler may move them between barriers).
extern __shared__ __align__(16) uint8_t g_decode_smem[];
__device__ __forceinline__ uint4 lds128(uint32_t a) { return *reinterpret_cast<const uint4*>(g_decode_smem + a); }
__device__ __forceinline__ uint32_t lds32(uint32_t a) { return *reinterpret_cast<const uint32_t*>(g_decode_smem + a); }
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Row g of an MMA's eight is row lane_row() of the eight in shared memory: eight consecutive lanes (two g) then
// read rows whose swizzle differs in bit 2, so a 16-byte load of four neighbouring chunks of each has no bank conflict.
__device__ __forceinline__ int lane_row(int g) { return (g >> 1) | ((g & 1) << 2); }
// Eight codes in column order -> the order in which the weights' widening pairs them: for INT4 the
// nibbles of a word come out as (0,4) (1,5) (2,6) (3,7), for MXFP4 as they are.
template <bool kMx>
__device__ __forceinline__ uint2 frag_order(uint2 c) {
    return kMx ? c : make_uint2(__byte_perm(c.x, c.y, 0x5140), __byte_perm(c.x, c.y, 0x7362));
}
// Eight codes in that order -> the B registers of two MMAs.
template <bool kMx>
__device__ __forceinline__ uint4 frag_f16(uint2 c) {
    uint4 r;
    asm("{\n\t.reg .b16 h0, h1, h2, h3;\n\tmov.b32 {h0, h1}, %4;\n\tmov.b32 {h2, h3}, %5;\n\tcvt.rn.f16x2.e4m3x2 %0, h0;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h1;\n\tcvt.rn.f16x2.e4m3x2 %2, h2;\n\tcvt.rn.f16x2.e4m3x2 %3, h3;\n\t}"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(c.x), "r"(c.y));
    if constexpr (!kMx) {   // the nibbles in bits 4..7 stand for 16 n: 2^-4
        const __half2 m = __half2half2(__ushort_as_half(0x2C00));
        const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&r.y), m), w = __hmul2(*reinterpret_cast<const __half2*>(&r.w), m);
        r.y = *reinterpret_cast<const uint32_t*>(&y);
        r.w = *reinterpret_cast<const uint32_t*>(&w);
    }
    return r;
}
// A token's (or pair's) row of B fragments: pieces of 256 columns; in a piece, word i = 4 h + j of lane t
// holds the eight columns that word j of the lane's weights in half h covers: 32 t + 8 j (INT4: a lane
// reads 16 bytes of a weight row at once) or 32 j + 8 t (MXFP4: the lanes' words j are one block).  As
// f16 a word is 16 bytes at 64 i + 16 t, as FP8 8 bytes at 64 (i / 2) + 16 t + 8 (i % 2).
template <bool kMx>
__device__ __forceinline__ void frag_place(int c8, int& piece, int& i, int& t) {
    const int idx = c8 & 15, j = kMx ? idx >> 2 : idx & 3;
    t = kMx ? idx & 3 : idx >> 2;
    piece = c8 >> 5;
    i = 4 * ((c8 >> 4) & 1) + j;
}

// Bytes of a row of fragments (64 more than they take: neighbouring rows then start in different banks).
template <bool kF8>
__host__ __device__ constexpr uint32_t frag_row_bytes(int pieces) { return pieces * (kF8 ? 256 : 512) + 64; }

constexpr float kNibbleOffset = -8.0f / 16777216.0f;   // -8 2^-24
// A routed product's sum times a scale.  INT4 sums lack 2^24: it is put back before the scale (exactly), since scale 2^24
// overflows for rows of 10^34 whose results do not.
template <bool kMx>
__device__ __forceinline__ float scaled(float acc, float scale) { return (kMx ? acc : acc * 16777216.0f) * scale; }

// A lane's scales (rows g and g + 8) of a piece, from the rows' scales in shared memory (offsets) or, where
// the buffers do not fit, in place.
template <bool kSmem>
struct DecodeScales {
    using At = std::conditional_t<kSmem, uint32_t, const uint8_t*>;
    At a, b;
    template <class V>
    static __device__ __forceinline__ V load(At at) {
        if constexpr (kSmem) return *reinterpret_cast<const V*>(g_decode_smem + at);
        else return __ldg(reinterpret_cast<const V*>(at));
    }
    __device__ __forceinline__ void int4(int halves, float (&s0)[2], float (&s1)[2]) const {
        const uint32_t second = halves > 1 ? 2 : 0;   // (the first again: its sums are dropped)
        s0[0] = bf16_bits_to_f32(load<uint16_t>(a));
        s1[0] = bf16_bits_to_f32(load<uint16_t>(b));
        s0[1] = bf16_bits_to_f32(load<uint16_t>(a + second));
        s1[1] = bf16_bits_to_f32(load<uint16_t>(b + second));
    }
    __device__ __forceinline__ void mx(int h, float (&s0)[4], float (&s1)[4]) const {
        e8m0x4_to_f32(load<uint32_t>(a + 4 * h), s0);
        e8m0x4_to_f32(load<uint32_t>(b + 4 * h), s1);
    }
};

// acc += the products of one piece (16 rows x 256 weights) with the B fragments f of eight token
// columns.  row_a / row_b: the lane's rows g and g + 8; sa / sb: those rows' scales at the piece;
// halves: 1 when only the first 128 columns lie inside the row.  off: INT4, where the accumulators of
// the lane's two columns start, by half: -8 2^-24 sum q.
template <bool kMx, class Scales>
__device__ __forceinline__ void piece_mma(uint32_t row_a, uint32_t row_b, const Scales& sc, int halves,
                                          const uint4 (&f)[8], float2 off0, float2 off1, float (&acc)[4]) {
    const int lane = threadIdx.x & 31, g = lane_row(lane >> 2), t = lane & 3;
    if constexpr (!kMx) {
        const uint32_t at0 = (t ^ g) << 4;
        uint4 wa[2], wb[2];
        float p[2][2][4], s0[2], s1[2];   // [half][word parity]: four independent chains
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            wa[h] = lds128(row_a + (at0 ^ (h * 64)));
            wb[h] = lds128(row_b + (at0 ^ (h * 64)));
        }
        sc.int4(halves, s0, s1);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t a = word(wa[h], j) >> (8 * s), c = word(wb[h], j) >> (8 * s);
                    const uint32_t a0 = a & 0x000F000Fu, a1 = c & 0x000F000Fu, a2 = a & 0x00F000F0u, a3 = c & 0x00F000F0u;
                    const uint32_t b0 = s ? f[4 * h + j].z : f[4 * h + j].x, b1 = s ? f[4 * h + j].w : f[4 * h + j].y;
                    const float2 o = h ? off1 : off0;   // (columns 2 t and 2 t + 1)
                    if (j == 0 && s == 0) mma_f16(p[h][0], a0, a1, a2, a3, b0, b1, o.x, o.y, o.x, o.y);
                    else if (j == 1 && s == 0) mma_f16(p[h][1], a0, a1, a2, a3, b0, b1, 0.0f, 0.0f, 0.0f, 0.0f);
                    else mma_f16(p[h][j & 1], a0, a1, a2, a3, b0, b1);
                }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h && halves < 2) break;
            acc[0] = fmaf(s0[h], p[h][0][0] + p[h][1][0], acc[0]);
            acc[1] = fmaf(s0[h], p[h][0][1] + p[h][1][1], acc[1]);
            acc[2] = fmaf(s1[h], p[h][0][2] + p[h][1][2], acc[2]);
            acc[3] = fmaf(s1[h], p[h][0][3] + p[h][1][3], acc[3]);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h && halves < 2) break;
            float s0[4], s1[4];
            sc.mx(h, s0, s1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t at = (((h * 4 + j) ^ g) << 4) + 4 * t;
                uint32_t a[4], c[4];
                e2m1x8_to_f16(lds32(row_a + at), a);
                e2m1x8_to_f16(lds32(row_b + at), c);
                const uint4& q = f[4 * h + j];
                float p[4];
                mma_f16(p, a[0], c[0], a[1], c[1], q.x, q.y, 0.0f, 0.0f, 0.0f, 0.0f);
                mma_f16(p, a[2], c[2], a[3], c[3], q.z, q.w);
                acc[0] = fmaf(s0[j], p[0], acc[0]);
                acc[1] = fmaf(s0[j], p[1], acc[1]);
                acc[2] = fmaf(s1[j], p[2], acc[2]);
                acc[3] = fmaf(s1[j], p[3], acc[3]);
            }
        }
    }
}

// The same for 16 rows x 64 bf16 weights of one piece; b: the lane's eight values of each half (32 columns).
__device__ __forceinline__ void piece_mma_bf16(uint32_t row_a, uint32_t row_b, const uint4 (&b)[2], float (&acc)[4]) {
    const int lane = threadIdx.x & 31, g = lane_row(lane >> 2), t = lane & 3;
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

// Whether the phase of the given parity has completed (returns at once).
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(tc::smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
constexpr int kMul = 32 * kDecodeWarps;   // threads that multiply
__device__ __forceinline__ void multipliers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kMul) : "memory"); }

// The first unit of CTA c's even share of n units.
__device__ __forceinline__ int share(int n, int c, int G) { return static_cast<int>((unsigned)n * (unsigned)c / (unsigned)G); }   // n c < 2^32: n <= 2^17, a few hundred CTAs

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

// Row maxima are taken over the bits of the magnitudes: as integers they order like the values, and a NaN is the largest,
// so a row that holds one gets a scale and codes of NaN, and not the scale of the rest of it.
__device__ __forceinline__ unsigned magnitude_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ unsigned amax_bits8(const uint4& v) {   // of eight bf16
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    unsigned m = 0u;
#pragma unroll
    for (int q = 0; q < 4; ++q) m = max(m, max((u[q] << 16) & 0x7FFFFFFFu, u[q] & 0x7FFF0000u));
    return m;
}

// The FP8 codes of a row whose largest magnitude is amax: e4m3(x / s) with s = amax / 448, by r = RN(1 / s), q = RN(x r) and
// q + r (x - q s) with the remainder in a fused multiply-add (the correction of P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990).  q is off by up to 1.5 units in its last place, more than the
// theorem there allows, but the corrected quotient is within 2^-21 of one before it is rounded, so a code could differ from
// that of IEEE division only where x / s lies that near to the middle of two floats beside a tie of two codes; of all
// mantissas of x and s 255 pairs do, and every one of them is rounded right (tests/test_decode_division_cpu.py).  The method
// needs r normal and remainders that do not underflow where they matter; rows outside [2^-60, 2^60] divide plainly.
struct RowQuant {
    float s, r;
    bool plain;
    static __device__ __forceinline__ RowQuant of(float amax) {
        RowQuant q;
        q.s = __fdiv_rn(amax, kFp8Max);
        q.plain = !(q.s >= 0x1p-60f && q.s <= 0x1p60f);
        q.r = q.plain ? 0.0f : __frcp_rn(q.s);
        return q;
    }
    __device__ __forceinline__ float divide(float x) const {
        if (plain) return __fdiv_rn(x, s);
        const float q = x * r;
        return fmaf(fmaf(-q, s, x), r, q);
    }
    __device__ __forceinline__ uint2 codes(const float (&x)[8]) const {
        uint32_t c[2] = {0u, 0u};
        if (s != 0.0f) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c[i >> 1] |= static_cast<uint32_t>(f32x2_to_e4m3x2(divide(x[2 * i]), divide(x[2 * i + 1]))) << (16 * (i & 1));
        }
        return make_uint2(c[0], c[1]);
    }
};

// A wait ran out: the status word is set, and the warp stays until its CTA's copies in flight (microseconds) have landed.
__device__ __forceinline__ void give_up() {
    if ((threadIdx.x & 31) == 0) atomicOr(&g_device_status, kStatusTimeout);
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 10000000ull) __nanosleep(100000);
}

struct DecodeShared {
    uint64_t full[kDecodeWarps][kDecodeMaxSlots], empty[kDecodeWarps][kDecodeMaxSlots];
    int ids[kDecodeMaxPairs];
    float gates[kDecodeMaxPairs], gs[kDecodeMaxPairs];
    int expert[kDecodeMaxPairs];                     // the touched experts, ascending
    uint32_t tokens[kDecodeMaxPairs];                // bit t: token t is routed to it
    uint8_t list[kDecodeMaxPairs][kDecodeMaxT];      // those tokens, ascending
    uint8_t pair[kDecodeMaxPairs][kDecodeMaxT];      // and their pairs t k + j
    uint32_t bitmap[kMaxE / 32];
    unsigned amax[kDecodeMaxT];
    float sx[kDecodeMaxT];
    float red[2 * (kDecodeWarps + kDecodeStreams) * kDecodeMaxT];
    unsigned row_max[16 + kDecodeWarps];             // of the multiplying warps' shares of a row of h, for two rows in turn
    int first[4], end[4], per_expert[4];             // this CTA's units of each phase, and how many an expert has
    int need[kDecodeMaxT], n_need;                   // the tokens of this CTA's gate/up experts,
    uint8_t need_at[kDecodeMaxT];                    // and a token's place among them
    uint8_t place[kDecodeMaxPairs][kDecodeMaxT];     // of expert place_e + i's pairs among the pairs of this CTA's down rows
    uint8_t row_pair[kDecodeMaxPairs];               // and those pairs
    int place_e, n_rows, most_rows;                  // n_rows of them; the most that any CTA has
    int n_experts;
    volatile int abort;
};

// A lane of a streaming warp: it loads for multiplying warp `to`, chunk after chunk of the warp's sequence: phases 0 gate/up,
// 1 shared gate/up, 2 down, 3 shared down; in a phase every kDecodeWarps-th of the CTA's units; a unit's chunks.
template <bool kMx>
struct DecodeStream {
    const DecodeParams& p;
    DecodeShared& S;
    int to;
    uint32_t slots0, scales0;                 // shared-memory addresses of the warp's slots and scale buffers
    int ph = 0, u = 0, c = 0, e = 0, b = 0;   // unit u is the b-th of expert (place) e
    int slot = 0, buf = 0;                    // ring slot; scale buffer of the unit
    uint32_t parity = 1;
    int ahead = 0;                            // chunks of the down phases issued
    bool ok = true;

    // Enters phase n, or the next in which the warp has units (4: none).
    __device__ __forceinline__ void enter(int n) {
        while (n < 4 && S.first[n] + to >= S.end[n]) ++n;
        ph = n;
        if (n < 4) {
            u = S.first[n] + to;
            e = u / S.per_expert[n];
            b = u - e * S.per_expert[n];
        }
    }
    __device__ __forceinline__ void issue() {
        const bool sh = ph & 1, down = ph >= 2;
        const DecodeRows R = p.rows[ph];
        const int per = down ? 16 : 8;
        const int row = (sh ? e : S.expert[e]) * (down ? p.H : sh ? p.Ns : p.N) + b * per;
        const int K = down ? p.N : p.H;
        const uint32_t rs = kMx ? K / 32 : K / 64, bytes = per * rs;
        const bool scales = !sh && c == 0 && p.scale_bytes;
        uint64_t* bar = &S.full[to][slot];
        tc::mbar_arrive_expect_tx(bar, 2048u * R.cp + (scales ? 16u * rs : 0u));
        const uint32_t dst = slots0 + slot * p.slot_bytes;
        for (int i = 0; i < (down ? 1 : 2); ++i) {
            const int m = (sh ? 3 : 0) + (down ? 2 : i);
            if (!((p.flat >> m) & 1)) {
                tma_load_3d(dst + i * (1024u * R.cp), &p.map[m], 0, row, c * R.cp, bar);
            } else {
                for (int x = 0; x < R.cp; ++x)
                    tma_load_2d_at(dst + i * (1024u * R.cp) + x * per * 128, &p.map[m], (c * R.cp + x) * 128, row, bar);
            }
            if (scales) bulk_load(scales0 + buf * p.scale_bytes + i * bytes, p.scale[down ? 2 : i] + (int64_t)row * rs, bytes, bar);
        }
        ahead += down;
        if (++slot == p.slots) { slot = 0; parity ^= 1u; }
        if (++c < R.chunks) return;
        c = 0;
        if (++buf == p.slots) buf = 0;
        u += kDecodeWarps;
        if (u >= S.end[ph]) {
            enter(ph + 1);
        } else {
            b += kDecodeWarps;
            for (const int n = S.per_expert[ph]; b >= n; b -= n) ++e;
        }
    }
    // Issues until every lane is through, or (up_to_barrier) as far into the down phases as the slots reach.
    __device__ __forceinline__ void run(bool up_to_barrier) {
        uint64_t t0 = 0;
        for (uint32_t n = 1;; ++n) {
            const bool active = ok && ph < 4 && !(up_to_barrier && ahead >= p.slots);
            if (!__any_sync(0xffffffffu, active)) return;
            const bool ready = active && mbar_test_wait(&S.empty[to][slot], parity);
            if (ready) issue();
            if (__any_sync(0xffffffffu, ready)) {
                t0 = 0;
                continue;
            }
            __nanosleep(20);
            if (t0 == 0) t0 = tc::globaltimer_ns();
            else if ((n & 255) == 0 && (S.abort || tc::globaltimer_ns() - t0 > 2000000000ull)) { S.abort = 1; ok = false; }
        }
    }
};

// A multiplying warp.
template <bool kMx, bool kScaleSmem>
struct DecodeWarp {
    const DecodeParams& p;
    DecodeShared& S;
    int warp, lane, g, t, r;                        // r: the lane's row
    uint32_t slots0, scales0, frags, sums;          // offsets in the dynamic shared memory; slots0, scales0: the warp's
    int slot = 0, buf = 0;
    uint32_t parity = 0;
    bool ok = true;

    __device__ __forceinline__ void wait_full() {   // (the warp goes on or gives up as one)
        if (ok) ok = __all_sync(0xffffffffu, ws::wait(&S.full[warp][slot], parity, &S.abort));
    }
    __device__ __forceinline__ void release() {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.empty[warp][slot]);
        if (++slot == p.slots) { slot = 0; parity ^= 1u; }
    }
    // The B fragments: f16 or (kF8) FP8 in shared memory, or (kGlobal) f16 in the workspace.
    template <bool kDown, bool kGlobal, bool kF8>
    __device__ __forceinline__ void routed();
    template <bool kDown>
    __device__ __forceinline__ void shared();
};

template <bool kMx, bool kScaleSmem>
template <bool kDown, bool kGlobal, bool kF8>
__device__ __forceinline__ void DecodeWarp<kMx, kScaleSmem>::routed() {
    constexpr int ph = kDown ? 2 : 0;
    const DecodeRows R = p.rows[ph];
    const int K = kDown ? p.N : p.H, pieces = (K + 255) / 256, per = S.per_expert[ph], end = S.end[ph];
    const uint32_t rs = kMx ? K / 32 : K / 64, step = kDown ? 2048 : 1024, row_b = kDown ? 1024u : 1024u * R.cp;
    const uint32_t frag_row = frag_row_bytes<kF8>(pieces);
    for (int u = S.first[ph] + warp; u < end; u += kDecodeWarps) {
        const int e = u / per, b = u - e * per, n_tok = __popc(S.tokens[e]);
        // where the columns' fragments are: by pair in the workspace, in shared memory by the pair's place among the CTA's;
        // for gate/up by token
        const uint8_t* of = !kDown ? S.list[e] : kGlobal ? S.pair[e] : S.place[e - S.place_e];
        const int col = 2 * t;                               // the lane's accumulators' first column of a block
        DecodeScales<kScaleSmem> sc;
        if constexpr (kScaleSmem) {
            sc.a = scales0 + buf * p.scale_bytes + r * rs;
            sc.b = sc.a + 8 * rs;
            if (++buf == p.slots) buf = 0;
        } else {
            const int64_t row = (int64_t)S.expert[e] * (kDown ? p.H : p.N) + b * (kDown ? 16 : 8) + r;
            sc.a = p.scale[kDown ? 2 : 0] + row * rs;
            sc.b = kDown ? sc.a + 8 * rs : p.scale[1] + row * rs;
        }
        // an unused column takes its block's first token: the loads coincide, and nobody reads its sums
        auto column = [&](int n, int i) {
            const int x = of[8 * n + i < n_tok ? 8 * n + i : 8 * n];
            return kDown ? x : (int)S.need_at[x];
        };
        // a block's columns: its fragments' offset and its group sums'
        const int who0 = column(0, g), o00 = kMx ? 0 : column(0, col) * pieces, o01 = kMx ? 0 : column(0, col + 1) * pieces;
        const uint32_t at0 = frags + who0 * frag_row + t * 16;
        float acc[2][4] = {};
        for (int c = 0; c < R.chunks; ++c) {
            wait_full();
            const int first = c * R.cp, last = min(first + R.cp, R.pieces);
            auto block = [&](int who, uint32_t at, uint32_t o0, uint32_t o1, float (&a)[4]) {
                const uint8_t* src = kGlobal ? p.hq + who * (int64_t)frag_row + t * 16 : nullptr;
                uint32_t row = slots0 + slot * p.slot_bytes + r * 128;
#pragma unroll 1
                for (int piece = first; piece < last; ++piece, row += step) {
                    uint4 f[8];
                    if constexpr (kGlobal) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = *reinterpret_cast<const uint4*>(src + piece * 512 + i * 64);
                    } else if constexpr (kF8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 v = lds128(at + piece * 256 + i * 64);
                            f[2 * i] = frag_f16<kMx>(make_uint2(v.x, v.y));
                            f[2 * i + 1] = frag_f16<kMx>(make_uint2(v.z, v.w));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = lds128(at + piece * 512 + i * 64);
                    }
                    float2 off0 = {}, off1 = {};
                    if constexpr (!kMx) {
                        float2 x, y;
                        if constexpr (kGlobal) {
                            x = reinterpret_cast<const float2*>(p.hsum)[o0 + piece];
                            y = reinterpret_cast<const float2*>(p.hsum)[o1 + piece];
                        } else {
                            x = *reinterpret_cast<const float2*>(g_decode_smem + sums + (o0 + piece) * 8);
                            y = *reinterpret_cast<const float2*>(g_decode_smem + sums + (o1 + piece) * 8);
                        }
                        off0 = make_float2(x.x, y.x);
                        off1 = make_float2(x.y, y.y);
                    }
                    const DecodeScales<kScaleSmem> s{sc.a + piece * (kMx ? 8 : 4), sc.b + piece * (kMx ? 8 : 4)};
                    piece_mma<kMx>(row, row + row_b, s, K / 128 - 2 * piece, f, off0, off1, a);
                }
            };
            if (ok) {
                block(who0, at0, o00, o01, acc[0]);
                if (n_tok > 8) {                             // (seldom: more than eight tokens)
                    const int who = column(1, g);
                    block(who, frags + who * frag_row + t * 16, kMx ? 0 : column(1, col) * pieces, kMx ? 0 : column(1, col + 1) * pieces, acc[1]);
                }
            }
            release();
        }
        // outputs: the lane's rows and its two token columns
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int c1 = 0; c1 < 2; ++c1) {
                if (8 * n + col + c1 >= n_tok) continue;
                const int pr = S.pair[e][8 * n + col + c1];
                if constexpr (kDown) {
                    p.y[(int64_t)pr * p.H + b * 16 + r] = scaled<kMx>(acc[n][c1], S.gs[pr]);
                    p.y[(int64_t)pr * p.H + b * 16 + r + 8] = scaled<kMx>(acc[n][c1 + 2], S.gs[pr]);
                } else {
                    const float sx = S.sx[S.list[e][8 * n + col + c1]];
                    p.h[(int64_t)pr * p.N + b * 8 + r] = silu(scaled<kMx>(acc[n][c1], sx)) * scaled<kMx>(acc[n][c1 + 2], sx);
                }
            }
    }
}

template <bool kMx, bool kScaleSmem>
template <bool kDown>
__device__ __forceinline__ void DecodeWarp<kMx, kScaleSmem>::shared() {   // bf16 weights, every token
    constexpr int ph = kDown ? 3 : 1;
    const DecodeRows R = p.rows[ph];
    const int per = S.per_expert[ph], end = S.end[ph];
    const uint32_t step = kDown ? 2048 : 1024, row_b = kDown ? 1024u : 1024u * R.cp;
    for (int u = S.first[ph] + warp; u < end; u += kDecodeWarps) {
        const int e = u / per, b = u - e * per;
        float acc[2][4] = {};
        for (int c = 0; c < R.chunks; ++c) {
            const int first = c * R.cp, n_here = min(R.cp, R.pieces - first);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                if (8 * n >= p.T) break;
                const int tk = min(8 * n + g, p.T - 1);      // (an unused column takes the last token's)
                uint4 v[4][kDown ? 2 : 1][2];                // a chunk has at most four pieces: all loads in flight at once
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int piece = first + min(i, n_here - 1);
                        if constexpr (kDown) {
                            const int64_t at = ((int64_t)tk * p.n_shared + e) * (p.Ns / 8) + piece * 8 + h * 4 + t;
                            v[i][0][h] = reinterpret_cast<const uint4*>(p.act_hi)[at];
                            v[i][1][h] = reinterpret_cast<const uint4*>(p.act_lo)[at];
                        } else {
                            v[i][0][h] = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)tk * p.H) + piece * 8 + h * 4 + t);
                        }
                    }
                if (n == 0) wait_full();
                if (!ok) break;
                uint32_t row = slots0 + slot * p.slot_bytes + r * 128;
#pragma unroll
                for (int i = 0; i < 4; ++i, row += step) {
                    if (i >= n_here) break;
#pragma unroll
                    for (int part = 0; part < (kDown ? 2 : 1); ++part) piece_mma_bf16(row, row + row_b, v[i][part], acc[n]);
                }
            }
            release();
        }
        if (++buf == p.slots) buf = 0;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int c1 = 0; c1 < 2; ++c1) {
                const int tk = 8 * n + 2 * t + c1;
                if (tk >= p.T) continue;
                if constexpr (kDown) {
                    float* y = p.y + ((int64_t)p.T * p.k + e * p.T + tk) * p.H + b * 16 + r;
                    y[0] = acc[n][c1];
                    y[8] = acc[n][c1 + 2];
                } else {
                    const float a = silu(acc[n][c1]) * acc[n][c1 + 2];
                    const uint16_t hi = f32_to_bf16_bits(a);   // hi + lo: 16 bits of the activation
                    const int64_t at = ((int64_t)tk * p.n_shared + e) * p.Ns + b * 8 + r;
                    p.act_hi[at] = hi;
                    p.act_lo[at] = f32_to_bf16_bits(a - bf16_bits_to_f32(hi));
                }
            }
    }
}

template <bool kMx, bool kScaleSmem>
__global__ void __launch_bounds__(kDecodeThreads, 1) k_decode(const __grid_constant__ DecodeParams p) {
    namespace cg = cooperative_groups;
    __shared__ DecodeShared S;
    const uint32_t smem0 = tc::smem_u32(g_decode_smem);
    const uint32_t ring = ((smem0 + 1023u) & ~1023u) - smem0;           // offsets in the dynamic shared memory
    const uint32_t scales = ring + kDecodeWarps * p.slots * p.slot_bytes;
    const uint32_t frags = scales + kDecodeWarps * p.slots * p.scale_bytes;
    const int pieces_x = (p.H + 255) / 256, pieces_h = (p.N + 255) / 256;
    const uint32_t row_h = frag_row_bytes<false>(pieces_h);
    const uint32_t sums = frags + p.frag_bytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = gridDim.x, cta = blockIdx.x;
    const int T = p.T, k = p.k, P = T * k;

    // ---- prologue ----
    if (threadIdx.x == 0) {
        for (int i = 0; i < kDecodeWarps * p.slots; ++i) {
            tc::mbar_init(&S.full[i / p.slots][i % p.slots], 1);
            tc::mbar_init(&S.empty[i / p.slots][i % p.slots], 1);
        }
        tc::fence_mbar_init();
        S.abort = 0;
        S.most_rows = 0;
    }
    if (warp == 1 && lane < (p.n_shared ? 6 : 3)) ws::prefetch_map(&p.map[lane]);
    for (int i = threadIdx.x; i < kMaxE / 32; i += kDecodeThreads) S.bitmap[i] = 0u;
    for (int i = threadIdx.x; i < kDecodeMaxPairs; i += kDecodeThreads) S.tokens[i] = 0u;
    if (threadIdx.x < kDecodeMaxT) S.amax[threadIdx.x] = 0u;
    for (int i = threadIdx.x; i < T * p.H / 64; i += kDecodeThreads)   // the tokens' lines, on their way while the logits are ranked
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.x + (int64_t)i * 64));
    __syncthreads();

    const float* logits = p.logits;
    if (p.wr) {   // the logits of experts c and c + G (then c + 2 G ..): all warps two experts
        logits = p.ws_logits;
        const int HC = p.H / 8;
        for (int e = cta; e < p.E; e += 2 * G) {
            const bool two = e + G < p.E;
            const uint4* w0 = reinterpret_cast<const uint4*>(p.wr + (int64_t)e * p.H);
            const uint4* w1 = reinterpret_cast<const uint4*>(p.wr + (int64_t)(two ? e + G : e) * p.H);
#pragma unroll 1
            for (int n = 0; 8 * n < T; ++n) {
                float acc[2][8] = {};
#pragma unroll 2
                for (int c = threadIdx.x; c < HC; c += kDecodeThreads) {
                    float wf[2][8];
                    const uint4 wv = __ldg(w0 + c), wu = __ldg(w1 + c);
                    uint4 xv[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        xv[j] = 8 * n + j < T ? __ldg(reinterpret_cast<const uint4*>(p.x) + (int64_t)(8 * n + j) * HC + c) : make_uint4(0u, 0u, 0u, 0u);
                    bf16x8_to_f32(wv, wf[0]);
                    bf16x8_to_f32(wu, wf[1]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (8 * n + j >= T) break;
                        float xf[8];
                        bf16x8_to_f32(xv[j], xf);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            acc[0][j] = fmaf(xf[i], wf[0][i], acc[0][j]);
                            acc[1][j] = fmaf(xf[i], wf[1][i], acc[1][j]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (8 * n + j >= T) break;
                    const float a = warp_sum(acc[0][j]), b = warp_sum(acc[1][j]);
                    if (lane == 0) {
                        S.red[(8 * n + j) * (kDecodeWarps + kDecodeStreams) + warp] = a;
                        S.red[(kDecodeMaxT + 8 * n + j) * (kDecodeWarps + kDecodeStreams) + warp] = b;
                    }
                }
            }
            __syncthreads();
            if (threadIdx.x < 2 * kDecodeMaxT) {
                const int j = threadIdx.x % kDecodeMaxT, second = threadIdx.x / kDecodeMaxT;
                if (j < T && (two || !second)) {
                    float s = 0.0f;
                    for (int w = 0; w < kDecodeWarps + kDecodeStreams; ++w) s += S.red[threadIdx.x * (kDecodeWarps + kDecodeStreams) + w];
                    p.ws_logits[(int64_t)j * p.E + e + second * G] = s;
                }
            }
            __syncthreads();
        }
        cg::this_grid().sync();
    }

    // S2: a warp a token; meanwhile max |x| of the tokens by the others (half a warp's 16 chunks are one token's)
    for (int tt = warp; tt < T; tt += kDecodeWarps + kDecodeStreams) {
        const float* l = logits + (int64_t)tt * p.E;
        int* ids = S.ids + tt * k;
        float* gates = S.gates + tt * k;
        if (p.E <= 256) rank_row<8>(l, p.E, k, ids, gates, lane);
        else rank_row<kMaxE / 32>(l, p.E, k, ids, gates, lane);
        __syncwarp();
        if (lane < k) atomicOr(&S.bitmap[ids[lane] >> 5], 1u << (ids[lane] & 31));
    }
    __syncthreads();
    if (threadIdx.x < P) {       // the pair's expert's place among the touched ones
        const int e = S.ids[threadIdx.x], tt = threadIdx.x / k;
        int rank = __popc(S.bitmap[e >> 5] & ((1u << (e & 31)) - 1u));
        for (int i = 0; i < (e >> 5); ++i) rank += __popc(S.bitmap[i]);
        S.expert[rank] = e;
        atomicOr(&S.tokens[rank], 1u << tt);
        S.ids[threadIdx.x] = rank;
    }
    if (threadIdx.x == kDecodeThreads - 1) {
        int n = 0;
        for (int i = 0; i < (p.E + 31) / 32; ++i) n += __popc(S.bitmap[i]);
        S.n_experts = n;
    }
    __syncthreads();
    if (threadIdx.x < P) {       // the expert's tokens and pairs
        const int tt = threadIdx.x / k, rank = S.ids[threadIdx.x], at = __popc(S.tokens[rank] & ((1u << tt) - 1u));
        S.list[rank][at] = static_cast<uint8_t>(tt);
        S.pair[rank][at] = static_cast<uint8_t>(threadIdx.x);
    }
    if (threadIdx.x < 4) {       // this CTA's even share of each phase's units
        const int ph = threadIdx.x;
        const int per = ph == 0 ? p.N / 8 : ph == 1 ? p.Ns / 8 : p.H / 16, n = per * (ph & 1 ? p.n_shared : S.n_experts);
        S.per_expert[ph] = per;
        const int first = share(n, cta, G), end = share(n, cta + 1, G);
        S.first[ph] = first;
        S.end[ph] = end;
        if (ph == 0) {           // the tokens of its experts
            uint32_t m = 0;
            for (int e = first / per; e * per < end; ++e) m |= S.tokens[e];
            int c = 0;
            for (; m; m &= m - 1) {
                S.need[c] = __ffs(m) - 1;
                S.need_at[__ffs(m) - 1] = static_cast<uint8_t>(c++);
            }
            S.n_need = c;
        }
    }
    __syncthreads();

    if (warp >= kDecodeWarps) {
        const int to = lane * kDecodeStreams + warp - kDecodeWarps;
        DecodeStream<kMx> P{p, S, to, smem0 + ring + to * p.slots * p.slot_bytes, smem0 + scales + to * p.slots * p.scale_bytes};
        if (to < kDecodeWarps) P.enter(0);
        else P.ph = 4;
        P.run(true);
        cg::this_grid().sync();
        if (S.most_rows > p.max_rows) cg::this_grid().sync();
        P.run(false);
        cg::this_grid().sync();
        if (__any_sync(0xffffffffu, !P.ok)) give_up();
        return;
    }
    DecodeWarp<kMx, kScaleSmem> W{p, S, warp, lane, lane >> 2, lane & 3, lane_row(lane >> 2), ring + warp * p.slots * p.slot_bytes,
                                       scales + warp * p.slots * p.scale_bytes, frags, sums};
    // The pairs whose h the CTAs read in the down phase (units go by expert): where every CTA's fit its shared memory,
    // each quantizes its own, and no second barrier is needed.
    for (int c = threadIdx.x; c < G; c += kMul) {
        const int per = p.H / 16, n = per * S.n_experts, first = share(n, c, G), end = share(n, c + 1, G);
        int rows = 0;
        for (int e = first / per; first < end && e * per < end; ++e) rows += __popc(S.tokens[e]);
        atomicMax(&S.most_rows, rows);
    }
    if (warp == kDecodeWarps - 1) {   // this CTA's
        const int per = S.per_expert[2], first = S.first[2], end = S.end[2];
        int rows = 0;
        for (int e = first / per; first < end && e * per < end; ++e) {
            const int m = __popc(S.tokens[e]);
            if (lane < m) {
                S.place[e - first / per][lane] = static_cast<uint8_t>(rows + lane);
                S.row_pair[rows + lane] = S.pair[e][lane];
            }
            rows += m;
        }
        if (lane == 0) {
            S.place_e = first / per;
            S.n_rows = rows;
        }
    }
    // S1 of the tokens that this CTA's gate/up experts have: their FP8 codes as B fragments (half a warp's 16 chunks
    // of eight columns are one token's).  Rolled loops: this code runs once, from a cold instruction cache.
    const int xc = p.H / 8, n_x = S.n_need * xc;
    const bool f8 = S.n_need > p.max_tokens;   // too many for f16
    const uint32_t row_x = f8 ? frag_row_bytes<true>(pieces_x) : frag_row_bytes<false>(pieces_x);
    auto chunk_of = [&](int c, int& tk) {
        const int o = c / xc;
        tk = c < n_x ? S.need[o] : -1;
        return c < n_x ? __ldg(reinterpret_cast<const uint4*>(p.x) + tk * xc + c - o * xc) : make_uint4(0u, 0u, 0u, 0u);
    };
#pragma unroll 2
    for (int b0 = warp * 32; b0 < n_x; b0 += kMul) {
        int tk;
        unsigned a = amax_bits8(chunk_of(b0 + lane, tk));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
        if (tk >= 0 && (lane & 15) == 0) atomicMax(&S.amax[tk], a);
    }
    multipliers_sync();
    if (threadIdx.x < T) S.sx[threadIdx.x] = __fdiv_rn(__uint_as_float(S.amax[threadIdx.x]), kFp8Max);
#pragma unroll 1
    for (int b0 = warp * 32; b0 < n_x; b0 += kMul) {
        int tk;
        float x[8];
        bf16x8_to_f32(chunk_of(b0 + lane, tk), x);
        const int o = (b0 + lane) / xc, c8 = b0 + lane - o * xc;
        const RowQuant s = RowQuant::of(tk >= 0 ? __uint_as_float(S.amax[tk]) : 0.0f);
        const uint2 codes = s.codes(x);
        int piece, i, tt;
        frag_place<kMx>(c8, piece, i, tt);
        if (tk >= 0) {
            if (f8)
                *reinterpret_cast<uint2*>(g_decode_smem + frags + o * row_x + piece * 256 + (i >> 1) * 64 + tt * 16 + (i & 1) * 8) =
                    frag_order<kMx>(codes);
            else
                *reinterpret_cast<uint4*>(g_decode_smem + frags + o * row_x + piece * 512 + i * 64 + tt * 16) =
                    frag_f16<kMx>(frag_order<kMx>(codes));
        }
        if constexpr (!kMx) {
            const float sum = halfwarp_sum(e4m3x8_sum(codes));
            if (tk >= 0 && (lane & 15) == 0)
                *reinterpret_cast<float*>(g_decode_smem + sums + (o * pieces_x * 2 + (c8 >> 4)) * 4) = sum * kNibbleOffset;
        }
    }
    multipliers_sync();

    if (f8) W.template routed<false, false, true>();
    else W.template routed<false, false, false>();
    if (p.n_shared) W.template shared<false>();

    cg::this_grid().sync();
    // S5: rows of h as B fragments: this CTA's own pairs into shared memory, or pair r by CTA r into the workspace
    const bool own_rows = S.most_rows <= p.max_rows;   // the same for every CTA
    const int n_rows = own_rows ? S.n_rows : P, hc = p.N / 8;
#pragma unroll 1
    for (int q = own_rows ? 0 : cta, odd = 0; q < n_rows; q += own_rows ? 1 : G, odd ^= 16) {   // (the maxima of two rows in turn)
        const int r = own_rows ? S.row_pair[q] : q;
        const float4* src = reinterpret_cast<const float4*>(p.h + (int64_t)r * p.N);
        float x[8];
        unsigned a = 0u;
        auto load = [&](int c) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f), w = v;
            if (c < hc) { v = __ldcg(src + 2 * c); w = __ldcg(src + 2 * c + 1); }
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
            x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
        };
#pragma unroll 1
        for (int b0 = 0; b0 < hc; b0 += kMul) {
            load(b0 + threadIdx.x);
#pragma unroll
            for (int z = 0; z < 8; ++z) a = max(a, magnitude_bits(x[z]));
        }
        a = __reduce_max_sync(0xffffffffu, a);
        if (lane == 0) S.row_max[warp + odd] = a;
        multipliers_sync();
        const RowQuant s = RowQuant::of(__uint_as_float(__reduce_max_sync(0xffffffffu, lane < kDecodeWarps ? S.row_max[lane + odd] : 0u)));
#pragma unroll 1
        for (int b0 = 0; b0 < hc; b0 += kMul) {
            const int c = b0 + threadIdx.x;
            if (hc > kMul) load(c);      // else it is there already
            const uint2 codes = s.codes(x);
            int piece, z, tt;
            frag_place<kMx>(c, piece, z, tt);
            const uint32_t at = piece * 512 + z * 64 + tt * 16;
            uint8_t* row = own_rows ? g_decode_smem + frags + q * row_h : p.hq + (int64_t)r * row_h;
            if (c < hc) *reinterpret_cast<uint4*>(row + at) = frag_f16<kMx>(frag_order<kMx>(codes));
            if constexpr (!kMx) {
                const float sum = halfwarp_sum(e4m3x8_sum(codes)) * kNibbleOffset;
                float* to = own_rows ? reinterpret_cast<float*>(g_decode_smem + sums) + q * pieces_h * 2 : p.hsum + (int64_t)r * pieces_h * 2;
                if (c < hc && (lane & 15) == 0) to[c >> 4] = sum;
            }
        }
        if (threadIdx.x == 0) (own_rows ? S.gs : p.gs)[r] = S.gates[r] * s.s;
    }
    if (own_rows) {
        multipliers_sync();
        W.template routed<true, false, false>();
    } else {
        cg::this_grid().sync();
        if (threadIdx.x < P) S.gs[threadIdx.x] = __ldcg(p.gs + threadIdx.x);
        multipliers_sync();
        W.template routed<true, true, false>();
    }
    if (p.n_shared) W.template shared<true>();

    cg::this_grid().sync();
    // S7: the gated rows in selection order, then the shared experts
    for (int i = cta * kMul + threadIdx.x; i < T * p.H / 4; i += G * kMul) {
        const int tt = i / (p.H / 4), m4 = i - tt * (p.H / 4);
        float4 v[kMaxK];
#pragma unroll
        for (int j = 0; j < kMaxK; ++j)
            if (j < k) v[j] = __ldcg(reinterpret_cast<const float4*>(p.y + (int64_t)(tt * k + j) * p.H) + m4);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kMaxK; ++j)
            if (j < k) { o.x += v[j].x; o.y += v[j].y; o.z += v[j].z; o.w += v[j].w; }
        for (int s = 0; s < p.n_shared; ++s) {
            const float4 w = __ldcg(reinterpret_cast<const float4*>(p.y + (int64_t)(P + s * T + tt) * p.H) + m4);
            o.x += w.x; o.y += w.y; o.z += w.z; o.w += w.w;
        }
        uint2 packed;
        packed.x = static_cast<uint32_t>(f32_to_bf16_bits(o.x)) | (static_cast<uint32_t>(f32_to_bf16_bits(o.y)) << 16);
        packed.y = static_cast<uint32_t>(f32_to_bf16_bits(o.z)) | (static_cast<uint32_t>(f32_to_bf16_bits(o.w)) << 16);
        reinterpret_cast<uint2*>(p.out + (int64_t)tt * p.H)[m4] = packed;
    }
    if (!W.ok) give_up();
}

// ---- host ---------------------------------------------------------------------------------------

struct DecodePlan {
    size_t logits, h, hq, hsum, gs, act, y, total;
};

inline DecodePlan plan_decode(const DecodeLayer& L, int64_t T, int k) {
    DecodePlan p{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align_up(off + (bytes ? bytes : 1), 256);
        return at;
    };
    const size_t P = (size_t)T * k;
    p.logits = take((size_t)T * L.E * 4);
    p.h = take(P * L.N * 4);
    p.hq = take(P * frag_row_bytes<false>((L.N + 255) / 256));
    p.hsum = take(P * (align_up(L.N, 256) / 128) * 4);
    p.gs = take(P * 4);
    p.act = take((size_t)T * L.n_shared * L.shared_N * 4);     // hi, then lo
    p.y = take((P + (size_t)T * L.n_shared) * L.H * 4);        // routed rows, then the shared experts'
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

inline DecodeRows decode_rows(int64_t row_bytes, int cp) {
    DecodeRows r{};
    r.pieces = static_cast<int>((row_bytes + 127) / 128);
    r.cp = std::min(cp, r.pieces);
    r.chunks = (r.pieces + r.cp - 1) / r.cp;
    return r;
}

// Weight rows as [piece][row][128 bytes]: a 3-D view where rows are whole pieces, else a 2-D one.
inline bool decode_map(CUtensorMap* m, const void* w, uint64_t row_bytes, uint64_t rows, uint32_t box_rows, int cp, bool* flat) {
    *flat = row_bytes % 128 != 0;
    if (*flat) return make_map_u8(m, w, row_bytes, rows, 128, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
    const cuuint64_t dims[3] = {128, rows, row_bytes / 128};
    const cuuint64_t strides[2] = {row_bytes, 128};
    const cuuint32_t box[3] = {128, box_rows, static_cast<cuuint32_t>(cp)};
    return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, w, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Dynamic shared memory that a CTA may take.  Every launch allows a kernel this much and no call its own size: the
// allowance is the function's, shared by the host threads, and a smaller layer's call would lower it under another's.
constexpr size_t kDecodeSmem = 227 * 1024 - sizeof(DecodeShared) - 64;

// How a CTA's 227 KB are divided: the fragments (as f16 for up to six tokens: a CTA's experts seldom have more; room
// for all as FP8), their group sums, and the warps' rings: chunks of four pieces (8 KB) where two fit, else of two or
// one.  The rows' scales get buffers beside the slots where they fit, else they are read in place.
struct DecodeSmem {
    int cp, slots, scale_bytes, frag_bytes, max_tokens, max_rows;
    size_t bytes;
};

inline bool plan_decode_smem(const DecodeLayer& L, int64_t T, bool mx, DecodeSmem* out) {
    const int pieces = (L.H + 255) / 256, pieces_h = (L.N + 255) / 256;
    const size_t room = kDecodeSmem - 1024;   // (the rings start on a 1024-byte boundary)
    const size_t row16 = frag_row_bytes<false>(pieces), row_h = frag_row_bytes<false>(pieces_h);
    const size_t scale = align_up((size_t)16 * std::max(L.H, L.N) / (mx ? 32 : 64), 128);
    for (int in_smem = 1; in_smem >= 0; --in_smem) {
        const size_t frag = std::max(std::max<size_t>(T * frag_row_bytes<true>(pieces), in_smem ? std::min<int64_t>(T, 6) * row16 : 0), 2 * row_h);
        const size_t sums = mx ? 0 : std::max<size_t>(T * pieces, frag / row_h * pieces_h) * 8;
        for (int cp = 4; cp >= 1; cp >>= 1)
            for (int slots = kDecodeMaxSlots; slots >= 2; --slots) {
                const size_t ring = (size_t)kDecodeWarps * slots * (cp * 2048 + (in_smem ? scale : 0));
                if (frag + sums + ring > room) continue;
                out->cp = cp;
                out->slots = slots;
                out->scale_bytes = in_smem ? static_cast<int>(scale) : 0;
                out->frag_bytes = static_cast<int>(frag);
                out->max_tokens = static_cast<int>(frag / row16);
                out->max_rows = static_cast<int>(frag / row_h);
                out->bytes = 1024 + frag + sums + ring;
                return true;
            }
    }
    return false;
}

template <bool kMx, bool kScaleSmem>
inline int launch_decode(DecodeParams& q, size_t smem, cudaStream_t stream) {
    const void* fn = reinterpret_cast<const void*>(k_decode<kMx, kScaleSmem>);
    if (set_smem(fn, kDecodeSmem)) return MOE_ERR_CUDA;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return MOE_ERR_CUDA;
    void* args[] = {&q};
    if (cudaLaunchCooperativeKernel(fn, dim3(sms), dim3(kDecodeThreads), args, smem, stream) != cudaSuccess) {
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
    DecodeSmem m;
    if (!plan_decode_smem(L, T, kMx, &m)) return MOE_ERR_UNSUPPORTED_SHAPE;
    q.slots = m.slots;
    q.slot_bytes = m.cp * 2048;
    q.scale_bytes = m.scale_bytes;
    q.frag_bytes = m.frag_bytes;
    q.max_tokens = m.max_tokens;
    q.max_rows = m.max_rows;
    q.rows[0] = decode_rows(L.H / 2, m.cp);
    q.rows[1] = decode_rows((int64_t)L.H * 2, m.cp);
    q.rows[2] = decode_rows(L.N / 2, m.cp);
    q.rows[3] = decode_rows((int64_t)(L.n_shared > 0 ? L.shared_N : 128) * 2, m.cp);
    for (int i = 0; i < (L.n_shared > 0 ? 6 : 3); ++i) {
        const bool sh = i >= 3, down = i % 3 == 2;
        const uint64_t cols = down ? (sh ? L.shared_N : L.N) : L.H, rows = down ? L.H : (sh ? L.shared_N : L.N);
        bool flat;
        if (!decode_map(&q.map[i], sh ? static_cast<const void*>(L.sw[i - 3]) : L.w[i], sh ? cols * 2 : cols / 2,
                        rows * (sh ? L.n_shared : L.E), down ? 16 : 8, q.rows[(down ? 2 : 0) + (sh ? 1 : 0)].cp, &flat))
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
    q.y = reinterpret_cast<float*>(b + p.y);
    q.E = L.E; q.H = L.H; q.N = L.N; q.k = k; q.T = static_cast<int>(T);
    q.n_shared = L.n_shared;
    q.Ns = L.n_shared > 0 ? L.shared_N : 0;
    return m.scale_bytes ? launch_decode<kMx, true>(q, m.bytes, stream) : launch_decode<kMx, false>(q, m.bytes, stream);
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
