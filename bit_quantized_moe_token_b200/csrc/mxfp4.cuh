// mxfp4.cuh — MXFP4 rows: quantization from bf16, f16 or fp32, and back to values.
//
// The OCP microscaling format (OCP Microscaling Formats v1.0, sections 5.2, 5.3 and 6.3): K in
// blocks of 32, one E8M0 scale 2^(b - 127) for each block (b = 255: NaN), E2M1 codes (0, .5, 1,
// 1.5, 2, 3, 4, 6 for codes 0..7 and the negatives for 8..15), two codes a byte with the first
// in the low nibble.
//   b    = clamp(floor(log2 max|x|) - 2 + 127, 0, 254)     (2: the exponent of 6 = 1.5 * 2^2)
//   code = E2M1 value nearest to x / 2^(b - 127), ties to the even code, at most +-6, sign kept
// A block that holds a NaN or an infinity gets scale 255 and codes 0: all of it reads back as NaN.
//
// The scale is a power of two, so x / 2^(b - 127) is one exact multiplication and the codes do
// not depend on rounding.  Both directions are bound by HBM: 2 (4) bytes read and 17/32 written a
// value, and the reverse.  Four threads share a block: each takes eight values with one or two
// 16-byte loads (consecutive threads read consecutive chunks) and the block's maximum goes
// through two shuffles.  A thread has four such chunks in flight.
//
// Measured: 16384 x 4096 bf16 quantized and read back in 57 us (340 MB: 91 % of HBM's measured 6.56
// TB/s; with one chunk a thread 80 us); 1000 x 4128 fp32 rows of a wider buffer in 6.8 us, 8 x 4096
// in 3.4: two launches, which is what a few rows cost (the same inputs over and over, so from L2).
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include "common.cuh"

namespace moe {

constexpr int kMxBlock = 32;

// 2^(b - 127) of an E8M0 byte (255: NaN; 0: 2^-127, an fp32 subnormal).
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
    return b == 255u ? __uint_as_float(0x7FC00000u) : b == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

// Two floats -> two E2M1 codes, round to nearest even with saturation to +-6 (the hardware
// cvt.rn.satfinite.e2m1x2.f32).  The low nibble holds `lo`.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest));
}

// One byte (two E2M1 codes) -> two floats, the low nibble first (exact).
__device__ __forceinline__ float2 e2m1x2_to_f32(uint32_t byte) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four E8M0 bytes -> four floats.
__device__ __forceinline__ void e8m0x4_to_f32(uint32_t b, float (&s)[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 h0, h1;\n\tmov.b32 {h0, h1}, %2;\n\tcvt.rn.bf16x2.ue8m0x2 %0, h0;\n\tcvt.rn.bf16x2.ue8m0x2 %1, h1;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(b));
    s[0] = __uint_as_float(lo << 16);
    s[1] = __uint_as_float(lo & 0xFFFF0000u);
    s[2] = __uint_as_float(hi << 16);
    s[3] = __uint_as_float(hi & 0xFFFF0000u);
}
// Eight E2M1 codes -> four f16x2 in order.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\tcvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// D = A B + C, m16n8k16 on f16 with fp32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    mma_f16(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}
// Eight values of type kType (moe_dtype) at chunk index c of a row.
template <int kType>
__device__ __forceinline__ void load8(const void* row, int64_t c, float (&f)[8]) {
    if constexpr (kType == MOE_F32) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(row) + 2 * c);
        const float4 b = __ldg(reinterpret_cast<const float4*>(row) + 2 * c + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(row) + c);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (kType == MOE_F16) {
                const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&u[q]));
                f[2 * q] = p.x;
                f[2 * q + 1] = p.y;
            } else {
                f[2 * q] = __uint_as_float(u[q] << 16);
                f[2 * q + 1] = __uint_as_float(u[q] & 0xFFFF0000u);
            }
        }
    }
}

// Chunks of eight values, numbered through the rows (K / 8 a row), kMxUnroll a thread (256 apart, their loads all in
// flight before the first is used).  kFlat: the rows follow one another, so a chunk's number is its address.
constexpr int kMxUnroll = 4;

template <int kType, bool kFlat>
__global__ void __launch_bounds__(256) k_mxfp4_quant(const uint8_t* __restrict__ x, int64_t chunks, int per_row,
                                                      int64_t row_bytes, uint32_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales) {
    const int64_t c0 = blockIdx.x * (int64_t)(256 * kMxUnroll) + threadIdx.x;
    float f[kMxUnroll][8];
#pragma unroll
    for (int u = 0; u < kMxUnroll; ++u) {
        const int64_t c = c0 + 256 * u;
#pragma unroll
        for (int q = 0; q < 8; ++q) f[u][q] = 0.0f;
        if (c < chunks) {   // the four lanes of a block are live together
            if constexpr (kFlat) {
                load8<kType>(x, c, f[u]);
            } else {
                const int64_t r = c / per_row;
                load8<kType>(x + r * row_bytes, c - r * per_row, f[u]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kMxUnroll; ++u) {
        const int64_t c = c0 + 256 * u;
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(f[u][q]) & 0x7FFFFFFFu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t field = m >> 23;   // of the block's maximum: floor(log2) + 127; 255: not finite
        const uint32_t b = field == 255u ? 255u : field > 2u ? field - 2u : 0u;
        uint32_t w = 0;
        if (b != 255u) {
            const float inv = __uint_as_float((254u - b) << 23);
#pragma unroll
            for (int q = 0; q < 4; ++q) w |= f32x2_to_e2m1x2(f[u][2 * q] * inv, f[u][2 * q + 1] * inv) << (8 * q);
        }
        if (c < chunks) {
            codes[c] = w;
            if ((c & 3) == 0) scales[c >> 2] = static_cast<uint8_t>(b);
        }
    }
}

template <int kType>
__global__ void __launch_bounds__(256) k_mxfp4_dequant(const uint32_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales, int64_t chunks,
                                                        void* __restrict__ y) {
    const int64_t c0 = blockIdx.x * (int64_t)(256 * kMxUnroll) + threadIdx.x;
    uint32_t w[kMxUnroll], b[kMxUnroll];
#pragma unroll
    for (int u = 0; u < kMxUnroll; ++u) {
        const int64_t c = c0 + 256 * u;
        w[u] = c < chunks ? __ldg(codes + c) : 0u;
        b[u] = c < chunks ? __ldg(scales + (c >> 2)) : 0u;
    }
#pragma unroll
    for (int u = 0; u < kMxUnroll; ++u) {
        const int64_t c = c0 + 256 * u;
        if (c >= chunks) break;
        const float s = e8m0_to_f32(b[u]);
        float f[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 p = e2m1x2_to_f32((w[u] >> (8 * q)) & 0xFFu);
            f[2 * q] = p.x * s;
            f[2 * q + 1] = p.y * s;
        }
        if constexpr (kType == MOE_F32) {
            reinterpret_cast<float4*>(y)[2 * c] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4*>(y)[2 * c + 1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            uint32_t o[4];   // exact: two significant bits, and bf16 has fp32's exponents
#pragma unroll
            for (int q = 0; q < 4; ++q)
                o[q] = static_cast<uint32_t>(f32_to_bf16_bits(f[2 * q])) |
                       (static_cast<uint32_t>(f32_to_bf16_bits(f[2 * q + 1])) << 16);
            reinterpret_cast<uint4*>(y)[c] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

inline int mxfp4_rows_ok(int64_t rows, int64_t K) {
    if (rows < 0 || K <= 0) return MOE_ERR_INVALID_ARG;
    if (K % kMxBlock != 0 || K > (int64_t)1 << 30 || rows > ((int64_t)1 << 38) / K) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

}  // namespace moe

extern "C" int mxfp4_quant_rows(const void* x, int x_type, int64_t rows, int64_t K, int64_t row_stride,
                                uint8_t* codes, uint8_t* scales, moe_stream_t stream) {
    using namespace moe;
    int st = mxfp4_rows_ok(rows, K);
    if (st != MOE_OK) return st;
    if (x_type != MOE_BF16 && x_type != MOE_F16 && x_type != MOE_F32) return MOE_ERR_INVALID_ARG;
    if (rows > 1 && row_stride < K) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return MOE_ERR_INVALID_ARG;
    const int64_t row_bytes = (rows > 1 ? row_stride : K) * (x_type == MOE_F32 ? 4 : 2);
    if (!aligned(x, 16) || row_bytes % 16 != 0 || !aligned(codes, 4)) return MOE_ERR_MISALIGNED;
    const int64_t chunks = rows * (K / 8);
    const unsigned grid = static_cast<unsigned>((chunks + 256 * kMxUnroll - 1) / (256 * kMxUnroll));
    const uint8_t* xb = static_cast<const uint8_t*>(x);
    uint32_t* cw = reinterpret_cast<uint32_t*>(codes);
    const int per_row = static_cast<int>(K / 8);
    const bool flat = row_bytes == K * (x_type == MOE_F32 ? 4 : 2);
#define MOE_MQ(TYPE) (flat ? k_mxfp4_quant<TYPE, true><<<grid, 256, 0, stream>>>(xb, chunks, per_row, row_bytes, cw, scales) \
                           : k_mxfp4_quant<TYPE, false><<<grid, 256, 0, stream>>>(xb, chunks, per_row, row_bytes, cw, scales))
    if (x_type == MOE_BF16) MOE_MQ(MOE_BF16);
    else if (x_type == MOE_F16) MOE_MQ(MOE_F16);
    else MOE_MQ(MOE_F32);
#undef MOE_MQ
    return launch_status();
}

extern "C" int mxfp4_dequant_rows(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* y,
                                  int y_type, moe_stream_t stream) {
    using namespace moe;
    int st = mxfp4_rows_ok(rows, K);
    if (st != MOE_OK) return st;
    if (y_type != MOE_BF16 && y_type != MOE_F32) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!codes || !scales || !y) return MOE_ERR_INVALID_ARG;
    if (!aligned(codes, 4) || !aligned(y, 16)) return MOE_ERR_MISALIGNED;
    const int64_t chunks = rows * (K / 8);
    const unsigned grid = static_cast<unsigned>((chunks + 256 * kMxUnroll - 1) / (256 * kMxUnroll));
    const uint32_t* cw = reinterpret_cast<const uint32_t*>(codes);
    if (y_type == MOE_BF16)
        k_mxfp4_dequant<MOE_BF16><<<grid, 256, 0, stream>>>(cw, scales, chunks, y);
    else
        k_mxfp4_dequant<MOE_F32><<<grid, 256, 0, stream>>>(cw, scales, chunks, y);
    return launch_status();
}
