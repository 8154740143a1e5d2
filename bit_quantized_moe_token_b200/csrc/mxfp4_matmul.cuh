// mxfp4_matmul.cuh — out = A B^T with both operands in MXFP4 rows (mxfp4.cuh):
//   out[m, n] = sum_b 2^(sa[m,b] + sb[n,b] - 254) sum_{k in block b} A[m,k] B[n,k]
#pragma once
#include "mxfp4.cuh"

namespace moe {

// 64 x 64 outputs a CTA, K in blocks of 32: both tiles are widened to fp32 in shared memory and
// each thread sums a 4 x 4 patch.
template <int kType>
__global__ void __launch_bounds__(256) k_mxfp4_matmul(const uint8_t* __restrict__ a, const uint8_t* __restrict__ as,
                                                       const uint8_t* __restrict__ b, const uint8_t* __restrict__ bs,
                                                       int64_t M, int64_t N, int K, void* __restrict__ out) {
    __shared__ float ta[kMxBlock][65], tb[kMxBlock][65];
    const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
    const int row = threadIdx.x >> 2, part = threadIdx.x & 3;   // a row's block: 4 threads x 4 bytes
    const int tm = threadIdx.x >> 4, tn = threadIdx.x & 15;
    float acc[4][4] = {};
    for (int blk = 0; blk < K / kMxBlock; ++blk) {
        __syncthreads();
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const int64_t r = (side ? n0 : m0) + row;
            uint32_t w = 0;
            float s = 0.0f;
            if (r < (side ? N : M)) {
                w = __ldg(reinterpret_cast<const uint32_t*>((side ? b : a) + r * (K / 2) + blk * 16) + part);
                s = e8m0_to_f32(__ldg((side ? bs : as) + r * (K / kMxBlock) + blk));
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 p = e2m1x2_to_f32((w >> (8 * q)) & 0xFFu);
                (side ? tb : ta)[part * 8 + 2 * q][row] = p.x * s;
                (side ? tb : ta)[part * 8 + 2 * q + 1][row] = p.y * s;
            }
        }
        __syncthreads();
#pragma unroll 4
        for (int k = 0; k < kMxBlock; ++k) {
            float x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) { x[i] = ta[k][tm + 16 * i]; y[i] = tb[k][tn + 16 * i]; }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + tm + 16 * i, n = n0 + tn + 16 * j;
            if (m >= M || n >= N) continue;
            if constexpr (kType == MOE_F32) static_cast<float*>(out)[m * N + n] = acc[i][j];
            else static_cast<uint16_t*>(out)[m * N + n] = f32_to_bf16_bits(acc[i][j]);
        }
}

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
    const dim3 grid(static_cast<unsigned>((N + 63) / 64), static_cast<unsigned>((M + 63) / 64));
    if (grid.y > 65535) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (out_type == MOE_F32)
        k_mxfp4_matmul<MOE_F32><<<grid, 256, 0, stream>>>(a, a_scales, b, b_scales, M, N, (int)K, out);
    else
        k_mxfp4_matmul<MOE_BF16><<<grid, 256, 0, stream>>>(a, a_scales, b, b_scales, M, N, (int)K, out);
    return launch_status();
}
