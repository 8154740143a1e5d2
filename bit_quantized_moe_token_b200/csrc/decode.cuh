// decode.cuh — the whole routed MoE layer for a few tokens (T <= 16), on W4A8 or MXFP4 experts.
//
// The arithmetic of moe_w4a8_forward: S1 (FP8 of the tokens), S2 (top-k, gates), S4 (gate, up,
// SwiGLU), S5 (FP8 of h for each routed pair), S6 (down), S7 (the gated sum) and S8 (shared
// experts), with the experts' weights in pack-quantized INT4 or in MXFP4.
#pragma once
#include "forward.cuh"
#include "mxfp4.cuh"

namespace moe {

constexpr int kDecodeMaxT = 16;

struct DecodeLayer {
    int E, H, N;
    const uint8_t *w[3];          // gate, up [E, N, H/2], down [E, H, N/2]
    const void *s[3];             // INT4: bf16 [.., K/128]; MXFP4: E8M0 [.., K/32]
    int n_shared, shared_N;
    const uint16_t *sw[3];        // shared experts' gate, up, down (bf16)
};

// Eight values of word `c` of a weight row (codes 8 c .. 8 c + 7).
template <bool kMx>
__device__ __forceinline__ void weight8(const uint8_t* row, const void* srow, int c, float (&f)[8]) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(row) + c);
    if constexpr (kMx) {
        const float s = e8m0_to_f32(__ldg(static_cast<const uint8_t*>(srow) + (c >> 2)));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 p = e2m1x2_to_f32((w >> (8 * q)) & 0xFFu);
            f[2 * q] = p.x * s;
            f[2 * q + 1] = p.y * s;
        }
    } else {
        const float s = bf16_bits_to_f32(__ldg(static_cast<const uint16_t*>(srow) + (c >> 4)));
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = static_cast<float>((int)((w >> (4 * q)) & 15u) - 8) * s;
    }
}

// A warp's dot product of weight row `row` (K values) with a row of E4M3 codes.
template <bool kMx>
__device__ __forceinline__ float dot_codes(const uint8_t* row, const void* srow, const uint8_t* codes, int K) {
    float acc = 0.0f;
    for (int c = threadIdx.x & 31; c < K / 8; c += 32) {
        float f[8];
        weight8<kMx>(row, srow, c, f);
        const uint2 q = reinterpret_cast<const uint2*>(codes)[c];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = fmaf(f[i], e4m3_to_f32(((i < 4 ? q.x : q.y) >> (8 * (i & 3))) & 0xFF), acc);
    }
    return warp_sum(acc);
}

__device__ __forceinline__ float dot_bf16(const uint16_t* row, const uint16_t* x, const float* a, int K) {
    float acc = 0.0f;
    for (int c = threadIdx.x & 31; c < K; c += 32)
        acc = fmaf(bf16_bits_to_f32(__ldg(row + c)), x ? bf16_bits_to_f32(x[c]) : a[c], acc);
    return warp_sum(acc);
}

template <bool kMx>
__device__ __forceinline__ const void* scale_row(const void* s, int64_t row, int K) {
    return kMx ? static_cast<const void*>(static_cast<const uint8_t*>(s) + row * (K / 32))
               : static_cast<const void*>(static_cast<const uint16_t*>(s) + row * (K / 128));
}

// One warp for each (pair, n), then for each (token, shared expert, n).
template <bool kMx>
__global__ void __launch_bounds__(256) k_decode_gateup(DecodeLayer L, const uint16_t* x, int T, int k, const int32_t* ids,
                                                        const uint8_t* xq, const float* sx, float* h, float* act) {
    const int64_t w = blockIdx.x * 8ll + (threadIdx.x >> 5);
    const int64_t routed = (int64_t)T * k * L.N, sh = (int64_t)T * L.n_shared * L.shared_N;
    if (w < routed) {
        const int64_t p = w / L.N, r = (int64_t)ids[p] * L.N + w % L.N;
        const int t = (int)(p / k);
        const float g = dot_codes<kMx>(L.w[0] + r * (L.H / 2), scale_row<kMx>(L.s[0], r, L.H), xq + (int64_t)t * L.H, L.H) * sx[t];
        const float u = dot_codes<kMx>(L.w[1] + r * (L.H / 2), scale_row<kMx>(L.s[1], r, L.H), xq + (int64_t)t * L.H, L.H) * sx[t];
        if ((threadIdx.x & 31) == 0) h[w] = silu(g) * u;
    } else if (w < routed + sh) {
        const int64_t i = w - routed, t = i / (L.n_shared * L.shared_N), r = i % (L.n_shared * L.shared_N);
        const float g = dot_bf16(L.sw[0] + r * L.H, x + t * L.H, nullptr, L.H);
        const float u = dot_bf16(L.sw[1] + r * L.H, x + t * L.H, nullptr, L.H);
        if ((threadIdx.x & 31) == 0) act[i] = silu(g) * u;
    }
}

// S5: one CTA for each pair.
__global__ void __launch_bounds__(256) k_decode_requant(const float* h, int N, uint8_t* hq, float* sh) {
    __shared__ float red[32];
    const float* row = h + (int64_t)blockIdx.x * N;
    float a = 0.0f;
    for (int i = threadIdx.x; i < N; i += blockDim.x) a = fmaxf(a, fabsf(row[i]));
    const float s = __fdiv_rn(block_max(a, red), kFp8Max);
    for (int i = threadIdx.x; i < N; i += blockDim.x)
        hq[(int64_t)blockIdx.x * N + i] = s != 0.0f ? (uint8_t)f32x2_to_e4m3x2(__fdiv_rn(row[i], s), 0.0f) : 0;
    if (threadIdx.x == 0) sh[blockIdx.x] = s;
}

// One warp for each (token, m).
template <bool kMx>
__global__ void __launch_bounds__(256) k_decode_down(DecodeLayer L, int T, int k, const int32_t* ids, const float* gates,
                                                      const uint8_t* hq, const float* sh, const float* act, uint16_t* out) {
    const int64_t w = blockIdx.x * 8ll + (threadIdx.x >> 5);
    if (w >= (int64_t)T * L.H) return;
    const int64_t t = w / L.H, m = w % L.H;
    float acc = 0.0f;
    for (int j = 0; j < k; ++j) {
        const int64_t p = t * k + j, r = (int64_t)ids[p] * L.H + m;
        acc += gates[p] * (dot_codes<kMx>(L.w[2] + r * (L.N / 2), scale_row<kMx>(L.s[2], r, L.N), hq + p * L.N, L.N) * sh[p]);
    }
    for (int s = 0; s < L.n_shared; ++s)
        acc += dot_bf16(L.sw[2] + (s * (int64_t)L.H + m) * L.shared_N, nullptr, act + (t * L.n_shared + s) * L.shared_N, L.shared_N);
    if ((threadIdx.x & 31) == 0) out[w] = f32_to_bf16_bits(acc);
}

struct DecodePlan {
    size_t ids, gates, logits, cnt, xq, sx, h, hq, sh, act, total;
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
    p.ids = take(P * 4);
    p.gates = take(P * 4);
    p.logits = take((size_t)T * L.E * 4);
    p.cnt = take((size_t)router_counter_words(T) * 4);
    p.xq = take((size_t)T * L.H);
    p.sx = take((size_t)T * 4);
    p.h = take(P * L.N * 4);
    p.hq = take(P * L.N);
    p.sh = take(P * 4);
    p.act = take((size_t)T * L.n_shared * L.shared_N * 4);
    p.total = off;
    return p;
}

inline int decode_args_ok(const DecodeLayer& L, int64_t T, int k) {
    if (T < 0 || L.E < 1 || L.H <= 0 || L.N <= 0 || k < 1 || L.n_shared < 0) return MOE_ERR_INVALID_ARG;
    if (T > kDecodeMaxT || L.H % 128 || L.N % 128 || L.H > 16384 || L.N > 8192) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (L.H * ((T + 7) / 8) > 16384) return MOE_ERR_UNSUPPORTED_SHAPE;
    const int st = route_args_ok(T, L.E, k);
    if (st != MOE_OK) return st;
    if (L.n_shared > 0 && (L.shared_N <= 0 || L.shared_N % 128 || L.shared_N > 8192)) return MOE_ERR_UNSUPPORTED_SHAPE;
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
    int32_t* ids = reinterpret_cast<int32_t*>(b + p.ids);
    float* gates = reinterpret_cast<float*>(b + p.gates);
    float* sx = reinterpret_cast<float*>(b + p.sx);
    float* h = reinterpret_cast<float*>(b + p.h);
    float* sh = reinterpret_cast<float*>(b + p.sh);
    float* act = reinterpret_cast<float*>(b + p.act);
    if (router) {
        float* lg = reinterpret_cast<float*>(b + p.logits);
        unsigned* cnt = reinterpret_cast<unsigned*>(b + p.cnt);
        int launches;
        if (cudaMemsetAsync(cnt, 0, router_counter_words(T) * 4, stream) != cudaSuccess) return MOE_ERR_CUDA;
        if ((st = launch_router_topk(x, router, T, L.H, L.E, k, lg, ids, gates, cnt, b + p.xq, sx, nullptr, stream, &launches)))
            return st;
    } else if ((st = launch_quant_topk(logits, x, T, L.E, k, L.H, ids, gates, b + p.xq, sx, nullptr, stream))) {
        return st;
    }
    const int64_t units = T * k * (int64_t)L.N + T * (int64_t)L.n_shared * L.shared_N;
    k_decode_gateup<kMx><<<(unsigned)((units + 7) / 8), 256, 0, stream>>>(L, x, (int)T, k, ids, b + p.xq, sx, h, act);
    k_decode_requant<<<(unsigned)(T * k), 256, 0, stream>>>(h, L.N, b + p.hq, sh);
    k_decode_down<kMx><<<(unsigned)((T * L.H + 7) / 8), 256, 0, stream>>>(L, (int)T, k, ids, gates, b + p.hq, sh, act, out);
    return launch_status();
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
