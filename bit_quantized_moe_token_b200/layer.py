"""Convenience wrappers: torch allocation around the C entry points."""
from __future__ import annotations

import math

from ._binding import (Layer, Layer4, Layer8, LayerH, LayerMX, moe_hybrid_forward, moe_hybrid_workspace_bytes,
                       moe_mxfp4_decode, moe_mxfp4_decode_router, moe_mxfp4_decode_workspace_bytes,
                       moe_nvfp4_forward, moe_nvfp4_workspace_bytes,
                       moe_w4a8_decode, moe_w4a8_decode_router, moe_w4a8_decode_workspace_bytes,
                       moe_w4a8_forward, moe_w4a8_workspace_bytes, moe_w8a8_forward,
                       moe_w8a8_workspace_bytes, mxfp4_dequant_rows, mxfp4_matmul, mxfp4_quant_rows,
                       nvfp4_quant_weights, w4a8_pack_weights,
                       w8a8_quant_weights)


def pack_expert_weights(w, group: int = 128, stream=None):
    """bf16 weights [..., rows, K] on the GPU -> (int32 packed [..., rows, K/8],
    bf16 scales [..., rows, K/group]) in pack-quantized storage."""
    import torch
    *lead, rows, K = w.shape
    packed = torch.empty(*lead, rows, K // 8, dtype=torch.int32, device=w.device)
    scales = torch.empty(*lead, rows, K // group, dtype=torch.bfloat16, device=w.device)
    w4a8_pack_weights(w.contiguous(), packed, scales, group=group, stream=stream)
    return packed, scales


def make_layer(gate_w, up_w, down_w, sh_gate=None, sh_up=None, sh_down=None,
               stream=None) -> Layer:
    """Quantize and pack bf16 expert weights gate/up [E, N, H], down [E, H, N]."""
    E, N, H = gate_w.shape
    gp, gs = pack_expert_weights(gate_w, stream=stream)
    up, us = pack_expert_weights(up_w, stream=stream)
    dp, ds = pack_expert_weights(down_w, stream=stream)
    return Layer(E, H, N, gp, up, dp, gs, us, ds, sh_gate=sh_gate, sh_up=sh_up, sh_down=sh_down)


def quant_expert_weights_w8a8(w, stream=None):
    """bf16 weights [..., rows, K] on the GPU -> (E4M3 codes uint8 [..., rows, K],
    fp32 row scales [..., rows])."""
    import torch
    *lead, rows, K = w.shape
    q = torch.empty(*lead, rows, K, dtype=torch.uint8, device=w.device)
    s = torch.empty(*lead, rows, dtype=torch.float32, device=w.device)
    w8a8_quant_weights(w.contiguous(), q, s, stream=stream)
    return q, s


def make_layer_w8a8(gate_w, up_w, down_w, sh_gate=None, sh_up=None, sh_down=None,
                    stream=None) -> Layer8:
    """Row-quantize bf16 expert weights gate/up [E, N, H], down [E, H, N] to FP8."""
    E, N, H = gate_w.shape
    gq, gs = quant_expert_weights_w8a8(gate_w, stream=stream)
    uq, us = quant_expert_weights_w8a8(up_w, stream=stream)
    dq, ds = quant_expert_weights_w8a8(down_w, stream=stream)
    return Layer8(E, H, N, gq, uq, dq, gs, us, ds, sh_gate=sh_gate, sh_up=sh_up, sh_down=sh_down)


def quant_expert_weights_nvfp4(w, stream=None):
    """bf16 weights [experts, rows, K] on the GPU -> (E2M1 codes uint8 [experts, rows, K/2],
    E4M3 block scales uint8 [experts, rows, K/16], fp32 scale2 [experts])."""
    import torch
    E, rows, K = w.shape
    codes = torch.empty(E, rows, K // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(E, rows, K // 16, dtype=torch.uint8, device=w.device)
    s2 = torch.empty(E, dtype=torch.float32, device=w.device)
    nvfp4_quant_weights(w.contiguous(), codes, scales, s2, stream=stream)
    return codes, scales, s2


def make_layer_nvfp4(gate_w, up_w, down_w, sh_gate=None, sh_up=None, sh_down=None,
                     stream=None) -> Layer4:
    """NVFP4-quantize bf16 expert weights gate/up [E, N, H], down [E, H, N]."""
    E, N, H = gate_w.shape
    g = quant_expert_weights_nvfp4(gate_w, stream=stream)
    u = quant_expert_weights_nvfp4(up_w, stream=stream)
    d = quant_expert_weights_nvfp4(down_w, stream=stream)
    return Layer4(E, H, N, g[0], u[0], d[0], g[1], u[1], d[1], g[2], u[2], d[2],
                  sh_gate=sh_gate, sh_up=sh_up, sh_down=sh_down)


def hybrid_from(w4: Layer, f4: Layer4, hot_ids) -> LayerH:
    """A hybrid layer from a W4A8 layer and an NVFP4 layer of the same experts: the hot experts
    (hot_ids, in slab order) take their NVFP4 slabs, the others their W4A8 slabs."""
    import torch
    dev = w4.gate_packed.device
    hot = torch.as_tensor(hot_ids, dtype=torch.int32).to(dev)
    mask = torch.ones(w4.E, dtype=torch.bool, device=dev)
    mask[hot.long()] = False
    cold = torch.arange(w4.E, dtype=torch.int32, device=dev)[mask]
    hi, ci = hot.long(), cold.long()
    h = Layer4(len(hot_ids), f4.H, f4.N, f4.gate_f4[hi].contiguous(), f4.up_f4[hi].contiguous(),
               f4.down_f4[hi].contiguous(), f4.gate_bs[hi].contiguous(), f4.up_bs[hi].contiguous(),
               f4.down_bs[hi].contiguous(), f4.gate_s2[hi].contiguous(), f4.up_s2[hi].contiguous(),
               f4.down_s2[hi].contiguous())
    c = Layer(int(cold.numel()), w4.H, w4.N, w4.gate_packed[ci].contiguous(), w4.up_packed[ci].contiguous(),
              w4.down_packed[ci].contiguous(), w4.gate_scales[ci].contiguous(), w4.up_scales[ci].contiguous(),
              w4.down_scales[ci].contiguous(), group=w4.group, sh_gate=w4.sh_gate, sh_up=w4.sh_up,
              sh_down=w4.sh_down)
    return LayerH(w4.E, h, c, hot.contiguous(), cold.contiguous())


def _not_mxfp4(layer):
    if isinstance(layer, LayerMX):
        raise ValueError("forward: expected a layer of type Layer or Layer8 or Layer4 or LayerH, got LayerMX, which is decode's")


def _few_token(layer, call: str):
    if not isinstance(layer, (Layer, LayerMX)):
        raise ValueError(f"{call}: expected a layer of type Layer or LayerMX, got {type(layer).__name__}")


def alloc_workspace(layer, T: int, k: int, device=None):
    import torch
    _not_mxfp4(layer)
    if isinstance(layer, LayerH):
        n, ref = moe_hybrid_workspace_bytes(layer, T, k), layer.hot_ids
    elif isinstance(layer, Layer8):
        n, ref = moe_w8a8_workspace_bytes(layer, T, k), layer.gate_w8
    elif isinstance(layer, Layer4):
        n, ref = moe_nvfp4_workspace_bytes(layer, T, k), layer.gate_f4
    else:
        n, ref = moe_w4a8_workspace_bytes(layer, T, k), layer.gate_packed
    if n == 0 and T > 0:
        raise ValueError("unsupported layer shape for the MoE forward")
    dev = device if device is not None else ref.device
    return torch.empty(max(n, 256), dtype=torch.uint8, device=dev)


def forward(layer, x, logits, k: int, out=None, ws=None, stream=None):
    """The layer on x for any expert format but MXFP4 (Layer: W4A8, Layer8: row-scaled FP8, Layer4: NVFP4, LayerH:
    hybrid).  LayerMX, for up to 16 tokens, is decode()'s."""
    import torch
    _not_mxfp4(layer)
    if out is None:
        out = torch.empty_like(x)
    if ws is None:
        ws = alloc_workspace(layer, x.shape[0], k, x.device)
    if isinstance(layer, LayerH):
        moe_hybrid_forward(layer, x, logits, k, out, ws, stream=stream)
    elif isinstance(layer, Layer8):
        moe_w8a8_forward(layer, x, logits, k, out, ws, stream=stream)
    elif isinstance(layer, Layer4):
        moe_nvfp4_forward(layer, x, logits, k, out, ws, stream=stream)
    else:
        moe_w4a8_forward(layer, x, logits, k, out, ws, stream=stream)
    return out


def _on(stream):
    """The context of a stream (torch stream or handle): what a wrapper allocates or copies then belongs to the stream
    that its kernels run on, and scratch freed on return is not handed out while they still use it."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def quant_mxfp4(x, stream=None):
    """bf16, f16 or fp32 values [..., K] on the GPU -> (E2M1 codes uint8 [..., K/2], E8M0 scales
    uint8 [..., K/32]).  Two-dimensional x may have strided rows."""
    if stream is not None:
        with _on(stream):
            return quant_mxfp4(x)
    import torch
    if x.dim() != 2:
        *lead, K = x.shape
        codes, scales = quant_mxfp4(x.reshape(math.prod(lead), K))
        return codes.view(*lead, K // 2), scales.view(*lead, K // 32)
    rows, K = x.shape
    if K % 32:
        raise ValueError("K must be a multiple of 32")
    codes = x.new_empty((rows, K // 2), dtype=torch.uint8)
    scales = x.new_empty((rows, K // 32), dtype=torch.uint8)
    mxfp4_quant_rows(x, codes, scales)
    return codes, scales


def dequant_mxfp4(codes, scales, dtype=None, stream=None):
    """The values [..., K] of MXFP4 codes [..., K/2] and scales [..., K/32], bf16 (the default) or
    fp32, both exact."""
    if stream is not None:
        with _on(stream):
            return dequant_mxfp4(codes, scales, dtype)
    import torch
    if codes.dim() != 2:
        *lead, half = codes.shape
        if tuple(scales.shape) != (*lead, half // 16):
            raise ValueError(f"scales: expected {[*lead, half // 16]}, got {list(scales.shape)}")
        y = dequant_mxfp4(codes.reshape(math.prod(lead), half), scales.reshape(math.prod(lead), half // 16), dtype)
        return y.view(*lead, 2 * half)
    y = codes.new_empty((codes.shape[0], 2 * codes.shape[1]), dtype=dtype or torch.bfloat16)
    mxfp4_dequant_rows(codes, scales, y)
    return y


def matmul_mxfp4(a, a_scales, b, b_scales, dtype=None, out=None, stream=None):
    """A B^T [M, N] of MXFP4 rows A [M, K] and B [N, K], as bf16 (the default) or fp32; into `out`, of its type, if given."""
    if out is not None and dtype is not None and out.dtype != dtype:
        raise ValueError(f"dtype {dtype}, but out is {out.dtype}")
    if stream is not None:
        with _on(stream):
            return matmul_mxfp4(a, a_scales, b, b_scales, dtype, out)
    import torch
    if out is None:
        out = torch.empty(a.shape[0], b.shape[0], dtype=dtype or torch.bfloat16, device=a.device)
    mxfp4_matmul(a, a_scales, b, b_scales, out)
    return out


def make_layer_mxfp4(gate_w, up_w, down_w, sh_gate=None, sh_up=None, sh_down=None,
                     stream=None) -> LayerMX:
    """MXFP4-quantize bf16 expert weights gate/up [E, N, H], down [E, H, N]."""
    E, N, H = gate_w.shape
    g, u, d = (quant_mxfp4(w, stream=stream) for w in (gate_w, up_w, down_w))
    return LayerMX(E, H, N, g[0], u[0], d[0], g[1], u[1], d[1], sh_gate=sh_gate, sh_up=sh_up, sh_down=sh_down)


def alloc_decode_workspace(layer, T: int, k: int, device=None):
    """Scratch for decode / decode_router on a W4A8 or MXFP4 layer."""
    import torch
    _few_token(layer, "decode")
    if isinstance(layer, LayerMX):
        n, ref = moe_mxfp4_decode_workspace_bytes(layer, T, k), layer.gate_f4
    else:
        n, ref = moe_w4a8_decode_workspace_bytes(layer, T, k), layer.gate_packed
    if n == 0 and T > 0:
        raise ValueError("unsupported layer shape or token count for the few-token layer")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device if device is not None else ref.device)


def decode(layer, x, logits, k: int, out=None, ws=None, stream=None):
    """The whole layer on up to 16 tokens (Layer: W4A8, LayerMX: MXFP4) from router logits [T, E]."""
    if stream is not None:
        with _on(stream):
            return decode(layer, x, logits, k, out, ws)
    import torch
    _few_token(layer, "decode")
    if out is None:
        out = torch.empty_like(x)
    if ws is None:
        ws = alloc_decode_workspace(layer, x.shape[0], k, x.device)
    (moe_mxfp4_decode if isinstance(layer, LayerMX) else moe_w4a8_decode)(layer, x, logits, k, out, ws)
    return out


def decode_router(layer, x, wr, k: int, out=None, ws=None, stream=None):
    """decode() with the logits computed from the router weight wr [E, H]."""
    if stream is not None:
        with _on(stream):
            return decode_router(layer, x, wr, k, out, ws)
    import torch
    _few_token(layer, "decode_router")
    if out is None:
        out = torch.empty_like(x)
    if ws is None:
        ws = alloc_decode_workspace(layer, x.shape[0], k, x.device)
    fn = moe_mxfp4_decode_router if isinstance(layer, LayerMX) else moe_w4a8_decode_router
    fn(layer, x, wr, k, out, ws)
    return out
