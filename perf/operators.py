"""The cases on which the MXFP4 operators and the few-token MoE layers are measured.

Operators:
  quant    rows of bf16, f16 or fp32 -> MXFP4 (E2M1 codes, one power-of-two scale for 32 columns) and back to values
  matmul   out = A B^T with both operands in MXFP4
  w4a8     the whole routed MoE layer for a few tokens, INT4 experts (groups of 128, bf16 scales), FP8 activations
  mxfp4    the same layer with MXFP4 experts

`own` false: the plain forms in elementary torch operations.  `own` true: the package's calls.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------------------------

def listed():
    moe = {"E": 256, "H": 4096, "N": 2048, "k": 6, "router": False, "shared": 0}
    return [
        # one decode step's activations: latency
        {"name": "quant_tokens_t8", "op": "quant", "rows": 8, "K": 4096, "pad": 0, "dtype": "bf16"},
        # fp32 rows cut out of a wider buffer, an odd number of blocks
        {"name": "quant_f32_strided", "op": "quant", "rows": 1000, "K": 4128, "pad": 32, "dtype": "f32"},
        # the gate or up projections of eight experts, quantized when a model is loaded
        {"name": "quant_weights", "op": "quant", "rows": 16384, "K": 4096, "pad": 0, "dtype": "bf16"},
        # a dense projection of one token
        {"name": "matmul_t1", "op": "matmul", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16"},
        # odd sizes: no dimension a multiple of a tile, K ends inside one
        {"name": "matmul_t77_odd", "op": "matmul", "M": 77, "N": 1001, "K": 2080, "dtype": "f32"},
        # a prefill chunk through a dense projection
        {"name": "matmul_t2048", "op": "matmul", "M": 2048, "N": 4096, "K": 4096, "dtype": "bf16"},
        # the largest prefill
        {"name": "matmul_t16384", "op": "matmul", "M": 16384, "N": 4096, "K": 4096, "dtype": "bf16"},
        # one sequence decoding
        {"name": "w4a8_t1", "op": "w4a8", "T": 1, **moe},
        # eight sequences, fed by the router weight
        {"name": "w4a8_t8_router", "op": "w4a8", "T": 8, **moe, "router": True},
        # sixteen sequences, with two always-on bf16 experts
        {"name": "w4a8_t16_shared", "op": "w4a8", "T": 16, **moe, "shared": 2},
        # one and eight sequences on MXFP4 experts
        {"name": "mxfp4_t1_router", "op": "mxfp4", "T": 1, **moe, "router": True},
        {"name": "mxfp4_t8", "op": "mxfp4", "T": 8, **moe},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "matmul", "w4a8", "mxfp4"])
    if op == "quant":
        K = 32 * _log_int(rng, 1, 512)
        rows = _log_int(rng, 1, min(40000, (16384 * 4096) // K))
        return {"op": op, "rows": rows, "K": K, "pad": rng.choice([0, 0, 8, 64]), "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op == "matmul":
        K = 32 * _log_int(rng, 2, 256)
        N = _log_int(rng, 64, 8192)
        M = _log_int(rng, 1, min(16384, (16384 * 4096 * 4096) // (N * K)))
        return {"op": op, "M": M, "N": N, "K": K, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    E = rng.choice([8, 16, 60, 64, 128, 256])
    return {"op": op, "T": rng.randint(1, 16), "E": E, "H": 128 * rng.randint(2, 32), "N": 128 * rng.randint(1, 16),
            "k": rng.randint(1, min(8, E)), "router": rng.random() < 0.4, "shared": rng.choice([0, 0, 1])}


def work(case):
    """Bytes and operations of one pass: each input once, each output once.  quant: the rows in, codes and scales
    out, and back to bf16 values.  MoE: the weights of the experts that T tokens reach on average."""
    if case["op"] == "quant":
        n = case["rows"] * case["K"]
        four = n / 2 + n / 32
        return {"bytes": n * DTYPES[case["dtype"]].itemsize + 2 * four + 2 * n, "flops": 4 * n}
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K / 2 + K / 32) + M * N * DTYPES[case["dtype"]].itemsize, "flops": 2.0 * M * N * K}
    T, E, H, N, k = (case[n] for n in ("T", "E", "H", "N", "k"))
    touched = E * (1 - (1 - k / E) ** T)
    scale = 2 / 128 if case["op"] == "w4a8" else 1 / 32
    shared = case["shared"] * 3 * H * N * 2
    routing = E * H * 2 if case["router"] else T * E * 4
    return {"bytes": touched * 3 * H * N * (0.5 + scale) + shared + routing + 2 * T * H * 2,
            "flops": T * (k + case["shared"]) * 6.0 * H * N}


# ---- inputs ----------------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, rows, K, dtype):
    """Unit normals with one channel in a hundred twenty times as large, as hidden states have them."""
    x = _randn(g, rows, K)
    x[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 20.0
    return x.to(dtype)


def _words(g, mask, *shape):
    r = torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    return r.bitwise_and_(mask)


def _mx_rows(g, rows, K):
    """MXFP4 rows: random codes, scales of a few neighbouring powers of two."""
    codes = torch.randint(0, 256, (rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(118, 123, (rows, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales


def _projection(g, op, E, rows, K):
    """Random expert weights [E, rows, K] in the operator's format."""
    if op == "mxfp4":
        codes, scales = _mx_rows(g, E * rows, K)
        return codes.view(E, rows, K // 2), scales.view(E, rows, K // 32)
    # nibbles are the sum of two 3-bit numbers and one bit: 0..15, most of them near 7.5
    packed = _words(g, 0x77777777, E, rows, K // 8)
    packed += _words(g, 0x77777777, E, rows, K // 8)
    packed += _words(g, 0x11111111, E, rows, K // 8)
    scales = (0.004 + 0.006 * torch.rand(E, rows, K // 128, generator=g, device="cuda")).to(torch.bfloat16)
    return packed, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}
    if op == "quant":
        x = _activations(g, case["rows"], case["K"] + case["pad"], DTYPES[case["dtype"]])
        s["x"] = x[:, :case["K"]]
        return s
    if op == "matmul":
        s["a"], s["a_scales"] = _mx_rows(g, case["M"], case["K"])
        s["b"], s["b_scales"] = _mx_rows(g, case["N"], case["K"])
        return s
    T, E, H, N = (case[n] for n in ("T", "E", "H", "N"))
    s["gate"], s["gate_scales"] = _projection(g, op, E, N, H)
    s["up"], s["up_scales"] = _projection(g, op, E, N, H)
    s["down"], s["down_scales"] = _projection(g, op, E, H, N)
    s["x"] = _activations(g, T, H, torch.bfloat16)
    if case["router"]:
        s["wr"] = (_randn(g, E, H) / math.sqrt(H)).to(torch.bfloat16)
    else:
        s["logits"] = _randn(g, T, E)
    n = case["shared"]
    s["shared"] = tuple((0.02 * _randn(g, *d)).to(torch.bfloat16) for d in ((n, N, H), (n, N, H), (n, H, N))) if n else None
    if own:   # the layer's handle and the buffers that a serving loop keeps
        import bit_quantized_moe_token_b200 as moe
        kind = moe.Layer if op == "w4a8" else moe.LayerMX
        sh = s["shared"] or (None, None, None)
        s["layer"] = kind(E, H, N, s["gate"], s["up"], s["down"], s["gate_scales"], s["up_scales"], s["down_scales"],
                          sh_gate=sh[0], sh_up=sh[1], sh_down=sh[2])
        s["ws"] = moe.alloc_decode_workspace(s["layer"], T, case["k"])
    return s


# ---- the plain forms ---------------------------------------------------------------------------

def _e2m1_values(codes):
    """uint8 [..., n], low nibble first -> fp32 [..., 2 n]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    return table[torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).int()]


def _mx_values(codes, scales):
    v = _e2m1_values(codes)
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(scales.float() - 127.0).unsqueeze(-1)).flatten(-2)


def _int4_values(packed, scales):
    shifts = torch.arange(0, 32, 4, device=packed.device, dtype=torch.int32)
    v = ((packed.unsqueeze(-1) >> shifts) & 15).flatten(-2).float() - 8.0
    return (v.unflatten(-1, (-1, 128)) * scales.float().unsqueeze(-1)).flatten(-2)


def _plain_quant(x):
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)    # floor(log2 amax) - 2
    v = torch.ldexp(b, -e)
    a = v.abs()
    m = torch.zeros_like(a)
    m = torch.where(a > 0.25, 0.5, m)
    m = torch.where(a >= 0.75, 1.0, m)
    m = torch.where(a > 1.25, 1.5, m)
    m = torch.where(a >= 1.75, 2.0, m)
    m = torch.where(a > 2.5, 3.0, m)
    m = torch.where(a >= 3.5, 4.0, m)
    m = torch.where(a > 5.0, 6.0, m)
    return torch.ldexp(torch.where(v < 0, -m, m), e).flatten(-2).to(torch.bfloat16), (e + 127).squeeze(-1)


def _fp8(x):
    """Per-row FP8: the codes' values and the scale (divided by a tensor: by a number, torch multiplies with its
    rounded reciprocal)."""
    s = x.abs().amax(-1, keepdim=True)
    s = s / torch.full_like(s, 448.0)
    q = torch.where(s > 0, x / s, torch.zeros_like(x)).to(torch.float8_e4m3fn).float()
    return q, s


def _plain_moe(s):
    c = s["case"]
    T, k = c["T"], c["k"]
    values = _int4_values if c["op"] == "w4a8" else _mx_values
    x = s["x"].float()
    logits = x @ s["wr"].float().T if c["router"] else s["logits"]
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k].reshape(-1)
    e = torch.exp(top - top[:, :1])
    gates = e / e.sum(-1, keepdim=True)
    q, sx = _fp8(x)
    q, sx = q.repeat_interleave(k, 0).unsqueeze(-1), sx.repeat_interleave(k, 0)
    g = (values(s["gate"][ids], s["gate_scales"][ids]) @ q).squeeze(-1) * sx
    u = (values(s["up"][ids], s["up_scales"][ids]) @ q).squeeze(-1) * sx
    h = g / (1.0 + torch.exp(-g)) * u
    hq, sh = _fp8(h)
    y = (values(s["down"][ids], s["down_scales"][ids]) @ hq.unsqueeze(-1)).squeeze(-1) * sh
    out = (y.view(T, k, -1) * gates.unsqueeze(-1)).sum(1)
    if s["shared"]:
        wg, wu, wd = s["shared"]
        g, u = x @ wg.float().transpose(1, 2), x @ wu.float().transpose(1, 2)      # [n, T, N]
        out = out + (g / (1.0 + torch.exp(-g)) * u @ wd.float().transpose(1, 2)).sum(0)
    return out.to(torch.bfloat16)


def run(state):
    c = state["case"]
    if own:
        import bit_quantized_moe_token_b200 as moe
        if c["op"] == "quant":
            codes, scales = moe.quant_mxfp4(state["x"])
            return moe.dequant_mxfp4(codes, scales), scales
        if c["op"] == "matmul":
            return moe.matmul_mxfp4(state["a"], state["a_scales"], state["b"], state["b_scales"], dtype=DTYPES[c["dtype"]])
        if c["router"]:
            return moe.decode_router(state["layer"], state["x"], state["wr"], c["k"], ws=state["ws"])
        return moe.decode(state["layer"], state["x"], state["logits"], c["k"], ws=state["ws"])
    if c["op"] == "quant":
        v, e = _plain_quant(state["x"])
        return v, e.to(torch.uint8)
    if c["op"] == "matmul":
        out = _mx_values(state["a"], state["a_scales"]) @ _mx_values(state["b"], state["b_scales"]).T
        return out.to(DTYPES[c["dtype"]])
    return _plain_moe(state)


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _exact_rows(codes, scales):
    """MXFP4 rows from the format's fields: sign, two exponent bits, one mantissa bit."""
    n = torch.stack((codes % 16, codes // 16), dim=-1).flatten(-2).long()
    e, m = (n // 2) % 4, (n % 2).double()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e.double() - 1)) * torch.where(n >= 8, -1.0, 1.0)
    return v * (2.0 ** (scales.double() - 127)).repeat_interleave(32, -1)


def _exact_int4(packed, scales):
    u = packed.long() % 2 ** 32
    v = torch.stack([u // 16 ** i % 16 - 8 for i in range(8)], dim=-1).flatten(-2).double()
    return v * scales.double().repeat_interleave(128, -1)


def _exact_e4m3(x):
    """x rounded to E4M3 (3 mantissa bits, smallest step 2^-9, at most 448), scaled by its row's maximum.  Both
    divisions are the definition's own, in the type of x: hidden states are bf16 numbers, whose quotients fall on the
    border between two codes often enough that their rounding in fp32 is part of the definition."""
    s = x.abs().max(0, keepdim=True).values
    s = s / torch.full_like(s, 448)
    if s == 0:
        return torch.zeros_like(x).double(), s.double()
    y, s = (x / s).double(), s.double()
    step = 2.0 ** (torch.frexp(y.abs().clamp_min(2.0 ** -6)).exponent.double() - 4)
    return (torch.round(y / step) * step).clamp(-448, 448), s


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        b = s["x"].double().unflatten(-1, (-1, 32))
        top = b.abs().amax(-1, keepdim=True)
        e = torch.where(top > 0, torch.frexp(top).exponent.double() - 3, torch.full_like(top, -127.0))
        e = e.clamp(-127, 127)
        v = b / 2.0 ** e
        step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).double()
        v = (torch.round(v / step) * step).clamp(-6, 6)
        return (v * 2.0 ** e).flatten(-2), None
    if case["op"] == "matmul":
        a, b = _exact_rows(s["a"], s["a_scales"]), _exact_rows(s["b"], s["b_scales"])
        return a @ b.T
    dense = _exact_int4 if case["op"] == "w4a8" else _exact_rows
    silu = lambda v: v / (1 + torch.exp(-v))   # noqa: E731
    rows = []
    for t in range(case["T"]):
        x = s["x"][t].double()
        l = (s["wr"].double() @ x if case["router"] else s["logits"][t].double()).tolist()
        ids = sorted(range(case["E"]), key=lambda i: (-l[i], i))[:case["k"]]
        z = sum(math.exp(l[i] - l[ids[0]]) for i in ids)
        q, sx = _exact_e4m3(s["x"][t].float())
        out = torch.zeros_like(x)
        for i in ids:
            g = dense(s["gate"][i], s["gate_scales"][i]) @ q * sx
            u = dense(s["up"][i], s["up_scales"][i]) @ q * sx
            hq, sh = _exact_e4m3(silu(g) * u)
            out += math.exp(l[i] - l[ids[0]]) / z * sh * (dense(s["down"][i], s["down_scales"][i]) @ hq)
        for j in range(case["shared"]):
            wg, wu, wd = (w[j].double() for w in s["shared"])
            out += wd @ (silu(wg @ x) * (wu @ x))
        rows.append(out)
    return torch.stack(rows)
