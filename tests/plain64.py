"""Plain 64-bit forms of the MXFP4 operators and of the few-token layer, for the tests.

Tolerances: a value rounded once to bf16 is off by at most 2^-8 of itself, to fp32 by 2^-24.  An fp32 sum of n terms is
off by at most n 2^-23 times the sum of their magnitudes, in any order and with truncating additions."""
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def quant_mxfp4(x):
    """(codes [.., K/2], scales [.., K/32]) of MXFP4 rows: the nearest E2M1 value by distance, ties to the even code."""
    b = x.double().unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    b = torch.where(bad, torch.zeros_like(b), b)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1, torch.full_like(amax, -999)).double() - 2
    e = e.clamp(-127, 127)
    v = b * torch.exp2(-e)
    grid = E2M1.to(x.device)
    d = (v.abs().clamp(max=6.0).unsqueeze(-1) - grid).abs()
    # the smaller distance; of two equal ones the even code: add less than any real difference to the odd codes
    odd = (torch.arange(8, device=x.device) % 2).double() * 1e-12
    code = (d + odd).argmin(-1) + 8 * torch.signbit(x.double().unflatten(-1, (-1, 32))).long()
    code = torch.where(bad, torch.zeros_like(code), code).flatten(-2)
    codes = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
    scales = torch.where(bad, torch.full_like(e, 255), e + 127).squeeze(-1).to(torch.uint8)
    return codes, scales


def mxfp4_values(codes, scales):
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = E2M1.to(codes.device)[n & 7] * (1.0 - 2.0 * (n >> 3))
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return v * s.repeat_interleave(32, -1)


def int4_values(packed, scales):
    n = torch.stack([(packed >> (4 * i)) & 15 for i in range(8)], -1).flatten(-2)
    return (n.double() - 8) * scales.double().repeat_interleave(128, -1)


def matmul_tolerance(a, b, ref, dtype):
    return HALF[dtype] * ref.abs() + a.shape[-1] * 2.0 ** -23 * (a.abs() @ b.abs().T)


def e4m3(x, single=False):
    """(values of the FP8 codes, scale) of a row; single: the two divisions in fp32, as the definition has them."""
    x = x.float() if single else x.double()
    s = x.abs().max(0, keepdim=True).values
    s = s / torch.full_like(s, 448)          # by a tensor: by a number, torch multiplies with its rounded reciprocal
    if s == 0:
        return torch.zeros_like(x).double(), s.double()
    y = (x / s).double()
    step = torch.exp2(torch.frexp(y.abs().clamp_min(2.0 ** -6)).exponent.double() - 4)
    return (torch.round(y / step) * step).clamp(-448, 448), s.double()


def few_token_layer(x, logits, k, expert, shared=None):
    """(out [T, H], tolerance [T, H]) of the layer in 64 bits.  expert(e) -> its gate, up [N, H] and down [H, N] values;
    shared: (gate, up [n, Ns, H], down [n, H, Ns]).  logits: [T, E], NaN ranked last.

    Tolerance: half a bf16 step of the result, the bound of the fp32 sums, and for every FP8 code of h that lies so
    near a border that the sums' error can decide it one code step through its down weight."""
    outs, tols = [], []
    eps = 2.0 ** -23
    for t in range(x.shape[0]):
        l = torch.where(torch.isnan(logits[t]), torch.full_like(logits[t], float("-inf")), logits[t]).double().tolist()
        ids = sorted(range(len(l)), key=lambda i: (-l[i], i))[:k]
        gates = torch.softmax(torch.tensor([l[i] for i in ids], dtype=torch.float64), 0).tolist()
        q, sx = e4m3(x[t], single=True)
        out = torch.zeros(x.shape[1], dtype=torch.float64, device=x.device)
        tol = torch.zeros_like(out)
        for i, gate in zip(ids, gates):
            wg, wu, wd = expert(i)
            g, u = wg @ q * sx, wu @ q * sx
            # sums of 128 (or 32) products inside a group, then over the groups; INT4 codes carry an offset of 8 in
            # the sum, at most 16 / 7 times the magnitudes of the rest at the ends of the range and 16 below them
            n_sum = 160 + wg.shape[1] // 32
            dg, du = (n_sum * eps * 4 * (w.abs() @ q.abs()) * sx for w in (wg, wu))
            sg = torch.sigmoid(g)
            h = g * sg * u
            dh = (sg * (1 + g.abs() * (1 - sg)) * u.abs() * dg + (g * sg).abs() * du + 16 * eps * h.abs())
            hq, sh = e4m3(h)
            lo, hi = (torch.round((h + d) / (sh + (sh == 0)) / st) * st for d, st in ((-dh, _steps(h, sh)), (dh, _steps(h, sh))))
            flips = torch.where((hi - lo).abs() > 0, _steps(h, sh), torch.zeros_like(h))
            y = wd @ hq * sh
            out += gate * y
            tol += gate * sh * (wd.abs() @ (2 * flips + (160 + wd.shape[1] // 32) * eps * 4 * hq.abs()))
        if shared is not None:
            for wg, wu, wd in zip(*(w.double() for w in shared)):
                xd = x[t].double()
                g, u = wg @ xd, wu @ xd
                a = g * torch.sigmoid(g) * u
                out += wd @ a
                # fp32 sums on both projections, and an activation held in at least 16 bits between them
                ea = (wg.abs() @ xd.abs()) * u.abs() + (wu.abs() @ xd.abs()) * g.abs()
                tol += wd.abs() @ (wg.shape[1] * eps * 2 * ea + (2.0 ** -16 + wd.shape[1] * eps) * a.abs())
        outs.append(out)
        tols.append(tol)
    ref, tol = torch.stack(outs), torch.stack(tols)
    return ref, tol + HALF[torch.bfloat16] * (ref.abs() + tol) + 1e-30


def _steps(h, sh):
    y = (h / (sh + (sh == 0))).abs().clamp(2.0 ** -6, 448)
    return torch.exp2(torch.frexp(y).exponent.double() - 4)
