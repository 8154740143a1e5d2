"""A bound on the norm of each token's error of the few-token layer, beside the bound of each element in plain64.

The kernel's output is off from the 64-bit form by
  - the rounding to bf16: at most 2^-8 of each value, so 2^-8 of the norm;
  - FP8 codes of h on the other side of a border: only those whose quotient lies as near to one as the fp32 sums of gate
    and up are off.  Each addition of a group's sum rounds by at most 2^-24 of what is summed so far, which is about the
    root sum of squares of the products; with random signs the whole is off by about sqrt(groups / 6) 2^-24 of it.  The
    band taken here is 6 sqrt(groups + 8) 2^-24 of it, some 15 times that (and 2^-20 of h for SwiGLU and the scale), and every code
    in the band counts with one step through its down column, as a root sum of squares, since their signs are random;
  - the sums of the down product: the same estimate, far below a bf16 step.
The shared experts' terms are bf16 products with fp32 sums, and an activation held in 16 bits: 2^-14 of their norm."""
import torch

import plain64


def _off(w, q, groups):
    """The band of the fp32 sums w q."""
    return 6 * (groups + 8) ** 0.5 * 2.0 ** -24 * torch.sqrt((w * w) @ (q * q))


def few_token_layer(x, logits, k, expert, shared=None, gates_of=None):
    """(out [T, H], bound [T] on the norm of a token's error).  gates_of: of the selected logits (softmax)."""
    outs, bounds = [], []
    for t in range(x.shape[0]):
        l = logits[t].double().tolist()
        ids = sorted(range(len(l)), key=lambda i: (-l[i], i))[:k]
        gates = torch.softmax(torch.tensor([l[i] for i in ids], dtype=torch.float64), 0)
        gates = (gates_of(gates) if gates_of else gates).tolist()
        q, sx = plain64.e4m3(x[t], single=True)
        out = torch.zeros(x.shape[1], dtype=torch.float64, device=x.device)
        var = torch.zeros((), dtype=torch.float64, device=x.device)
        extra = torch.zeros_like(var)
        for i, gate in zip(ids, gates):
            wg, wu, wd = expert(i)
            groups = wg.shape[1] // 32
            g, u = wg @ q * sx, wu @ q * sx
            sg = torch.sigmoid(g)
            h = g * sg * u
            dh = (sg * (1 + g.abs() * (1 - sg)) * u.abs() * _off(wg, q, groups) * sx
                  + (g * sg).abs() * _off(wu, q, groups) * sx + 2.0 ** -20 * h.abs())
            hq, sh = plain64.e4m3(h)
            sh = sh[0]
            if sh == 0:
                continue
            y, dy = (h / sh).abs(), dh / sh
            step = torch.exp2(torch.frexp(y.clamp(2.0 ** -6, 448)).exponent.double() - 4)
            near = torch.round((y + dy) / step) != torch.round((y - dy) / step)
            out += gate * sh * (wd @ hq)
            var += (gate * sh) ** 2 * ((wd * wd).sum(0) * step * step)[near].sum()
            extra += gate * sh * torch.linalg.norm(_off(wd, hq, wd.shape[1] // 32))
        if shared is not None:
            for wg, wu, wd in zip(*(w.double() for w in shared)):
                xd = x[t].double()
                g, u = wg @ xd, wu @ xd
                y = wd @ (g * torch.sigmoid(g) * u)
                out += y
                extra += 2.0 ** -14 * torch.linalg.norm(y)
        outs.append(out)
        bounds.append(2.0 ** -8 * torch.linalg.norm(out) + 2 * torch.sqrt(var) + extra)
    return torch.stack(outs), torch.stack(bounds)
