"""The bound of norm64 is tight enough to tell: layers with a fault in them lie outside it at every size that the GPU
tests run, on inputs drawn as theirs are."""
import pytest
import torch

import norm64
import plain64
from test_decode_gpu import SHAPES

MUTATIONS = ["last 128 of gate", "last 128 of up", "last 32 of down", "gate 2 % off", "down 2 % off", "one scale of gate doubled",
             "first gate 5 % off", "gate and up swapped"]


def _weights(fmt, g, rows, K):
    if fmt == "w4a8":
        w = torch.randint(-2 ** 31, 2 ** 31, (rows, K // 8), generator=g, dtype=torch.int64).int()
        return plain64.int4_values(w, (0.004 + 0.006 * torch.rand(rows, K // 128, generator=g)).bfloat16())
    w = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    return plain64.mxfp4_values(w, torch.randint(116, 123, (rows, K // 32), generator=g, dtype=torch.uint8))


def _mutate(how, wg, wu, wd):
    wg, wu, wd = wg.clone(), wu.clone(), wd.clone()
    if how == "last 128 of gate":
        wg[:, -128:] = 0
    elif how == "last 128 of up":
        wu[:, -128:] = 0
    elif how == "last 32 of down":
        wd[:, -32:] = 0
    elif how == "gate 2 % off":
        wg *= 1.02
    elif how == "down 2 % off":
        wd *= 1.02
    elif how == "one scale of gate doubled":
        wg[:, :32] *= 2
    elif how == "gate and up swapped":
        wg, wu = wu, wg
    return wg, wu, wd


@pytest.mark.parametrize("fmt", ["w4a8", "mxfp4"])
@pytest.mark.parametrize("E,H,N,k,T", SHAPES)
def test_faults_lie_outside_the_bound(fmt, E, H, N, k, T):
    g = torch.Generator()
    g.manual_seed(E + H + N + T)
    x = torch.randn(1, H, generator=g)
    x[:, ::97] *= 20.0
    x, logits = x.bfloat16(), torch.randn(1, E, generator=g)
    experts = {}

    def expert(e):
        if e not in experts:
            experts[e] = (_weights(fmt, g, N, H), _weights(fmt, g, N, H), _weights(fmt, g, H, N))
        return experts[e]

    ref, bound = norm64.few_token_layer(x, logits, k, expert)
    assert bound[0] <= 0.02 * torch.linalg.norm(ref[0])      # a bf16 step, and a code or two of h at a border
    # the rounded result itself lies inside
    assert torch.linalg.norm(ref[0].bfloat16().double() - ref[0]) <= bound[0]
    for how in MUTATIONS:
        if how.startswith("first gate"):
            bad, _ = norm64.few_token_layer(x, logits, k, expert, gates_of=lambda p: torch.cat([1.05 * p[:1], p[1:]]))
        else:
            bad, _ = norm64.few_token_layer(x, logits, k, lambda e: _mutate(how, *expert(e)))
        err = torch.linalg.norm(bad[0] - ref[0])
        assert err > bound[0], f"{how}: {float(err / bound[0]):.3g} of the bound"
