"""The few-token layer's error by its norm, token by token: tight enough that a dropped group or a scale of 2 % shows
(test_decode_norm_cpu)."""
import pytest
import torch

import norm64
from conftest import cuda_ok
from test_decode_gpu import FMT, SHAPES, Case, _dirty_ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not cuda_ok():
        pytest.skip("no CUDA device")


@pytest.fixture
def moe():
    import bit_quantized_moe_token_b200 as m
    return m


def _check(c, out, x, logits, k):
    ref, bound = norm64.few_token_layer(x, logits, k, c.expert, c.shared)
    err = torch.linalg.norm(out.double() - ref, dim=1)
    assert (err <= bound).all(), f"worst {float((err / bound).max()):.3g} of the bound"


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("E,H,N,k,T", SHAPES)
def test_shapes(moe, fmt, E, H, N, k, T):
    c = Case(moe, fmt, E, H, N, E + H + N + T)
    x, lg = c.tokens(T)
    _check(c, moe.decode(c.layer, x, lg, k, ws=_dirty_ws(moe, c.layer, T, k)), x, lg, k)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("n_shared,Ns,T,H,N", [(1, 128, 1, 256, 128), (3, 256, 16, 640, 128), (2, 2048, 2, 4096, 2048)])
def test_shared_experts(moe, fmt, n_shared, Ns, T, H, N):
    c = Case(moe, fmt, 8, H, N, n_shared + Ns + T, n_shared, Ns)
    x, lg = c.tokens(T)
    _check(c, moe.decode(c.layer, x, lg, 3, ws=_dirty_ws(moe, c.layer, T, 3)), x, lg, 3)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("E,H,N,k,T", [(60, 1152, 256, 6, 7), (256, 4096, 128, 6, 8)])
def test_router_form(moe, fmt, E, H, N, k, T):
    c = Case(moe, fmt, E, H, N, E * 3 + T)
    x, _ = c.tokens(T)
    wr = (torch.randn(E, H, generator=c.g, device="cuda") / H ** 0.5).bfloat16()
    lg = x.double() @ wr.double().T
    top = lg.sort(dim=1, descending=True).values
    assert ((top[:, k - 1] - top[:, k]) > 1e-5).all()      # no two logits at the selection's edge nearer than fp32 sums are off
    _check(c, moe.decode_router(c.layer, x, wr, k, ws=_dirty_ws(moe, c.layer, T, k)), x, lg, k)


def test_the_forward_too(moe):
    """moe_w4a8_forward on the same weights lies inside the same bound."""
    c = Case(moe, "w4a8", 64, 2048, 1024, 16, n_shared=2, Ns=512)
    x, lg = c.tokens(8)
    _check(c, moe.decode(c.layer, x, lg, 6), x, lg, 6)
    _check(c, moe.forward(c.layer, x, lg, 6), x, lg, 6)
