"""The few-token layer at the ends of its inputs' range."""
import ctypes
import threading

import pytest
import torch

from conftest import cuda_ok
from test_decode_gpu import FMT, Case, _dirty_ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not cuda_ok():
        pytest.skip("no CUDA device")


@pytest.fixture
def moe():
    import bit_quantized_moe_token_b200 as m
    return m


def _run(moe, c, x, routing, k, router):
    ws = _dirty_ws(moe, c.layer, x.shape[0], k)
    return (moe.decode_router if router else moe.decode)(c.layer, x, routing, k, ws=ws)


# E, H, N, k, T.  The last two have more routed rows of h for one CTA's down units than its shared memory holds, so that
# the rows go through the workspace.
NOT_FINITE = [(6, 512, 256, 3, 1), (6, 512, 256, 3, 9), (40, 1152, 640, 2, 4), (3, 640, 384, 3, 16), (2, 256, 8192, 2, 9)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("router", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("E,H,N,k,T", NOT_FINITE)
def test_a_token_that_is_not_finite_has_nan_outputs(moe, fmt, router, bad, E, H, N, k, T):
    """Without a shared expert: its routed sums are NaN, so its outputs are, and its neighbours' stay bit for bit."""
    c = Case(moe, fmt, E, H, N, 31 + T)
    x, lg = c.tokens(T)
    wr = (torch.randn(E, H, generator=c.g, device="cuda") / H ** 0.5).bfloat16()
    routing = wr if router else lg
    want = _run(moe, c, x, routing, k, router)
    assert torch.isfinite(want).all()
    t = T // 2
    x[t, 17] = bad
    got = _run(moe, c, x, routing, k, router)
    assert torch.isnan(got[t]).all()
    rest = [i for i in range(T) if i != t]
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("T", [1, 9])
def test_a_token_of_zeros_but_one_that_is_not_finite(moe, fmt, bad, T):
    c = Case(moe, fmt, 6, 512, 256, 32)
    x, lg = c.tokens(T)
    x[T - 1] = 0.0
    x[T - 1, 300] = bad
    got = moe.decode(c.layer, x, lg, 3, ws=_dirty_ws(moe, c.layer, T, 3))
    assert torch.isnan(got[T - 1]).all() and torch.isfinite(got[:T - 1]).all()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("E,H,N,T", [(5, 512, 256, 6), (2, 256, 8192, 9)])
def test_an_expert_whose_scales_are_nan(moe, fmt, which, E, H, N, T):
    """All scales of one expert's gate, up or down projection: its tokens' outputs are NaN, the others' as they were."""
    c = Case(moe, fmt, E, H, N, 33)
    x, lg = c.tokens(T)
    lg[:, 1] = -5.0
    lg[::3, 1] = 5.0
    want = moe.decode(c.layer, x, lg, 1, ws=_dirty_ws(moe, c.layer, T, 1))
    scales = c.w[which][1]
    scales[1] = 255 if fmt == "mxfp4" else float("nan")
    got = moe.decode(c.layer, x, lg, 1, ws=_dirty_ws(moe, c.layer, T, 1))
    mine = torch.arange(T, device="cuda") % 3 == 0
    assert torch.isnan(got[mine]).all()
    assert torch.equal(got[~mine], want[~mine])


@pytest.mark.parametrize("fmt", FMT)
def test_host_threads_with_layers_of_different_sizes(moe, fmt):
    """Two threads, each with its own stream, workspace and layer, whose kernels take different amounts of shared memory:
    the C calls at once (ctypes releases the interpreter's lock), as often as it takes them to meet."""
    call = getattr(moe.lib(), f"moe_{fmt}_decode")
    statuses, outs, threads = [], [], []

    def loop(struct, args):
        torch.cuda.set_device(0)
        statuses.append({call(ctypes.byref(struct), *args) for _ in range(20000)})

    for E, H, N, T in ((2, 128, 128, 1), (2, 1152, 640, 16)):
        c = Case(moe, fmt, E, H, N, 34)
        x, lg = c.tokens(T)
        out, ws, stream = torch.zeros_like(x), _dirty_ws(moe, c.layer, T, 1), torch.cuda.Stream()
        outs.append((out, moe.decode(c.layer, x, lg, 1), x, lg, ws, stream, c))
        args = (x.data_ptr(), lg.data_ptr(), T, 1, out.data_ptr(), ws.data_ptr(), ws.nbytes, stream.cuda_stream)
        threads.append(threading.Thread(target=loop, args=(c.layer.c_struct(), args)))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert statuses == [{moe.MOE_OK}, {moe.MOE_OK}]
    for out, want, *_ in outs:
        assert torch.equal(out, want)


def _scale_by(c, which, power):
    """The projection's scales times 2^power."""
    scales = c.w[which][1]
    if c.fmt == "mxfp4":
        scales += power
    else:
        scales *= 2.0 ** power


# x and the gate and up scales times powers of two: g and u stay near 2^56, h near 2^112
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("x_power,w_power", [(0, 56), (113, -57), (-100, 100)])
@pytest.mark.parametrize("E,H,N,k,T", [(6, 512, 256, 2, 1), (6, 512, 256, 2, 9), (2, 256, 2048, 1, 16)])
def test_large_and_small_values_that_cancel(moe, fmt, x_power, w_power, E, H, N, k, T):
    """Tokens, and rows of h, near the ends of fp32's range: outputs that bf16 holds come out as such."""
    if x_power == -100:
        w_power -= 44 if fmt == "mxfp4" else 40   # g and u near 2^-40
    c = Case(moe, fmt, E, H, N, 35 + T)
    x, lg = c.tokens(T)
    x *= 2.0 ** x_power
    for which in (0, 1):
        _scale_by(c, which, w_power)
    out = moe.decode(c.layer, x, lg, k, ws=_dirty_ws(moe, c.layer, T, k))
    assert torch.isfinite(out).all()
    c.check(out, x, lg, k)
