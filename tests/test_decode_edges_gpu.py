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


def _identity(fmt, rows, K, columns):
    """Weights [1, rows, K] with a one in column columns[n] of row n."""
    w = torch.zeros(1, rows, K, device="cuda", dtype=torch.int64)
    w[0, torch.arange(rows, device="cuda"), columns] = 1
    if fmt == "mxfp4":     # E2M1 code 2 is 1, E8M0 scale 127 is 1
        codes = (2 * w).unflatten(-1, (-1, 2))
        return ((codes[..., 0] + 16 * codes[..., 1]).to(torch.uint8),
                torch.full((1, rows, K // 32), 127, dtype=torch.uint8, device="cuda"))
    n = (w + 8).unflatten(-1, (-1, 8))
    packed = (n << torch.arange(0, 32, 4, device="cuda")).sum(-1)
    packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).int()
    return packed, torch.ones(1, rows, K // 128, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T", [4, 16])
def test_tokens_codes_are_those_of_ieee_division(moe, fmt, T):
    """Every quotient of bf16 numbers that a token's quantization meets, x / (amax / 448): 128 mantissas of amax (a token
    each) by 128 mantissas and 18 exponents of x (the columns), as f16 (T = 4) and FP8 (T = 16) fragments.

    The layer reads them out: one expert, whose gate rows all take the column of amax (so that silu(g) is one positive
    number), its up row n column n, its down row n h[n].  h[n] is then proportional to code[n], so is its FP8 code, and
    out[n] / out[at amax] = code[n] / 448 to bf16's rounding, 2^-7 in all: neighbouring codes differ by 2^-4 or more.

    W4A8 sums codes times nibbles n = 8 (a zero) or 9 onto -8 sum q, in fp32: with S the sum of a group's |q|, no partial
    sum exceeds 8 S + 9 S, and each of the group's some 20 additions (16 MMAs in chains, which may truncate, and the joins) is
    off by at most 2^-23 of that, so a code read out is off by 20 17 2^-23 S."""
    H = 128 * 18
    mantissa = torch.arange(128, 256, device="cuda").double() / 128
    x = (mantissa[:, None] * 2.0 ** -torch.arange(18, device="cuda").double()).flatten()      # column c: 2^-(c % 18)
    top = H - 1
    cols = torch.arange(H, device="cuda")
    gate, up = _identity(fmt, H, H, torch.full_like(cols, top)), _identity(fmt, H, H, cols)
    kind = moe.Layer if fmt == "w4a8" else moe.LayerMX
    layer = kind(1, H, H, gate[0], up[0], up[0], gate[1], up[1], up[1])
    lg = torch.zeros(T, 1, device="cuda")
    ws = moe.alloc_decode_workspace(layer, T, 1)
    for first in range(0, 128, T):
        amax = mantissa[first:first + T]
        tokens = x.repeat(T, 1)
        tokens = torch.where(tokens > amax[:, None], tokens / 2, tokens)
        tokens[:, 1::2] *= -1
        tokens[:, top] = amax
        tokens = tokens.bfloat16()
        out = moe.decode(layer, tokens, lg, 1, ws=ws).double()
        scale = amax.float() / torch.full_like(amax, 448).float()
        want = (tokens.float() / scale[:, None]).to(torch.float8_e4m3fn).double()
        got = out / out[:, top:] * 448
        assert (want[:, top] == 448).all()
        tol = 2.0 ** -6 * want.abs()
        if fmt == "w4a8":
            groups = want.abs().unflatten(1, (-1, 128)).sum(2)
            tol += 20 * 17 * 2.0 ** -23 * groups.repeat_interleave(128, 1)
        assert ((got - want).abs() <= tol).all()
