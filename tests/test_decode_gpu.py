"""The few-token layer (W4A8 and MXFP4 experts) against the plain 64-bit form."""
import pytest
import torch

import plain64
from conftest import cuda_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not cuda_ok():
        pytest.skip("no CUDA device")


@pytest.fixture
def moe():
    import bit_quantized_moe_token_b200 as m
    return m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(fmt, g, E, rows, K):
    """Random expert weights: every nibble as likely as any other."""
    if fmt == "w4a8":
        w = torch.randint(-2 ** 31, 2 ** 31, (E, rows, K // 8), generator=g, device="cuda", dtype=torch.int64).int()
        return w, (0.004 + 0.006 * torch.rand(E, rows, K // 128, generator=g, device="cuda")).bfloat16()
    w = torch.randint(0, 256, (E, rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    return w, torch.randint(116, 123, (E, rows, K // 32), generator=g, device="cuda", dtype=torch.uint8)


class Case:
    def __init__(self, moe, fmt, E, H, N, seed, n_shared=0, Ns=128):
        g = _gen(seed)
        self.fmt = fmt
        self.w = [_rows(fmt, g, E, N, H), _rows(fmt, g, E, N, H), _rows(fmt, g, E, H, N)]
        self.shared = None
        if n_shared:
            self.shared = tuple((0.02 * torch.randn(n_shared, *d, generator=g, device="cuda")).bfloat16()
                                for d in ((Ns, H), (Ns, H), (H, Ns)))
        kind = moe.Layer if fmt == "w4a8" else moe.LayerMX
        sh = self.shared or (None, None, None)
        (a, sa), (b, sb), (c, sc) = self.w
        self.layer = kind(E, H, N, a, b, c, sa, sb, sc, sh_gate=sh[0], sh_up=sh[1], sh_down=sh[2])
        self.E, self.H, self.N, self.g = E, H, N, g

    def tokens(self, T):
        x = torch.randn(T, self.H, generator=self.g, device="cuda")
        x[:, ::97] *= 20.0
        return x.bfloat16(), torch.randn(T, self.E, generator=self.g, device="cuda")

    def expert(self, e):
        f = plain64.int4_values if self.fmt == "w4a8" else plain64.mxfp4_values
        return tuple(f(w[e], s[e]) for w, s in self.w)

    def check(self, out, x, logits, k):
        ref, tol = plain64.few_token_layer(x, logits, k, self.expert, self.shared)
        err = (out.double() - ref).abs()
        assert (err <= tol).all(), f"worst {float((err / tol).max()):.3g} of the tolerance"
        # all outputs together: a bf16 rounding each, and what the tolerance adds for codes at a border
        extra = torch.linalg.norm(tol - 2.0 ** -8 * ref.abs())
        assert torch.linalg.norm(err) <= 2.0 ** -8 * torch.linalg.norm(ref) + extra


def _dirty_ws(moe, layer, T, k):
    ws = moe.alloc_decode_workspace(layer, T, k)
    ws.fill_(0xFF)
    return ws


FMT = ["w4a8", "mxfp4"]
SHAPES = [  # E, H, N, k, T
    (1, 128, 128, 1, 1), (8, 256, 128, 2, 1), (5, 384, 256, 3, 7), (16, 1152, 640, 4, 9), (60, 512, 896, 4, 16),
    (3, 640, 384, 3, 16), (64, 2048, 1024, 6, 3), (256, 1024, 512, 8, 16), (1024, 256, 128, 8, 13), (33, 4096, 2048, 6, 2),
    (12, 4096, 2048, 6, 16), (9, 4224, 2176, 2, 5), (4, 8192, 1024, 2, 8), (4, 8192, 256, 2, 16), (2, 16384, 256, 1, 5),
    (2, 256, 8192, 2, 3), (2, 1920, 4096, 2, 12)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("E,H,N,k,T", SHAPES)
def test_shapes(moe, fmt, E, H, N, k, T):
    c = Case(moe, fmt, E, H, N, E + H + N + T)
    x, lg = c.tokens(T)
    out = moe.decode(c.layer, x, lg, k, ws=_dirty_ws(moe, c.layer, T, k))
    c.check(out, x, lg, k)
    assert moe.moe_last_device_status() == 0


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("n_shared,Ns,T,H,N", [(1, 128, 1, 256, 128), (2, 384, 5, 1152, 256), (3, 256, 16, 640, 128),
                                               (2, 2048, 2, 4096, 2048), (1, 8192, 9, 512, 256)])
def test_shared_experts(moe, fmt, n_shared, Ns, T, H, N):
    c = Case(moe, fmt, 8, H, N, n_shared + Ns + T, n_shared, Ns)
    x, lg = c.tokens(T)
    out = moe.decode(c.layer, x, lg, 3, ws=_dirty_ws(moe, c.layer, T, 3))
    c.check(out, x, lg, 3)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("E,H,N,k,T,n_shared", [(16, 256, 128, 2, 1, 0), (60, 1152, 256, 6, 7, 1), (256, 4096, 128, 6, 8, 0),
                                                (1024, 512, 128, 8, 16, 0), (4, 16384, 128, 2, 3, 0)])
def test_router_form(moe, fmt, E, H, N, k, T, n_shared):
    """The router form is the layer on x wr^T: the 64-bit form with the logits summed in 64 bits, where no two of them
    are nearer at the selection's edge than fp32 sums can be off."""
    c = Case(moe, fmt, E, H, N, E * 3 + T, n_shared)
    x, _ = c.tokens(T)
    wr = (torch.randn(E, H, generator=c.g, device="cuda") / H ** 0.5).bfloat16()
    lg = x.double() @ wr.double().T
    top = lg.sort(dim=1, descending=True).values
    assert k == E or ((top[:, k - 1] - top[:, k]) > 1e-5).all()
    out = moe.decode_router(c.layer, x, wr, k, ws=_dirty_ws(moe, c.layer, T, k))
    c.check(out, x, lg, k)


@pytest.mark.parametrize("fmt", FMT)
def test_routing_corners(moe, fmt):
    """Equal logits (lower index first), NaN logits (last), all tokens on the same experts, a token of zeros."""
    c = Case(moe, fmt, 40, 512, 256, 11)
    x, lg = c.tokens(6)
    lg[0] = 0.0
    lg[1, :38] = float("nan")
    lg[2, 5:] = float("-inf")
    lg[3] = lg[4]
    x[5] = 0.0
    out = moe.decode(c.layer, x, lg, 2, ws=_dirty_ws(moe, c.layer, 6, 2))
    c.check(out, x, lg, 2)
    assert (out[5] == 0).all()
    same = torch.zeros(16, 40, device="cuda")
    same[:, 7], same[:, 31] = 2.0, 1.0
    x, _ = c.tokens(16)
    out = moe.decode(c.layer, x, same, 2, ws=_dirty_ws(moe, c.layer, 16, 2))
    c.check(out, x, same, 2)


@pytest.mark.parametrize("fmt", FMT)
def test_rows_alone_and_in_a_batch(moe, fmt):
    """A token alone, in a batch, and in another place of the batch (where the kernel sums in another order)."""
    c = Case(moe, fmt, 32, 1024, 512, 12, n_shared=1)
    x, lg = c.tokens(8)
    full = moe.decode(c.layer, x, lg, 4)
    back = moe.decode(c.layer, x.flip(0).contiguous(), lg.flip(0).contiguous(), 4).flip(0)
    for t in range(8):
        one = moe.decode(c.layer, x[t:t + 1], lg[t:t + 1], 4)[0]
        ref, tol = plain64.few_token_layer(x[t:t + 1], lg[t:t + 1], 4, c.expert, c.shared)
        assert ((one.double() - ref[0]).abs() <= tol[0]).all()
        assert ((full[t].double() - ref[0]).abs() <= tol[0]).all()
        assert ((back[t].double() - ref[0]).abs() <= tol[0]).all()


@pytest.mark.parametrize("fmt", FMT)
def test_out_may_be_x_and_neighbours_stay(moe, fmt):
    c = Case(moe, fmt, 8, 256, 128, 13)
    x, lg = c.tokens(3)
    want = moe.decode(c.layer, x, lg, 2)
    buf = torch.full((5, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    buf[1:4] = x
    n = moe.alloc_decode_workspace(c.layer, 3, 2).numel()
    ws = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    moe.decode(c.layer, buf[1:4], lg, 2, out=buf[1:4], ws=ws[256:256 + n])
    assert torch.equal(buf[1:4], want)
    assert (buf[[0, 4]] == 3.0).all() and (ws[:256] == 0x5A).all() and (ws[256 + n:] == 0x5A).all()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("router", [False, True])
def test_captured_graphs_share_a_workspace(moe, fmt, router):
    """Two graphs of different shapes on one workspace, replayed in turn with new inputs, an eager call between."""
    c = Case(moe, fmt, 32, 1024, 256, 14)
    wr = (torch.randn(32, 1024, generator=c.g, device="cuda") / 32).bfloat16()
    ws = torch.full((moe.alloc_decode_workspace(c.layer, 16, 6).numel(),), 0xFF, dtype=torch.uint8, device="cuda")

    def call(x, lg, k, out):
        return moe.decode_router(c.layer, x, wr, k, out=out, ws=ws) if router else moe.decode(c.layer, x, lg, k, out=out, ws=ws)

    graphs = []
    for T, k in ((2, 6), (11, 3)):
        x, lg = c.tokens(T)
        out = torch.empty_like(x)
        call(x, lg, k, out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(x, lg, k, out)
        graphs.append((g, x, lg, k, out))
    for _ in range(3):
        for g, x, lg, k, out in graphs:
            nx, nl = c.tokens(x.shape[0])
            x.copy_(nx)
            lg.copy_(nl)
            want = call(nx, nl, k, torch.empty_like(nx)).clone()
            out.zero_()
            g.replay()
            assert torch.equal(out, want)


@pytest.mark.parametrize("fmt", FMT)
def test_two_streams_at_once(moe, fmt):
    """Calls that overlap, each with its own workspace."""
    c = Case(moe, fmt, 64, 2048, 1024, 15)
    sets = []
    for _ in range(2):
        x, lg = c.tokens(4)
        sets.append((x, lg, moe.decode(c.layer, x, lg, 6), torch.empty_like(x), _dirty_ws(moe, c.layer, 4, 6), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, lg, _, out, ws, s in sets:
            moe.decode(c.layer, x, lg, 6, out=out, ws=ws, stream=s)
    torch.cuda.synchronize()
    for _, _, want, out, _, _ in sets:
        assert torch.equal(out, want)
    assert moe.moe_last_device_status() == 0


@pytest.mark.parametrize("fmt", FMT)
def test_scratch_of_a_call_on_another_stream(moe, fmt):
    """Without a workspace of its own the call takes one that the current stream's next allocations do not get."""
    c = Case(moe, fmt, 64, 2048, 1024, 18)
    x, lg = c.tokens(4)
    wr = (torch.randn(64, 2048, generator=c.g, device="cuda") / 45.0).bfloat16()
    want, routed = moe.decode(c.layer, x, lg, 6), moe.decode_router(c.layer, x, wr, 6)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for at in (s, s.cuda_stream):
        outs = []
        for _ in range(10):
            outs.append((moe.decode(c.layer, x, lg, 6, stream=at), moe.decode_router(c.layer, x, wr, 6, stream=at)))
            n = moe.alloc_decode_workspace(c.layer, 4, 6).fill_(0xFF).numel()
        torch.cuda.synchronize()
        assert n > 0
        for a, b in outs:
            assert torch.equal(a, want) and torch.equal(b, routed)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_token_that_is_not_finite_stays_alone(moe, fmt, bad):
    """Its own outputs are NaN; its neighbours' on the same experts are, bit for bit, what they were."""
    c = Case(moe, fmt, 6, 512, 256, 19, n_shared=1)
    x, lg = c.tokens(9)
    want = moe.decode(c.layer, x, lg, 3)
    x[4, 17] = bad
    got = moe.decode(c.layer, x, lg, 3)
    rest = [t for t in range(9) if t != 4]
    assert torch.equal(got[rest], want[rest])
    assert torch.isnan(got[4]).all()


def test_agrees_with_the_forward(moe):
    """On W4A8 weights the few-token layer and moe_w4a8_forward compute the same layer: both within the tolerance."""
    c = Case(moe, "w4a8", 64, 2048, 1024, 16, n_shared=2, Ns=512)
    x, lg = c.tokens(8)
    c.check(moe.decode(c.layer, x, lg, 6), x, lg, 6)
    c.check(moe.forward(c.layer, x, lg, 6), x, lg, 6)


def test_quantized_model_as_it_is_used(moe):
    """bf16 weights -> make_layer_mxfp4 -> a dense MXFP4 projection -> decode_router, one token after another."""
    g = _gen(17)
    E, H, N, k = 16, 512, 256, 4
    w = [(0.02 * torch.randn(E, *d, generator=g, device="cuda")).bfloat16() for d in ((N, H), (N, H), (H, N))]
    layer = moe.make_layer_mxfp4(*w)
    wo = moe.quant_mxfp4((torch.randn(H, H, generator=g, device="cuda") / H ** 0.5).bfloat16())
    wr = (torch.randn(E, H, generator=g, device="cuda") / H ** 0.5).bfloat16()
    ws = moe.alloc_decode_workspace(layer, 2, k)
    x = torch.randn(2, H, generator=g, device="cuda").bfloat16()

    def expert(e):
        return tuple(plain64.mxfp4_values(c[e], s[e]) for c, s in ((layer.gate_f4, layer.gate_e8), (layer.up_f4, layer.up_e8), (layer.down_f4, layer.down_e8)))

    for _ in range(3):
        qx = moe.quant_mxfp4(x)
        y = moe.matmul_mxfp4(*qx, *wo)
        va, vb = plain64.mxfp4_values(*qx), plain64.mxfp4_values(*wo)
        ref = va @ vb.T
        assert ((y.double() - ref).abs() <= plain64.matmul_tolerance(va, vb, ref, torch.bfloat16)).all()
        out = moe.decode_router(layer, y, wr, k, ws=ws)
        ref, tol = plain64.few_token_layer(y, y.double() @ wr.double().T, k, expert)
        assert ((out.double() - ref).abs() <= tol).all()
        x = (x + 20 * out).bfloat16()


def test_no_tokens(moe):
    c = Case(moe, "mxfp4", 8, 256, 128, 18)
    x, lg = c.tokens(0)
    assert moe.decode(c.layer, x, lg, 2).shape == (0, 256)


def test_refusals(moe):
    c = Case(moe, "mxfp4", 8, 256, 128, 19)
    x, lg = c.tokens(17)
    with pytest.raises(ValueError):
        moe.decode(c.layer, x, lg, 2)                                   # more than 16 tokens
    x, lg = x[:4].contiguous(), lg[:4].contiguous()
    ws = moe.alloc_decode_workspace(c.layer, 4, 2)
    with pytest.raises(ValueError):
        moe.decode(c.layer, x.float(), lg, 2, ws=ws)
    with pytest.raises(ValueError):
        moe.decode(c.layer, x, lg[:, :7].contiguous(), 2, ws=ws)
    with pytest.raises(ValueError):
        moe.decode(c.layer, x, lg, 2, out=torch.empty(3, 256, dtype=torch.bfloat16, device="cuda"), ws=ws)
    with pytest.raises(moe.MoeError):
        moe.decode(c.layer, x, lg, 2, ws=ws[:128])
    with pytest.raises(moe.MoeError):
        moe.decode(c.layer, x, lg, 9, ws=ws)
    with pytest.raises(ValueError):
        moe.decode(c.layer, x.cpu(), lg, 2, ws=ws)
