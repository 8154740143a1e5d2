"""MXFP4 rows on the GPU: quantization, values and product against the plain 64-bit forms."""
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


def _values(g, rows, K, dtype):
    """Normals over many magnitudes, with ties, zeros of both signs and whole blocks of zeros."""
    x = torch.randn(rows, K, generator=g, device="cuda") * torch.exp2(torch.randint(-20, 12, (rows, K // 32, 1), generator=g, device="cuda").float()).expand(-1, -1, 32).reshape(rows, K)
    x[:, ::7] = torch.round(x[:, ::7] * 4) / 4
    x[:, 3::11] = -0.0
    x[rows // 2, :32] = 0.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,K,pad", [(1, 32, 0), (1, 4096, 0), (3, 96, 0), (7, 4128, 32), (257, 2080, 8), (1000, 64, 16), (5, 16384, 0)])
def test_quant_is_exact(moe, rows, K, pad, dtype):
    x = _values(_gen(rows + K), rows, K + pad + (-(K + pad)) % 32, dtype)[:, :K + pad]
    x = x.contiguous()[:, :K]
    codes, scales = moe.quant_mxfp4(x)
    rc, rs = plain64.quant_mxfp4(x)
    assert torch.equal(scales, rs)
    assert torch.equal(codes, rc)
    want = plain64.mxfp4_values(rc, rs)
    for out in (torch.bfloat16, torch.float32):
        got = moe.dequant_mxfp4(codes, scales, dtype=out)
        assert torch.equal(got.double(), want)          # exact in both types


def test_quant_ends_of_the_range(moe):
    """The largest and smallest fp32 and bf16 values, subnormals, ties at every border of the grid."""
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9375])
    rows = [torch.cat([s * borders, torch.zeros(32 - 2 * len(borders)), -s * borders]) for s in (1.0, 2.0 ** -100, 2.0 ** 100)]
    top = torch.zeros(32)
    top[:2] = torch.tensor([3.3895313892515355e38, -3.3895313892515355e38])
    tiny = torch.zeros(32)
    tiny[:3] = torch.tensor([2.0 ** -126, -(2.0 ** -128), 2.0 ** -127])
    sub = torch.zeros(32)
    sub[5] = 2.0 ** -133
    x = torch.stack(rows + [top, tiny, sub]).cuda()
    for t in (torch.float32, torch.bfloat16):
        codes, scales = moe.quant_mxfp4(x.to(t))
        rc, rs = plain64.quant_mxfp4(x.to(t))
        assert torch.equal(scales, rs) and torch.equal(codes, rc)
        assert torch.equal(moe.dequant_mxfp4(codes, scales, dtype=torch.float32).double(), plain64.mxfp4_values(rc, rs))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quant_not_finite_blocks_read_back_as_nan(moe, bad):
    x = torch.randn(4, 128, device="cuda", generator=_gen(1)).bfloat16()
    x[1, 40] = bad
    codes, scales = moe.quant_mxfp4(x)
    rc, rs = plain64.quant_mxfp4(x)
    assert torch.equal(codes, rc) and torch.equal(scales, rs)
    y = moe.dequant_mxfp4(codes, scales)
    hit = torch.zeros(4, 128, dtype=torch.bool, device="cuda")
    hit[1, 32:64] = True
    assert torch.equal(torch.isnan(y), hit)


def test_quant_leaves_what_lies_beside_its_outputs(moe):
    x = torch.randn(5, 96, device="cuda", generator=_gen(2)).bfloat16()
    codes = torch.full((7, 48), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((7, 3), 0xA5, dtype=torch.uint8, device="cuda")
    moe.mxfp4_quant_rows(x, codes[1:6], scales[1:6])
    assert (codes[[0, 6]] == 0xA5).all() and (scales[[0, 6]] == 0xA5).all()
    rc, rs = plain64.quant_mxfp4(x)
    assert torch.equal(codes[1:6], rc) and torch.equal(scales[1:6], rs)


def _operands(g, M, N, K, spread=4):
    a = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    b = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sa = torch.randint(127 - spread, 128 + spread, (M, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    sb = torch.randint(120 - spread, 121 + spread, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    return a, sa, b, sb


SHAPES = [(1, 1, 32), (1, 128, 32), (1, 4096, 4096), (2, 77, 96), (5, 1001, 2080), (8, 256, 1024), (9, 129, 4128),
          (16, 4096, 512), (17, 130, 160), (31, 64, 8192), (77, 1001, 2080), (127, 255, 224), (128, 128, 256),
          (129, 257, 288), (200, 3, 64), (300, 1, 4096), (512, 640, 4096), (1025, 513, 1056), (2433, 2299, 544), (4097, 2600, 288),
          (8, 4736, 64), (1, 4800, 352), (12, 2401, 96), (2500, 2300, 1024), (130, 70, 512)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(moe, M, N, K, dtype):
    a, sa, b, sb = _operands(_gen(M * 7 + N * 3 + K), M, N, K)
    got = moe.matmul_mxfp4(a, sa, b, sb, dtype=dtype)
    va, vb = plain64.mxfp4_values(a, sa), plain64.mxfp4_values(b, sb)
    ref = va @ vb.T
    assert got.dtype == dtype
    assert ((got.double() - ref).abs() <= plain64.matmul_tolerance(va, vb, ref, dtype)).all()


@pytest.mark.parametrize("M,N", [(3, 40), (50, 90), (2500, 2300)])
def test_matmul_scales_at_any_whole_word(moe, M, N):
    """Scales 4 bytes past a 16-byte boundary, which the wide loads do not take: the same product."""
    a, sa, b, sb = _operands(_gen(8), M, N, 512)
    want = moe.matmul_mxfp4(a, sa, b, sb)
    off = []
    for s in (sa, sb):
        buf = torch.full((s.numel() + 16,), 0xFF, dtype=torch.uint8, device="cuda")
        buf[4:4 + s.numel()] = s.flatten()
        off.append(buf[4:4 + s.numel()].view(s.shape))
    assert torch.equal(moe.matmul_mxfp4(a, off[0], b, sb), want)
    assert torch.equal(moe.matmul_mxfp4(a, sa, b, off[1]), want)


@pytest.mark.parametrize("M,N,K", [(1, 300, 256), (150, 300, 320)])
def test_matmul_ends_of_the_scale_range(moe, M, N, K):
    """Scales from 2^-127 on one side against large ones on the other; 255 (NaN) takes its row or column alone."""
    g = _gen(9)
    a, sa, b, sb = _operands(g, M, N, K)
    sa[:, :] = torch.randint(0, 3, sa.shape, generator=g, device="cuda", dtype=torch.uint8)
    sb[:, :] = torch.randint(200, 203, sb.shape, generator=g, device="cuda", dtype=torch.uint8)
    sb[4, 1] = 255
    if M > 1:
        sa[140, 2] = 255
    got = moe.matmul_mxfp4(a, sa, b, sb, dtype=torch.float32)
    va, vb = plain64.mxfp4_values(a, sa), plain64.mxfp4_values(b, sb)
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    nan[:, 4] = True
    if M > 1:
        nan[140] = True
    assert torch.equal(torch.isnan(got), nan)
    va, vb = torch.nan_to_num(va), torch.nan_to_num(vb)
    ref = va @ vb.T
    ok = (got.double() - ref).abs() <= plain64.matmul_tolerance(va, vb, ref, torch.float32)
    assert (ok | nan).all()


@pytest.mark.parametrize("M,N", [(1, 100), (100, 75)])
def test_matmul_leaves_what_lies_beside_its_output(moe, M, N):
    a, sa, b, sb = _operands(_gen(3), M, N, 256)
    buf = torch.full((M * N + 64,), 7.5, device="cuda")
    out = buf[32:32 + M * N].view(M, N)
    moe.mxfp4_matmul(a, sa, b, sb, out)
    assert (buf[:32] == 7.5).all() and (buf[32 + M * N:] == 7.5).all()
    va, vb = plain64.mxfp4_values(a, sa), plain64.mxfp4_values(b, sb)
    ref = va @ vb.T
    assert ((out.double() - ref).abs() <= plain64.matmul_tolerance(va, vb, ref, torch.float32)).all()


@pytest.mark.parametrize("M", [1, 12, 260, 8000])
def test_matmul_repeats_bit_for_bit_captured_and_on_another_stream(moe, M):
    a, sa, b, sb = _operands(_gen(4), M, 520, 2048)
    first = moe.matmul_mxfp4(a, sa, b, sb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(first)
    moe.mxfp4_matmul(a, sa, b, sb, out, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.mxfp4_matmul(a, sa, b, sb, out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)


def test_matmul_two_streams_at_once(moe):
    """Products that overlap, one of them with both operands the same rows."""
    a, sa, b, sb = _operands(_gen(7), 2304, 2560, 1024)
    sets = [((a, sa, b, sb), torch.cuda.Stream()), ((a, sa, a, sa), torch.cuda.Stream())]
    want = [moe.matmul_mxfp4(*ops, dtype=torch.float32) for ops, _ in sets]
    got = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for (ops, s), out in zip(sets, got):
            moe.matmul_mxfp4(*ops, out=out, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(got[1], got[1].T)
    assert moe.moe_last_device_status() == 0


@pytest.mark.parametrize("handle", [False, True])
def test_on_another_stream_everything_runs_there(moe, handle):
    """What the wrappers copy and allocate for a call on a stream does not wait for, or race with, the current one."""
    g = _gen(6)
    x = torch.randn(64, 8, 256, generator=g, device="cuda").bfloat16()
    w = torch.randn(96, 256, generator=g, device="cuda").bfloat16()
    qw, turned = moe.quant_mxfp4(w), x.transpose(0, 1)
    want = moe.quant_mxfp4(turned.contiguous())
    product = moe.matmul_mxfp4(want[0][0], want[1][0], *qw)
    values = moe.dequant_mxfp4(*want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    at = s.cuda_stream if handle else s
    torch.cuda._sleep(100_000_000)                       # the current stream is busy for some 50 ms
    c, e = moe.quant_mxfp4(turned, stream=at)
    y = moe.dequant_mxfp4(c, e, stream=at)
    p = moe.matmul_mxfp4(c[0], e[0], *qw, stream=at)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    c, e, y, p = (t.cpu() for t in (c, e, y, p))
    assert torch.equal(c, want[0].cpu()) and torch.equal(e, want[1].cpu())
    assert torch.equal(y, values.cpu()) and torch.equal(p, product.cpu())


def test_empty(moe):
    u8 = torch.uint8
    c, s = moe.quant_mxfp4(torch.empty(0, 64, device="cuda", dtype=torch.bfloat16))
    assert c.shape == (0, 32) and s.shape == (0, 2)
    assert moe.dequant_mxfp4(c, s).shape == (0, 64)
    w, ws = torch.zeros(5, 32, dtype=u8, device="cuda"), torch.zeros(5, 2, dtype=u8, device="cuda")
    assert moe.matmul_mxfp4(c, s, w, ws).shape == (0, 5)
    assert moe.matmul_mxfp4(w, ws, c, s).shape == (5, 0)


def test_quantized_linear_as_it_is_used(moe):
    """bf16 tokens and weights quantized and multiplied: the product of the quantized values, and near the product of
    the values themselves.  E2M1 at a scale within a factor 2 of the block's maximum is off by at most 1/4 of a value or
    a sixteenth of the block's maximum; over 1024 products of independent errors that leaves 0.2 of the norm."""
    g = _gen(5)
    x = torch.randn(33, 1024, generator=g, device="cuda").bfloat16()
    w = torch.randn(200, 1024, generator=g, device="cuda").bfloat16()
    qx, qw = moe.quant_mxfp4(x), moe.quant_mxfp4(w)
    got = moe.matmul_mxfp4(*qx, *qw).double()
    va, vb = plain64.mxfp4_values(*qx), plain64.mxfp4_values(*qw)
    ref = va @ vb.T
    assert ((got - ref).abs() <= plain64.matmul_tolerance(va, vb, ref, torch.bfloat16)).all()
    full = x.double() @ w.double().T
    assert torch.linalg.norm(got - full) <= 0.2 * torch.linalg.norm(full)


@pytest.mark.parametrize("K,stride,off", [(33, None, 0), (48, None, 0)])
def test_quant_refuses_columns_that_are_not_whole_blocks(moe, K, stride, off):
    with pytest.raises(ValueError):
        moe.quant_mxfp4(torch.zeros(2, K, device="cuda", dtype=torch.bfloat16))


def test_refusals(moe):
    x = torch.zeros(4, 72, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError):
        moe.quant_mxfp4(torch.zeros(4, 65, device="cuda", dtype=torch.bfloat16)[:, :64])      # 130-byte rows
    with pytest.raises(moe.MoeError):
        moe.quant_mxfp4(torch.zeros(4 * 72 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(4, 72)[:, :64])
    with pytest.raises(ValueError):
        moe.mxfp4_quant_rows(x[:, :64].t(), *moe.quant_mxfp4(x[:, :64]))                      # columns apart
    with pytest.raises(ValueError):
        moe.quant_mxfp4(x[:, :64].double())
    c, s = moe.quant_mxfp4(x[:, :64])
    with pytest.raises(ValueError):
        moe.mxfp4_quant_rows(x[:, :64], c[:3], s)
    with pytest.raises(ValueError):
        moe.mxfp4_dequant_rows(c, s[:, :1], torch.zeros(4, 64, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.dequant_mxfp4(c, s, dtype=torch.float16)                                          # would overflow
    with pytest.raises(ValueError):
        moe.matmul_mxfp4(c, s, c[:, :16].contiguous(), s)
    with pytest.raises(moe.MoeError):
        moe.matmul_mxfp4(c, s, c, s, dtype=torch.float16)
