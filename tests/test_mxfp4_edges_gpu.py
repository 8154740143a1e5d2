"""MXFP4 rows in tensors of other ranks than two, empty ones among them, and the product by pairs of CTAs."""
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


@pytest.mark.parametrize("lead", [(), (3,), (0,), (0, 5), (5, 0), (2, 3), (2, 0, 3), (2, 1, 3), (1, 1, 1, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_any_rank(moe, lead, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(1 + len(lead))
    x = torch.randn(*lead, 96, generator=g, device="cuda").to(dtype)
    codes, scales = moe.quant_mxfp4(x)
    assert codes.shape == (*lead, 48) and scales.shape == (*lead, 3)
    y = moe.dequant_mxfp4(codes, scales, dtype=dtype)
    assert y.shape == x.shape and y.dtype == dtype
    if x.numel():
        rc, rs = plain64.quant_mxfp4(x)
        assert torch.equal(codes, rc) and torch.equal(scales, rs)
        assert torch.equal(y.double(), plain64.mxfp4_values(rc, rs))


def test_no_experts_make_no_layer_rows(moe):
    w = torch.empty(0, 128, 256, device="cuda", dtype=torch.bfloat16)
    assert moe.quant_mxfp4(w)[0].shape == (0, 128, 128)


@pytest.mark.parametrize("shape", [(2, 3, 2), (3, 2, 3), (6, 3), (2, 3, 4)])
def test_scales_of_other_rows_are_refused(moe, shape):
    codes, _ = moe.quant_mxfp4(torch.zeros(2, 3, 96, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        moe.dequant_mxfp4(codes, torch.full(shape, 127, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("M,N,K,dtype", [(2304, 2560, 512, torch.bfloat16), (2500, 2300, 1056, torch.float32), (4097, 2600, 288, torch.bfloat16)])
def test_pairs_of_ctas_repeat_bit_for_bit(moe, M, N, K, dtype):
    """Sizes that pairs of CTAs compute (with the scales by TMA and by loads), many products of changing operands in a
    row: what the second CTA hands to the first is there before it is used."""
    g = torch.Generator(device="cuda")
    g.manual_seed(M)

    def rows(R):
        return (torch.randint(0, 256, (R, K // 2), generator=g, device="cuda", dtype=torch.uint8),
                torch.randint(118, 123, (R, K // 32), generator=g, device="cuda", dtype=torch.uint8))

    sets = [(rows(M), rows(N)) for _ in range(3)]
    want = []
    for (a, sa), (b, sb) in sets:
        va, vb = plain64.mxfp4_values(a, sa), plain64.mxfp4_values(b, sb)
        ref = va @ vb.T
        want.append(moe.matmul_mxfp4(a, sa, b, sb, dtype=dtype))
        assert ((want[-1].double() - ref).abs() <= plain64.matmul_tolerance(va, vb, ref, dtype)).all()
    outs = [torch.empty_like(want[0]) for _ in range(3)]
    for _ in range(50):
        for ((a, sa), (b, sb)), out, first in zip(sets, outs, want):
            moe.matmul_mxfp4(a, sa, b, sb, out=out)
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert moe.moe_last_device_status() == 0
