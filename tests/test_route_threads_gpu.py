"""Routing from two host threads at once, with expert counts whose permutations take different amounts of shared memory."""
import threading

import pytest
import torch

from conftest import cuda_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not cuda_ok():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("T", [4, 1100])
def test_two_threads(T):
    """T = 4 is permuted by one CTA, T = 1100 (k = 4) by one for each 1024 pairs."""
    import bit_quantized_moe_token_b200 as moe
    call, k = moe.lib().moe_route_topk, 4
    statuses, sets, threads = [], [], []

    def loop(args):
        torch.cuda.set_device(0)
        statuses.append({call(*args) for _ in range(10000)})

    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    for E in (512, 1024):
        lg = torch.randn(T, E, generator=g, device="cuda")
        ids, rows = (torch.empty(T * k, dtype=torch.int32, device="cuda") for _ in range(2))
        gates, sorted_pairs = torch.empty(T * k, device="cuda"), torch.empty_like(rows)
        offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        ws = torch.empty(moe.moe_route_workspace_bytes(T, E, k) + 256, dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        sets.append((lg, ids, rows, gates, sorted_pairs, offsets, ws, stream))
        args = (lg.data_ptr(), T, E, k, ids.data_ptr(), gates.data_ptr(), offsets.data_ptr(), sorted_pairs.data_ptr(),
                rows.data_ptr(), ws.data_ptr(), ws.numel(), stream.cuda_stream)
        assert call(*args) == moe.MOE_OK
        threads.append(threading.Thread(target=loop, args=(args,)))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert statuses == [{moe.MOE_OK}, {moe.MOE_OK}]
    for lg, ids, rows, gates, sorted_pairs, offsets, *_ in sets:
        want = lg.topk(k, dim=1).indices.flatten()
        assert torch.equal(ids.long(), want)
        assert torch.equal(sorted_pairs.long(), want.sort(stable=True).indices)
        assert torch.equal(rows[sorted_pairs.long()].long(), torch.arange(T * k, device="cuda"))
        assert offsets[-1] == T * k


def test_router_weights_of_two_widths():
    """The router's logits from two threads, H = 2048 and 4096: 64 and 128 KB of tokens in shared memory."""
    import bit_quantized_moe_token_b200 as moe
    call = moe.lib().moe_router_logits
    statuses, sets, threads = [], [], []

    def loop(args):
        torch.cuda.set_device(0)
        statuses.append({call(*args) for _ in range(5000)})

    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for H in (2048, 4096):
        x, wr = ((torch.randn(n, H, generator=g, device="cuda")).bfloat16() for n in (40, 60))
        out = torch.empty(40, 60, device="cuda")
        stream = torch.cuda.Stream()
        sets.append((x, wr, out, stream))
        threads.append(threading.Thread(target=loop, args=((x.data_ptr(), wr.data_ptr(), 40, H, 60, out.data_ptr(), stream.cuda_stream),)))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert statuses == [{moe.MOE_OK}, {moe.MOE_OK}]
    for x, wr, out, _ in sets:
        ref = x.double() @ wr.double().T
        # an fp32 sum of H terms in any order
        assert ((out.double() - ref).abs() <= x.shape[1] * 2.0 ** -24 * (x.double().abs() @ wr.double().abs().T)).all()
