"""Calls on a stream beside the current one: what a call allocates for itself is not handed to the current stream's
next tensors while the call runs, and a call does no work on the current stream.

Each call waits on its stream behind a long sleep.  Its result is dropped, tensors of the same sizes are made and
filled on the current stream, and after everything has run their values must still be there.
"""
import pytest
import torch

from test_gpu_block_fp8 import make_experts

pytestmark = pytest.mark.gpu

SLEEP = 100_000_000  # cycles: about 50 ms


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


@pytest.fixture(scope="module")
def calls(moe):
    """name -> (call(stream), outputs' and workspace's sizes in bytes)"""
    T, H, I, E, k = 200, 512, 256, 8, 2
    d = make_experts(T, H, I, E, k, torch.Generator().manual_seed(0))
    c = {n: v.cuda() for n, v in d.items()}
    wr = (torch.randn(E, H, generator=torch.Generator().manual_seed(1)) / 16).to(torch.bfloat16).cuda()
    logits, _, _ = moe.moe_route(c["x"], wr, k, True)
    q, s = moe.moe_quant_block(c["x"])
    gu = torch.randn(T, 2 * I, device="cuda")
    need = moe.moe_workspace_size(T, H, I, E, k, moe.MOE_BF16, moe.MOE_E4M3_B128)
    w = (c["w13"], c["w2"])
    sc = (c["s13"], c["s2"])
    torch.cuda.synchronize()
    return {
        "topk": (lambda st: moe.moe_topk_grouped(logits, k, stream=st), [T * k * 4, T * k * 4]),
        "route": (lambda st: moe.moe_route_grouped(c["x"], wr, k, stream=st), [T * E * 4, T * k * 4, T * k * 4]),
        "quant": (lambda st: moe.moe_quant_block(c["x"], stream=st), [T * H, T * H // 32]),
        "silu_quant": (lambda st: moe.moe_silu_quant_block(gu, stream=st), [T * I, T * I // 32]),
        "gemm": (lambda st: moe.moe_gemm_block(q, s, c["w13"][0], c["s13"][0], stream=st), [T * 2 * I * 2]),
        "align": (lambda st: moe.moe_align(c["ids"], E, 16, stream=st), [(T * k + E * 15) * 4, 16, E * 4]),
        "routed": (lambda st: moe.moe_forward_routed(c["x"], c["tw"], c["ids"], *w, *sc, w_format="e4m3_block", stream=st),
                   [need, T * H * 2]),
        "forward": (lambda st: moe.moe_forward(c["x"], wr, *w, k, True, *sc, w_format="e4m3_block", stream=st),
                    [need, T * H * 2]),
    }


def tensors(out):
    return [out] if isinstance(out, torch.Tensor) else list(out)


NAMES = ["topk", "route", "quant", "silu_quant", "gemm", "align", "routed", "forward"]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_another_stream(moe, calls, name, handle):
    call, sizes = calls[name]
    side = torch.cuda.Stream()
    call(side)  # (first launches of a kernel load it)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    call(side.cuda_stream if handle else side)  # its tensors are dropped while it waits
    fresh = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert moe.moe_get_status() == 0
    assert all(bool((t == 0x5A).all()) for t in fresh)


@pytest.mark.parametrize("name", NAMES)
def test_result_on_another_stream(moe, calls, name):
    call, _ = calls[name]
    ref = [t.clone() for t in tensors(call(None))]
    side = torch.cuda.Stream()
    torch.cuda._sleep(SLEEP)  # the current stream is busy: nothing of the call may wait there or run late
    out = tensors(call(side))
    side.synchronize()
    with torch.cuda.stream(side):
        got = [t.clone() for t in out]
        if name == "align":  # (capacities: entries behind the padded length are not written)
            n = int(ref[2])
            ref[0], got[0], ref[1], got[1] = ref[0][:n], got[0][:n], ref[1][: n // 16], got[1][: n // 16]
        same = [torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(ref, got)]
    torch.cuda.synchronize()
    assert all(same)
    after = [t.clone() for t in out]  # (the current stream's late work, if there were any, is done)
    assert all(torch.equal(a.view(torch.uint8)[: len(b.view(torch.uint8))], b.view(torch.uint8)) for a, b in zip(after, got))
