"""Host side of the block-scaled operators and of the calls beside them: what the plan says, and which arguments
are taken (no call below reaches the device)."""
import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__

    __graft_entry__._builder().build()
    import mixture_experts_layer_scan_gb300 as m

    return m


@pytest.mark.parametrize("T,k,options,launches", [
    (1, 8, None, 6), (4, 8, None, 6), (16, 2, None, 6),           # sorted and quantised by one launch
    (5, 8, None, 7), (17, 2, None, 7), (64, 8, None, 7), (4096, 8, None, 7),
    (4, 8, {"orientation": 2}, 7)])                               # CTA pairs: two launches at every size
def test_plan_counts_the_launches_of_a_block_scaled_layer(moe, T, k, options, launches):
    """router, top-k, permutation, quantisation, two products and the combine."""
    p = moe.moe_plan_info(T, 2048, 768, 128, k, moe.MOE_BF16, moe.MOE_E4M3_B128, options)
    assert p["kernel_launches"] == launches


class Recorder:
    """Stands in for the library: keeps the arguments of each call and answers 0."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0

        return call


@pytest.fixture
def recorded(moe, monkeypatch):
    r = Recorder()
    monkeypatch.setattr(moe, "_lib", r)
    return r


def test_routings_of_other_shapes(moe, recorded):
    """What counts is the memory: T x k values in front, in a flat topk_w and in buffers of a larger batch too."""
    T, H, I, E, k = 5, 256, 128, 4, 2
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    w13, w2 = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16), torch.zeros(E, H, I, dtype=torch.bfloat16)
    ws = torch.empty(16, dtype=torch.uint8)
    ids, big = torch.zeros(T, k, dtype=torch.int32), torch.zeros(64, k, dtype=torch.int32)
    for tw, ti in ((torch.zeros(T, k), ids), (torch.zeros(T * k), ids), (torch.zeros(64, k), big),
                   (torch.zeros(T, k, 1), big), (torch.zeros(T * k), big)):
        moe.moe_forward_routed(x, tw, ti, w13, w2, workspace=ws, stream=0)
        name, args = recorded.calls.pop()
        assert name == "moe_forward_routed" and args[1:3] == (tw.data_ptr(), ti.data_ptr()) and args[5:10] == (T, H, I, E, k)
    for tw, ti in ((torch.zeros(T, k - 1), ids), (torch.zeros(T - 1, k), ids), (torch.zeros(T, k), ids[:4]),
                   (torch.zeros(T, k, dtype=torch.float64), ids), (torch.zeros(T, k), ids.long())):
        with pytest.raises(ValueError):
            moe.moe_forward_routed(x, tw, ti, w13, w2, workspace=ws, stream=0)
    assert not recorded.calls


def test_names_of_weight_formats(moe, recorded):
    """A name of the weights' own type says nothing new; an unknown name is refused, not guessed."""
    T, H, I, E, k = 3, 256, 128, 4, 2
    x, wr = torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(E, H, dtype=torch.bfloat16)
    ws = torch.empty(16, dtype=torch.uint8)
    for dtype, code in ((torch.bfloat16, moe.MOE_BF16), (torch.float8_e4m3fn, moe.MOE_E4M3)):
        w13, w2 = torch.zeros(E, 2 * I, H, dtype=dtype), torch.zeros(E, H, I, dtype=dtype)
        for name in (None, "", "bf16", "e4m3", "fp8"):
            moe.moe_forward(x, wr, w13, w2, k, True, workspace=ws, stream=0, w_format=name)
            args = [a for n, a in recorded.calls if n == "moe_forward"]
            assert args and args[-1][11] == code
            moe.moe_forward_noalloc(x, wr, w13, w2, k, True, stream=0, w_format=name)
            args = [a for n, a in recorded.calls if n == "moe_forward_noalloc"]
            assert args and args[-1][11] == code
        for name in ("int8", "e4m3-block", "E4M3_BLOCK"):
            with pytest.raises(ValueError):
                moe.moe_forward(x, wr, w13, w2, k, True, workspace=ws, stream=0, w_format=name)


def test_a_routing_rule_is_its_values(moe, recorded):
    """The scale may come as a tensor or an array: what it holds at the call counts, not what it held before."""
    logits = torch.zeros(2, 8)
    scale = torch.tensor(2.5)
    seen = []
    for value in (2.5, 1.0, 16.0):
        scale.fill_(value)
        for s in (scale, scale.numpy()):
            moe.moe_topk_grouped(logits, 2, n_group=4, topk_group=torch.tensor(2), scale=s, stream=0)
            rule = recorded.calls[-1][1][5]._obj
            seen.append((rule.scale, rule.n_group, rule.topk_group, rule.score))
    assert seen == [(v, 4, 2, 1) for v in (2.5, 2.5, 1.0, 1.0, 16.0, 16.0)]
    with pytest.raises(ValueError):
        moe.moe_topk_grouped(logits, 2, score="tanh", stream=0)


@pytest.mark.parametrize("size", [2 ** 31 - 2 ** 24, 2 ** 31 - 16])
def test_dimensions_whose_counts_pass_32_bits(moe, size):
    """The last rows or columns below 2^31 would round up past it: refused before anything is launched."""
    lib, at = moe.lib(), 0x1000
    assert lib.moe_gemm_block(at, at, at, at, size, 128, 16, moe.MOE_BF16, at, None) == moe.MOE_ERR_ARG
    assert lib.moe_gemm_block(at, at, at, at, 4, size, 16, moe.MOE_BF16, at, None) == moe.MOE_ERR_ARG
    assert lib.moe_gemm_block(at, at, at, at, 4, 128, size, moe.MOE_BF16, at, None) == moe.MOE_ERR_ARG
    for f in (lib.moe_quant_block, lib.moe_silu_quant_block):
        assert f(at, 1, size, moe.MOE_BF16, at, at, None) == moe.MOE_ERR_ARG
