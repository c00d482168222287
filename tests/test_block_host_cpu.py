"""Host side of the block-scaled operators and of the calls beside them: what the plan says, and which arguments
are taken (no call below reaches the device)."""
import pytest


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
