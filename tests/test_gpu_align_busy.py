"""Permutations of long batches, whose one kernel is a cluster of 16 CTAs, while another stream holds the SMs."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


@pytest.mark.parametrize("T,k,E", [(2048, 8, 64), (8192, 8, 256), (16385, 8, 40)])
def test_beside_a_busy_stream(moe, T, k, E):
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn(T, 136, generator=g, device="cuda")
    rows = torch.zeros(moe.moe_align_capacity(T, k, E, 64)[0], 136, device="cuda")
    ref = moe.moe_permute(x, ids, E, 64, rows=rows.clone())
    h, w = torch.randn(32768, 4096, generator=g, device="cuda").to(torch.bfloat16), torch.ones(4096, device="cuda")
    big = torch.randn(4096, 4096, generator=g, device="cuda").to(torch.bfloat16)
    moe.moe_get_status()  # (ids of -1 are flagged)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        moe.moe_prenorm(h, w)  # (CTAs that fill the SMs, and those of a library product)
        torch.matmul(big, big)
        with torch.cuda.stream(side):
            got.append(moe.moe_permute(x, ids, E, 64, rows=rows.clone()))
    torch.cuda.synchronize()
    n = int(ref.num_post_pad)
    for p in got:
        assert int(p.num_post_pad) == n and torch.equal(p.row_of, ref.row_of)
        assert torch.equal(p.expert_counts, ref.expert_counts) and torch.equal(p.rows, ref.rows)
        assert torch.equal(p.sorted_ids[:n], ref.sorted_ids[:n]) and torch.equal(p.expert_ids[: n // 64], ref.expert_ids[: n // 64])
    assert moe.moe_get_status() == moe.MOE_ERR_DEVICE_INDEX
