"""The block-scaled layer and the permutation over the ranges that their kernels' branches depend on: pairs beyond
what the permutation keeps in registers, expert counts of each width of its ballots, more than 8 experts a token,
rows of several column blocks, both orientations, whole-layer calls on CTA pairs, replay from a CUDA graph, and a
workspace that held anything.  Tolerances are those of the layer's own tests.
"""
import numpy as np
import pytest
import torch

from test_gpu_block_fp8 import check, experts_reference, make_experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


def layer(moe, c, **kw):
    return moe.moe_forward_routed(c["x"], c["tw"], c["ids"], c["w13"], c["w2"], c["s13"], c["s2"],
                                  w_format="e4m3_block", **kw)


# ---- permutation -----------------------------------------------------------------------------------


def align_reference(ids, E, block):
    """(sorted pairs, expert of each block, pairs of each expert), ids out of range left out."""
    flat = ids.reshape(-1)
    kept = np.nonzero((flat >= 0) & (flat < E))[0]
    count = np.bincount(flat[kept], minlength=E)
    order = kept[np.argsort(flat[kept], kind="stable")]
    pad = -(-count // block) * block
    sorted_ids = np.full(pad.sum(), flat.size, np.int64)
    at, start = 0, np.cumsum(pad) - pad
    for e in np.nonzero(count)[0]:
        sorted_ids[start[e] : start[e] + count[e]] = order[at : at + count[e]]
        at += count[e]
    return sorted_ids, np.repeat(np.arange(E), pad // block), count


@pytest.mark.parametrize("T,k,E,block,skew", [
    (8192, 8, 64, 128, False), (8193, 8, 64, 128, False),  # 65536 pairs and just above
    (20001, 9, 200, 16, False), (70000, 3, 511, 64, True), (9001, 17, 1000, 128, True), (16400, 4, 127, 1, False),
    (257, 4, 128, 16, False), (1025, 1, 512, 128, False), (3000, 2, 1024, 16, True)])
def test_permutation_of_many_pairs(moe, T, k, E, block, skew):
    g = torch.Generator().manual_seed(T + E)
    u = torch.rand(T, k, generator=g)
    ids = ((u ** 4 if skew else u) * E).to(torch.int32).clamp_(max=E - 1)
    ids[T // 3, 0], ids[T - 1, k - 1] = E, -1
    sorted_ids, experts, npp, counts = moe.moe_align(ids.cuda(), E, block)
    assert moe.moe_get_status() == moe.MOE_ERR_DEVICE_INDEX
    rs, re, rc = align_reference(ids.numpy(), E, block)
    assert int(npp) == len(rs)
    assert np.array_equal(sorted_ids.cpu().numpy()[: len(rs)], rs)
    assert np.array_equal(experts.cpu().numpy()[: len(re)], re)
    assert np.array_equal(counts.cpu().numpy(), rc)


def test_permutation_of_an_empty_batch(moe):
    junk = torch.full((4096,), 7, dtype=torch.int32, device="cuda")  # (what new memory would hold)
    del junk
    _, _, npp, counts = moe.moe_align(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 1024, 16)
    assert int(npp) == 0 and (counts == 0).all()


# ---- expert layer ----------------------------------------------------------------------------------

LAYERS = [
    # T, H, I, E, k
    (70, 256, 128, 24, 9), (130, 256, 256, 20, 17), (300, 256, 128, 33, 32),  # more than 8 experts a token
    (66, 2176, 128, 6, 3), (100, 4096, 128, 5, 2), (65, 2176, 256, 12, 9),    # rows of several column blocks
    (40, 256, 128, 130, 8), (200, 256, 128, 130, 8), (90, 128, 128, 300, 10), (2000, 128, 128, 300, 6),
    (700, 128, 128, 600, 4), (1, 7168, 256, 5, 4), (64, 7168, 128, 4, 2),
]


@pytest.mark.parametrize("orientation", [1, 2])
@pytest.mark.parametrize("T,H,I,E,k", LAYERS)
def test_experts_over_the_range(moe, T, H, I, E, k, orientation):
    d = make_experts(T, H, I, E, k, torch.Generator().manual_seed(T + H + E))
    c = {n: v.cuda() for n, v in d.items()}
    out = layer(moe, c, options={"orientation": orientation})
    assert moe.moe_get_status() == 0
    check(out, experts_reference(d), f"experts {T}x{H}x{I} E{E} k{k}")
    assert torch.equal(out, layer(moe, c, options={"orientation": orientation}))


@pytest.mark.parametrize("T,E,k", [(300, 8, 2), (90, 64, 4)])
def test_whole_layer_calls_beyond_64_tokens(moe, T, E, k):
    """CTA pairs (300 tokens) and swap-AB with bf16 rows (90), through every entry point of the layer."""
    d = make_experts(T, 256, 256, E, k, torch.Generator().manual_seed(T))
    c = {n: v.cuda() for n, v in d.items()}
    wr = (torch.randn(E, 256, generator=torch.Generator().manual_seed(1)) / 16).to(torch.bfloat16).cuda()
    _, c["tw"], c["ids"] = moe.moe_route(c["x"], wr, k, True)
    ref = layer(moe, c)
    args = (wr, c["w13"], c["w2"], k, True, c["s13"], c["s2"])
    assert torch.equal(moe.moe_forward(c["x"], *args, w_format="e4m3_block"), ref)
    assert torch.equal(moe.moe_forward_noalloc(c["x"], *args, w_format="e4m3_block"), ref)
    host = moe.moe_forward_host(d["x"].pin_memory(), *args, w_format="e4m3_block")
    torch.cuda.synchronize()
    assert torch.equal(host, ref.cpu()) and moe.moe_get_status() == 0
    check(ref, experts_reference(dict(d, tw=c["tw"].cpu(), ids=c["ids"].cpu())), f"T={T}")


@pytest.mark.parametrize("T", [2, 20, 48, 90, 400])
def test_workspace_contents_do_not_matter(moe, T):
    d = make_experts(T, 384, 256, 16, 3, torch.Generator().manual_seed(T))
    c = {n: v.cuda() for n, v in d.items()}
    need = moe.moe_workspace_size(T, 384, 256, 16, 3, moe.MOE_BF16, moe.MOE_E4M3_B128)
    outs = []
    for fill in (0x00, 0xFF, 0x7F, 0xA5):  # zeros, NaN patterns, large values, garbage
        buf = torch.full((T * 384 + 4096,), float("nan"), dtype=torch.bfloat16, device="cuda")
        out = layer(moe, c, out=buf[: T * 384].view(T, 384),
                    workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
        assert moe.moe_get_status() == 0
        assert torch.isfinite(out).all() and torch.isnan(buf[T * 384 :]).all()
        outs.append(out.clone())
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("T", [1, 40, 90, 300])
def test_replay_from_a_graph(moe, T):
    """Routing, experts and the shared expert's four calls captured once, replayed on other inputs."""
    H, I, E, k = 512, 256, 32, 4
    g = torch.Generator().manual_seed(T)
    d = make_experts(T, H, I, E, k, g)
    c = {n: v.cuda() for n, v in d.items()}
    wr = (torch.randn(E, H, generator=g) / 16).to(torch.bfloat16).cuda()
    bias = (torch.randn(E, generator=g) * 0.05).cuda()
    a13, a2 = (c["w13"][0], c["s13"][0]), (c["w2"][0], c["s2"][0])

    def step():
        logits, tw, ids = moe.moe_route_grouped(c["x"], wr, k, bias=bias, n_group=8, topk_group=4, scale=2.5)
        y = layer(moe, dict(c, tw=tw, ids=ids))
        q, s = moe.moe_quant_block(c["x"])
        q, s = moe.moe_silu_quant_block(moe.moe_gemm_block(q, s, *a13))
        return logits, ids, tw, y, moe.moe_gemm_block(q, s, *a2, out_dtype=torch.float32)

    step()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        captured = step()
    for seed in (1, 2):
        c["x"].copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in captured]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
    assert moe.moe_get_status() == 0
