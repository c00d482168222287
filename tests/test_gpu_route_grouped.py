"""Grouped routing (moe_topk_grouped, moe_route_grouped) against a plain 64-bit form.

Expert ids are compared exactly on the rows whose ranking does not hang on the last bits of a
32-bit score: every gap that decides (between the kept and the next group, and between consecutive
chosen experts) is over 1e-5 of the row's largest |score + bias|, some hundred times the error of
a 32-bit score (a few 2^-24).  Weights are within 1e-5: exp and the division err by a few 2^-23,
the sums of up to 1024 terms by far less than 64 of them.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


def reference(logits, bias, k, score, n_group, topk_group, group_sum, renorm, scale):
    """(weights, ids, clear): plain loops over numpy float64; clear marks the rows with wide gaps."""
    T, E = logits.shape
    gs = E // n_group
    w, ids, clear = np.zeros((T, k)), np.zeros((T, k), np.int64), np.ones(T, bool)
    for t in range(T):
        l = logits[t].astype(np.float64)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-l))
        else:
            s = np.exp(l - l.max())
            s /= s.sum()
        r = s if bias is None else s + bias.astype(np.float64)
        far = 1e-5 * np.abs(r[np.isfinite(r)]).max()
        groups = []
        for g in range(n_group):
            top = sorted(r[g * gs : (g + 1) * gs], reverse=True)
            groups.append(sum(top[:group_sum]))
        order = sorted(range(n_group), key=lambda g: (-groups[g], g))
        kept = order[:topk_group]
        if topk_group < n_group:
            clear[t] &= groups[order[topk_group - 1]] - groups[order[topk_group]] > far
        cand = [e for g in kept for e in range(g * gs, (g + 1) * gs)]
        cand.sort(key=lambda e: (-r[e], e))
        for a, b in zip(cand[:k], cand[1 : k + 1]):
            clear[t] &= r[a] - r[b] > far
        ids[t] = cand[:k]
        w[t] = s[ids[t]]
        if renorm:
            w[t] /= w[t].sum()
    return w * scale, ids, clear


RULES = [
    # T, E, k, groups, kept, group_sum, score, bias, renorm, scale
    (1, 256, 8, 8, 4, 2, "sigmoid", True, True, 2.5),
    (301, 256, 8, 8, 4, 2, "sigmoid", True, True, 2.5),
    (65, 160, 6, 8, 3, 1, "softmax", False, False, 16.0),
    (33, 160, 6, 8, 3, 2, "softmax", False, True, 1.0),     # summed group scores: ranks the scores, not the logits
    (33, 72, 5, 6, 2, 2, "sigmoid", True, False, 1.0),      # six groups: five lanes a group, two lanes idle
    (40, 96, 4, 3, 2, 2, "softmax", True, True, 1.0),       # eight lanes a group, eight idle
    (17, 64, 64 // 2, 1, 1, 1, "sigmoid", False, True, 1.0),  # 32 of 64, no groups
    (9, 1024, 8, 1, 1, 1, "softmax", False, True, 1.0),     # 32 experts in a lane
    (9, 1020, 8, 17, 5, 2, "sigmoid", True, True, 1.0),     # one lane a group, 60 experts in it
    (9, 1024, 32, 32, 32, 2, "sigmoid", True, True, 1.0),   # every group kept
    (12, 32, 3, 32, 7, 2, "sigmoid", True, True, 1.0),      # groups of one expert
    (5, 1, 1, 1, 1, 1, "sigmoid", False, True, 1.0),        # a single expert
    (6, 7, 7, 7, 7, 1, "softmax", False, False, 1.0),       # all experts chosen
    (8, 8, 2, 2, 1, 2, "sigmoid", True, True, 0.0),         # a scale of zero
]


@pytest.mark.parametrize("T,E,k,g,kept,gsum,score,bias,renorm,scale", RULES)
def test_against_64_bits(moe, T, E, k, g, kept, gsum, score, bias, renorm, scale):
    gen = torch.Generator().manual_seed(E * 7 + T)
    logits = torch.randn(T, E, generator=gen) * 1.5
    b = torch.randn(E, generator=gen) * (0.1 if score == "sigmoid" else 0.1 / E) if bias else None
    w, ids = moe.moe_topk_grouped(logits.cuda(), k, bias=None if b is None else b.cuda(), score=score, n_group=g,
                                  topk_group=kept, group_sum=gsum, renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    assert moe.moe_get_status() == 0
    rw, rid, clear = reference(logits.numpy(), None if b is None else b.numpy(), k, score, g, kept, gsum, renorm, scale)
    assert clear.mean() >= 0.5  # (of the inputs alone: most rows are compared)
    assert np.array_equal(ids.cpu().numpy()[clear], rid[clear])
    assert np.allclose(w.cpu().numpy()[clear], rw[clear], rtol=1e-5, atol=1e-30)


def test_equal_scores_take_the_lower_group_and_expert(moe):
    logits = torch.zeros(3, 64, device="cuda")
    logits[1, 40:] = 1.0   # groups 5, 6, 7 tie above the rest
    logits[2, 63] = 2.0
    for score in ("sigmoid", "softmax"):
        _, ids = moe.moe_topk_grouped(logits, 6, score=score, n_group=8, topk_group=2, group_sum=1)
        assert ids.cpu().tolist() == [[0, 1, 2, 3, 4, 5], [40, 41, 42, 43, 44, 45], [63, 0, 1, 2, 3, 4]]
    # -0 and +0 are equal
    z = torch.tensor([[-0.0, 0.0, -0.0, 0.0]], device="cuda")
    _, ids = moe.moe_topk_grouped(z, 4, score="softmax")
    assert ids.cpu().tolist() == [[0, 1, 2, 3]]


def test_masked_experts_infinities_and_nan(moe):
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(torch.float32).min
    bias = torch.zeros(8, device="cuda")
    bias[[0, 1, 6]] = torch.tensor([-inf, -inf, low], device="cuda")
    logits = torch.arange(8, dtype=torch.float32, device="cuda").flip(0).repeat(4, 1) / 8
    logits[1, 3] = nan
    logits[2, 5] = inf
    logits[3, :] = -inf
    w, ids = moe.moe_topk_grouped(logits, 8, bias=bias, score="sigmoid", renorm=False)
    # the masked ones come last: the type's lowest value before -inf and NaN, those by index
    assert ids.cpu().tolist() == [[2, 3, 4, 5, 7, 6, 0, 1], [2, 4, 5, 7, 6, 0, 1, 3], [5, 2, 3, 4, 7, 6, 0, 1],
                                  [2, 3, 4, 5, 7, 6, 0, 1]]
    w = w.cpu().numpy()
    assert np.isnan(w[1, 7]) and np.isfinite(w[1, :7]).all()
    assert w[2, 0] == 1.0 and (w[3] == 0).all()
    # a row without any score: weights 0 after the renormalisation, not NaN
    w, _ = moe.moe_topk_grouped(logits[3:], 4, score="sigmoid", renorm=True)
    assert (w.cpu() == 0).all()
    # a mask that leaves no expert in any group
    _, ids = moe.moe_topk_grouped(logits[:1].contiguous(), 4, bias=torch.full((8,), -inf, device="cuda"), n_group=4,
                                  topk_group=2)
    assert ids.cpu().tolist() == [[0, 1, 2, 3]]


@pytest.mark.parametrize("T,E,k", [(77, 128, 8), (5, 300, 4)])
def test_no_groups_softmax_is_the_plain_router(moe, T, E, k):
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(3)).cuda()
    logits[0] -= 200 * torch.rand(E, generator=torch.Generator().manual_seed(4)).cuda()  # scores that underflow
    w0, i0 = moe.moe_topk_from_logits(logits, k, True)
    w1, i1 = moe.moe_topk_grouped(logits, k, score="softmax", renorm=True)
    assert torch.equal(i0, i1)
    assert torch.allclose(w0, w1, rtol=1e-5, atol=1e-30)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_route_grouped_is_logits_then_ranking(moe, dtype, T):
    gen = torch.Generator().manual_seed(T)
    x, wr = torch.randn(T, 512, generator=gen).to(dtype).cuda(), torch.randn(64, 512, generator=gen).to(dtype).cuda() / 22
    b = (torch.randn(64, generator=gen) * 0.1).cuda()
    rule = dict(score="sigmoid", n_group=8, topk_group=3, group_sum=2, renorm=True, scale=2.5)
    logits, w, ids = moe.moe_route_grouped(x, wr, 6, bias=b, **rule)
    base, _, _ = moe.moe_route(x, wr, 6, True)
    assert torch.equal(logits, base)
    w2, i2 = moe.moe_topk_grouped(logits, 6, bias=b, **rule)
    assert torch.equal(w, w2) and torch.equal(ids, i2)


def test_empty_batch_and_other_stream(moe):
    w, ids = moe.moe_topk_grouped(torch.empty(0, 64, device="cuda"), 4)
    assert w.shape == (0, 4) and ids.shape == (0, 4)
    logits = torch.randn(50, 64, generator=torch.Generator().manual_seed(1)).cuda()
    ref = moe.moe_topk_grouped(logits, 4, n_group=8, topk_group=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_topk_grouped(logits, 4, n_group=8, topk_group=4, stream=side)
    side.synchronize()
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
