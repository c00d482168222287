"""A caller's routing that names an expert several times for a token.

Up to T pairs of an expert, rounded up to a multiple of 16, every form computes them all.  Past that the swap-AB
forms whose tile holds all of an expert's tokens drop and flag the pairs that come last; a block-scaled layer and
the token-major forms compute them.  References replace repeated experts by others with the same weights (and
dropped pairs' routing weight by 0), so results are equal bit for bit: a row of the products depends on its token
and its expert's weights alone, and the plan is the same.
"""
import pytest
import torch

from moe_synth import make_layer, spec

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


def layer(name, **kw):
    """A layer whose experts all have the weights of the first."""
    L = make_layer(spec(name, **kw))
    for n in ("W13", "W2", "w13_scale", "w2_scale"):
        if L[n] is not None:
            raw = L[n].view(torch.uint8) if L[n].dtype == torch.float8_e4m3fn else L[n]
            L[n] = raw[:1].expand_as(raw).contiguous().view(L[n].dtype)
    return L["spec"], {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in L.items()}


def run(moe, sp, d, tw, ids, options):
    act = moe.MOE_F32 if sp.act == "f32" else moe.MOE_BF16
    wdt = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16, "e4m3": moe.MOE_E4M3, "int4": moe.MOE_INT4}[sp.w]
    need = moe.moe_workspace_size(sp.T, sp.H, sp.I, sp.E, sp.k, act, wdt, options)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    return moe.moe_forward_routed(d["X"], tw.cuda(), ids.cuda(), d["W13"], d["W2"], d["w13_scale"], d["w2_scale"],
                                  workspace=ws, options=options, w_format="int4" if sp.w == "int4" else None)


CASES = [
    # one expert for every pair; pairs: up to 32, up to 1024, more
    ("mixtral_decode", dict(T=9, H=512, I=384, E=8, k=3), {}), ("mixtral_decode", dict(T=5, H=512, I=256, E=32, k=8), {}),
    ("mixtral_decode", dict(T=5, H=512, I=256, E=32, k=8), {"split_k": 3}),
    ("mixtral_decode", dict(T=40, H=512, I=256, E=16, k=4), {}), ("mixtral_decode", dict(T=40, H=256, I=128, E=64, k=30), {}),
    ("mixtral_decode", dict(T=200, H=256, I=256, E=16, k=8), {"orientation": 1}),
    ("fp8_decode", dict(T=9, H=512, I=256, E=8, k=3), {}), ("fp8_decode", dict(T=64, H=512, I=256, E=32, k=20), {}),
    ("int4_decode", dict(T=4, H=512, I=512, E=16, k=8), {}), ("int4_decode", dict(T=100, H=256, I=256, E=16, k=12), {}),
    # forms that compute all of them
    ("tiny_f32", dict(T=9, H=128, I=96, E=8, k=3), {}), ("prefill", dict(T=90, H=512, I=256, E=8, k=3), {}),
    ("prefill", dict(T=90, H=512, I=256, E=8, k=3), {"cta_pair": 2}),
]


@pytest.mark.parametrize("name,kw,options", CASES)
def test_all_pairs_at_one_expert(moe, name, kw, options):
    sp, d = layer(name, **kw)
    if sp.w == "e4m3":  # (the largest intermediate, and with it its scale, is then the same without the dropped pairs)
        d["X"][:] = d["X"][0].clone()
    T, k, E = sp.T, sp.k, sp.E
    tw = torch.softmax(torch.randn(T, k, generator=torch.Generator().manual_seed(T)), 1)
    limit = -(-T // 16) * 16
    swap = moe.moe_plan_info(T, sp.H, sp.I, E, k, moe.MOE_F32 if sp.act == "f32" else moe.MOE_BF16,
                             {"f32": 0, "bf16": 1, "e4m3": 2, "int4": 3}[sp.w], options)["orientation"] == 1
    kept = (torch.arange(T * k).view(T, k) < limit) if swap else torch.ones(T, k, dtype=torch.bool)
    others = torch.arange(k, dtype=torch.int32).expand(T, k).contiguous()  # distinct experts, the same weights
    ref = run(moe, sp, d, torch.where(kept, tw, torch.zeros(())), others, options)
    assert moe.moe_get_status() == 0
    out = run(moe, sp, d, tw, torch.full((T, k), E // 2, dtype=torch.int32), options)
    assert moe.moe_get_status() == (0 if kept.all() else moe.MOE_ERR_DEVICE_INDEX)
    assert torch.isfinite(out).all() and torch.equal(out, ref)
    # as many as the tile holds: nothing is dropped
    few = others.clone()
    few.view(-1)[: min(limit, T * k)] = E // 2
    rest = torch.arange(max(0, T * k - limit), dtype=torch.int32) % (E - 1)
    few.view(-1)[min(limit, T * k) :] = torch.where(rest >= E // 2, rest + 1, rest)
    assert max(int((few == e).sum()) for e in range(E)) <= limit or not swap
    out = run(moe, sp, d, tw, few, options)
    assert moe.moe_get_status() == 0
    assert torch.equal(out, run(moe, sp, d, tw, others, options))
