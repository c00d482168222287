"""A caller's routing with expert ids outside [0, E): those pairs are dropped, so they add nothing to their
token's output, whatever the workspace held.

Every call runs over a workspace of NaN bit patterns.  The result is compared bit for bit with a routing that
names a valid expert with weight 0 in the place of each dropped pair: fma(0, y, acc) = acc, every other pair's
row is computed from its own token and expert alone, and the plan is the same.  (The replacement repeats a pair
of the batch -- token 7 is a copy of token 6 -- so the FP8 path's largest intermediate is the same too.)
The block-scaled form is also compared with 64 bits, within the bars of the layer's own tests.
"""
import pytest
import torch

from moe_synth import make_layer, spec
from test_gpu_block_fp8 import check, experts_reference, make_experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


def routings(ids, tw, E):
    """(ids, weights) with dropped pairs, and with weight 0 in their place."""
    bad, ok, w0 = ids.clone(), ids.clone(), tw.clone()
    bad[3, 1], ok[3, 1], w0[3, 1] = E, ids[3, 0], 0
    bad[5, 0], ok[5, 0], w0[5, 0] = -2, ids[5, 1], 0
    bad[8, -1], ok[8, -1], w0[8, -1] = 2 ** 31 - 1, ids[8, 0], 0
    bad[7], ok[7], w0[7] = -1, ids[6, 0], 0  # a token without any expert
    return bad, ok, w0


def run(moe, X, tw, ids, w13, w2, s13, s2, E, w_dtype, options, w_format):
    T, H = X.shape
    act = moe.MOE_F32 if X.dtype == torch.float32 else moe.MOE_BF16
    I = w2.shape[2] * (2 if w_format == "int4" else 1)
    need = moe.moe_workspace_size(T, H, I, E, ids.shape[1], act, w_dtype, options)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(X, float("nan"))
    moe.moe_forward_routed(X, tw.cuda(), ids.cuda(), w13, w2, s13, s2, out=out, workspace=ws, options=options,
                           w_format=w_format)
    return out


LAYERS = [("tiny_f32", dict(T=9, H=128, I=96), {}), ("tiny_f32", dict(T=11, H=20, I=33), {}),
          ("mixtral_decode", dict(T=9, H=512, I=384), {}), ("mixtral_decode", dict(T=9, H=512, I=384), {"split_k": 3}),
          ("mixtral_decode", dict(T=48, H=512, I=256), {}), ("prefill", dict(T=90, H=512, I=256), {}),
          ("prefill", dict(T=90, H=384, I=256), {"cta_pair": 2}), ("prefill", dict(T=4100, H=256, I=128), {}),
          ("fp8_decode", dict(T=9, H=512, I=256), {}), ("fp8_decode", dict(T=90, H=512, I=256), {}),
          ("int4_decode", dict(T=9, H=512, I=512), {}), ("int4_decode", dict(T=40, H=512, I=512), {})]


@pytest.mark.parametrize("name,kw,options", LAYERS)
def test_dropped_pairs_add_nothing(moe, name, kw, options):
    E, k = 32, 3
    L = make_layer(spec(name, E=E, k=k, **kw))
    sp = L["spec"]
    d = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in L.items()}
    d["X"][7] = d["X"][6]
    v, ids = torch.randn(sp.T, E, generator=torch.Generator().manual_seed(sp.T)).topk(k, 1)
    bad, ok, w0 = routings(ids.to(torch.int32), torch.softmax(v, 1), E)
    wdt = {"f32": moe.MOE_F32, "bf16": moe.MOE_BF16, "e4m3": moe.MOE_E4M3, "int4": moe.MOE_INT4}[sp.w]
    args = (d["W13"], d["W2"], d["w13_scale"], d["w2_scale"], E, wdt, options, "int4" if sp.w == "int4" else None)
    ref = run(moe, d["X"], w0, ok, *args)
    assert moe.moe_get_status() == 0
    out = run(moe, d["X"], torch.softmax(v, 1), bad, *args)
    assert moe.moe_get_status() == moe.MOE_ERR_DEVICE_INDEX
    assert torch.isfinite(out).all() and torch.equal(out, ref) and (out[7] == 0).all()


# T, E, options: up to 32 pairs, swap-AB with fp32 rows, swap-AB with bf16 rows, CTA pairs
BLOCK = [(10, 4, {}), (20, 4, {}), (48, 16, {}), (90, 16, {}), (300, 4, {"orientation": 1}), (90, 4, {}),
         (48, 4, {"orientation": 2}), (700, 4, {})]


@pytest.mark.parametrize("T,E,options", BLOCK)
def test_dropped_pairs_of_block_scaled_experts(moe, T, E, options):
    d = make_experts(T, 256, 128, E, 3, torch.Generator().manual_seed(T))
    d["x"][7] = d["x"][6]
    bad, ok, w0 = routings(d["ids"], d["tw"], E)
    c = {n: v.cuda() for n, v in d.items()}
    args = (c["w13"], c["w2"], c["s13"], c["s2"], E, moe.MOE_E4M3_B128, options, "e4m3_block")
    ref = run(moe, c["x"], w0, ok, *args)
    assert moe.moe_get_status() == 0
    out = run(moe, c["x"], d["tw"], bad, *args)
    assert moe.moe_get_status() == moe.MOE_ERR_DEVICE_INDEX
    assert torch.isfinite(out).all() and torch.equal(out, ref) and (out[7] == 0).all()
    check(out, experts_reference(dict(d, ids=bad)), f"dropped pairs T={T}")
