"""The example layer (grouped routing, block-scaled experts and shared expert) against a plain 64-bit
form, over batches that run each kind of tile."""
import os
import sys

import numpy as np
import pytest
import torch

from moe_synth import make_block_layer
from test_gpu_block_fp8 import TABLE, check, quant_reference, weights64
from test_gpu_route_grouped import reference as route_reference

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def rows(x):
    q, s = quant_reference(x)
    return torch.from_numpy(TABLE[q] * np.repeat(s.astype(np.float64), 128, 1)[:, : x.shape[1]])


def mlp(x, w13, s13, w2, s2):
    v = x @ weights64(w13, s13).t()
    g, u = v.split(v.shape[1] // 2, 1)
    return rows((g / (1 + torch.exp(-g)) * u).float().numpy()) @ weights64(w2, s2).t()


@pytest.mark.parametrize("T", [1, 30, 100, 600])
def test_layer(T):
    import block_fp8_layer as ex
    import mixture_experts_layer_scan_gb300 as moe

    H, I, E = 512, 256, 32
    w = make_block_layer(H, I, E, I_shared=400, seed=T)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    layer = ex.BlockFp8Layer({k: v.cuda() for k, v in w.items()}, T)
    out = layer(x.cuda())
    assert moe.moe_get_status() == 0
    logits, tw, ids = moe.moe_route_grouped(x.cuda(), layer.w["router"], ex.TOPK, bias=layer.w["bias"], **ex.RULE)
    # routing from the device's logits, as the layer's
    rw, rid, clear = route_reference(logits.cpu().numpy(), w["bias"].numpy(), ex.TOPK, "sigmoid", 8, 4, 2, True, 2.5)
    ids = ids.cpu().numpy()
    assert clear.any() and np.array_equal(ids[clear], rid[clear])
    rid[~clear], rw[~clear] = ids[~clear], tw.cpu().numpy()[~clear]
    xq = rows(x.float().numpy())
    ref = mlp(xq, w["shared13"], w["shared13_scale"], w["shared2"], w["shared2_scale"])
    for e in range(E):
        t, j = np.nonzero(rid == e)
        if len(t):
            y = mlp(xq[t], w["w13"][e], w["w13_scale"][e], w["w2"][e], w["w2_scale"][e])
            ref.index_add_(0, torch.from_numpy(t), y * torch.from_numpy(rw[t, j])[:, None])
    # (the shared expert's gate_up is bf16 here: one more rounding of 2^-9 before its SiLU product is coded)
    got = out.float().cpu().numpy()
    assert np.linalg.norm(got - ref.numpy()) <= 2e-2 * np.linalg.norm(ref.numpy())
