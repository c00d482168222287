"""The example's expert block: the served form against 64-bit formulas of what the block's new calls add, and a
training step's gradients against torch's differentiation in 64 bits."""
import os
import sys

import pytest
import torch

from moe_synth import make_block_layer

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

EPS = 1e-6


def normed(v, w):
    return v * ((v * v).mean(1, keepdim=True) + EPS) ** -0.5 * w


def near(got, ref, tol):
    """Relative to the reference's norm."""
    got, ref = got.double().cpu(), ref.double().cpu()
    assert got.shape == ref.shape
    err = float((got - ref).norm() / ref.norm())
    assert err <= tol, err


@pytest.mark.parametrize("T", [1, 33, 200, 1500])
def test_served_block(T):
    import expert_block as ex
    import mixture_experts_layer_scan_gb300 as moe

    H, I, E, Is, r, L = 512, 256, 32, 384, 16, 5
    g = torch.Generator().manual_seed(T)
    w = {n: v.cuda() for n, v in make_block_layer(H, I, E, I_shared=Is, seed=T).items()}
    a = dict(a=(torch.randn(L, r, H, generator=g) * H ** -0.5).bfloat16(), b=torch.randn(L, 2 * Is, r, generator=g).bfloat16(),
             scale=torch.rand(L, generator=g) + 0.5)
    n = {k: (1 + 0.3 * torch.randn(H, generator=g)).bfloat16() for k in ("pre", "post", "gate", "next")}
    layer = ex.ServedBlock(w, {k: v.cuda() for k, v in a.items()}, {k: v.cuda() for k, v in n.items()}, scale=0.25)
    x = torch.randn(T, H, generator=g).bfloat16()
    who = torch.randint(-1, L, (T,), generator=g).int()
    h = layer.first(x.cuda())
    near(h, normed(x.double(), n["pre"].double()), 2.0 ** -8)  # (each element off by half a step of bf16 at most)
    # the adapters, on the shared expert's projections without them
    q, s = moe.moe_quant_block(h)
    plain = moe.moe_gemm_block(q, s, w["shared13"], w["shared13_scale"]).double().cpu()
    z, gate_up = layer.shared(h, who.cuda())
    ref = plain.clone()
    for t in range(T):
        if who[t] >= 0:
            l = int(who[t])
            ref[t] += float(a["scale"][l]) * (a["b"][l].double() @ (a["a"][l].double() @ h[t].double().cpu()))
    near(gate_up, ref, 2.0 ** -8)
    y = layer.experts(h)
    y += z
    out, h2 = layer(x.cuda(), h, who.cuda())
    ref = x.double() + 0.25 * n["gate"].double() * normed(y.double().cpu(), n["post"].double())
    near(out, ref, 2.0 ** -8)
    near(h2, normed(ref, n["next"].double()), 2.0 ** -8)
    assert moe.moe_get_status() == 0


@pytest.mark.parametrize("T,k,E,block", [(7, 2, 4, 16), (65, 3, 8, 4), (300, 2, 16, 16)])
def test_training_step(T, k, E, block):
    import expert_block as ex
    import mixture_experts_layer_scan_gb300 as moe

    H = 96
    g = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    ids = torch.rand(T, E, generator=g).topk(k, 1)[1].int()
    v = dict(x=r(T, H), topk_w=torch.rand(T, k, generator=g), matrices=r(E, H, H) / H ** 0.5, pre=1 + r(H) / 4,
             post=1 + r(H) / 4, gate=r(H), nxt=1 + r(H) / 4)
    d_out, d_h = r(T, H), r(T, H)
    c = {n: t.cuda() for n, t in v.items()}
    out, h, grads = ex.train_step(c["x"], ids.cuda(), c["topk_w"], c["matrices"], c["pre"], c["post"], c["gate"], c["nxt"],
                                  d_out.cuda(), d_h.cuda(), block)
    assert moe.moe_get_status() == 0
    d = {n: t.double().requires_grad_() for n, t in v.items()}
    n = normed(d["x"], d["pre"])
    y = (d["topk_w"][:, :, None] * torch.einsum("tkgh,th->tkg", d["matrices"][ids.long()], n)).sum(1)
    o = d["x"] + torch.sigmoid(d["gate"]) * normed(y, d["post"])
    hh = normed(o, d["nxt"])
    ((o * d_out.double()).sum() + (hh * d_h.double()).sum()).backward()
    # (fp32 throughout; the products' 96 terms are rounded to 2^-24 each, and tf32 is off by default)
    near(out, o.detach(), 1e-5)
    near(h, hh.detach(), 1e-5)
    for name, got in grads.items():
        near(got, d[name].grad, 1e-5)
