"""Results of the norms in their inputs' places, bit for bit those in places of their own."""
import pytest
import torch

from test_gpu_norms import DT, EPS, cuda, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


# through the ring and from memory, whole units and rows that share one with a neighbour of another CTA
PLACES = [(6000, 512), (700, 2047), (2500, 33), (20, 16383), (450, 4160), (9, 16384), (40000, 3), (700, 5120)]


@pytest.mark.parametrize("gate", ["channel", "full"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", PLACES)
def test_in_place(moe, T, H, dtype, gate):
    g = torch.Generator().manual_seed(T + H)
    d = {n: cuda(v) for n, v in inputs(T, H, DT[dtype], torch.float32, g, True, gate, True).items()}
    kw = dict(post_w=d["post_w"], gate=d["gate"], scale=0.5, next_w=d["next_w"], eps=EPS)
    out, h = moe.moe_postnorm(d["x"], d["y"], **kw)
    for swap in (False, True):
        x, y = d["x"].clone(), d["y"].clone()
        to, th = (y, x) if swap else (x, y)
        moe.moe_postnorm(x, y, out=to, h=th, **kw)
        assert torch.equal(to, out) and torch.equal(th, h), swap
    ref = moe.moe_postnorm_backward(d["d_out"], d["d_h"], d["x"], d["y"], **kw)
    for places in (("x", "y"), ("y", "x"), ("d_out", "d_h"), ("d_h", "d_out"), ("x", "d_out"), ("d_h", "y")):
        c = {n: d[n].clone() for n in ("x", "y", "d_out", "d_h")}
        got = moe.moe_postnorm_backward(c["d_out"], c["d_h"], c["x"], c["y"], d_x=c[places[0]], d_y=c[places[1]], **kw)
        assert got.d_x is c[places[0]] and got.d_y is c[places[1]]
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), places
    ref = moe.moe_prenorm_backward(d["d_h"], d["x"], d["next_w"], EPS)
    for place in ("x", "d_h"):
        c = {n: d[n].clone() for n in ("x", "d_h")}
        got = moe.moe_prenorm_backward(c["d_h"], c["x"], d["next_w"], EPS, d_x=c[place])
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), place
    assert moe.moe_get_status() == 0
