"""Norms and their gradients where a factor of the formula is absent."""
import pytest
import torch

from test_gpu_norms import DT, EPS, cuda, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


def grads(moe, d, sigmoid=False, scale=0.5, res=1.25, **over):
    c = {n: cuda(v) for n, v in {**d, **over}.items()}
    return moe.moe_postnorm_backward(c["d_out"], c["d_h"], c["x"], c["y"], post_w=c["post_w"], gate=c["gate"],
                                     sigmoid=sigmoid, scale=scale, res_scale=res, next_w=c["next_w"], eps=EPS)


def same(a, b):
    """Equal bits (a result that a call has not: neither has it)."""
    return all((u is None and v is None) or torch.equal(u, v) for u, v in zip(a, b))


def spoil(t, rows):
    """An infinity, a NaN and a row of infinities in the given three rows."""
    t = t.clone()
    t[rows[0], t.shape[1] // 2] = float("inf")
    t[rows[1], -1] = float("nan")
    t[rows[2]] = float("-inf")
    return t


# each form of the gradient: rows from memory and through the ring, whole units and not, short and long, two CTAs to an SM
EDGES = [(9, 264), (11, 1023), (6000, 512), (700, 2047), (500, 4096), (5, 16384), (4, 16383), (700, 5120)]


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", EDGES)
def test_gradient_without_a_next_norm_does_not_see_x(moe, T, H, dtype, gate):
    """Without the next norm out is a sum, and no gradient has x in it: what x holds changes no bit of any, those of
    the weights and of a channel gate included.  So too beside a next norm that gets no gradient, whose weight's is 0."""
    g = torch.Generator().manual_seed(T + H)
    d = inputs(T, H, DT[dtype], torch.float32, g, True, gate, True)
    d["d_h"] = None
    bad = spoil(d["x"], (1, T // 2, T - 1))
    for post in (True, False):
        for nxt in (True, False):
            e = {**d, "post_w": d["post_w"] if post else None, "next_w": d["next_w"] if nxt else None}
            ref, got = grads(moe, e, gate != "none"), grads(moe, e, gate != "none", x=bad)
            assert all(v is None or bool(v.isfinite().all()) for v in ref)
            assert same(got, ref), (post, nxt)
            assert not nxt or bool((got.d_next_w == 0).all())
    assert moe.moe_get_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", EDGES)
def test_gradient_without_norms_sees_y_in_the_gate_alone(moe, T, H, dtype):
    """out = res x + scale G y: d_x and d_y hold neither x nor y, and a gate's gradient holds y where it gates it."""
    g = torch.Generator().manual_seed(T + H)
    rows = (1, T // 2, T - 1)
    for gate in ("none", "channel", "token", "full"):
        d = inputs(T, H, DT[dtype], torch.float32, g, False, gate, False)
        bad = spoil(d["y"], rows)
        ref, got = grads(moe, d), grads(moe, d, y=bad)
        assert torch.equal(got.d_x, ref.d_x) and torch.equal(got.d_y, ref.d_y), gate
        if gate == "token":
            keep = torch.ones(T, dtype=torch.bool, device="cuda")
            keep[list(rows)] = False
            assert torch.equal(got.d_gate[keep], ref.d_gate[keep]) and not bool(got.d_gate[~keep].isfinite().any())
        elif gate == "full":
            finite = bad.isfinite().cuda()
            assert torch.equal(got.d_gate[finite], ref.d_gate[finite])
            assert not bool(got.d_gate[~finite & (d["d_out"].cuda() != 0)].isfinite().any())
    assert moe.moe_get_status() == 0
