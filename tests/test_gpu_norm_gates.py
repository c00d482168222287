"""Sigmoid gates that are nearly open or nearly shut."""
import pytest
import torch

from test_gpu_norms import DT, FUZZ, Ref, half, inputs, within
from test_gpu_norm_edges import grads

pytestmark = pytest.mark.gpu

SATURATED = [8.0, -8.0, 12.0, -12.0, 20.0, -20.0, 0.0, 30.0, -30.0, 60.0, -60.0]


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


def saturated(shape):
    n = torch.Size(shape).numel()
    return torch.tensor(SATURATED).repeat(n // len(SATURATED) + 1)[:n].view(shape)


@pytest.mark.parametrize("gate", ["channel", "token", "full"])
@pytest.mark.parametrize("dtype,gate_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,H", [(13, 264), (5, 99), (700, 1024), (700, 2047), (6, 16384)])
def test_gradient_of_a_saturated_gate(moe, T, H, dtype, gate_dtype, gate):
    """d_gate = s (1 - s) times the gate's own gradient, to the same relative error at either end: in 64 bits s(z) s(-z),
    with the gate's own gradient as that of a plain gate of s(z)."""
    g = torch.Generator().manual_seed(T + H)
    d = inputs(T, H, DT[dtype], torch.float32, g, True, gate, True, DT[gate_dtype])
    d["gate"] = saturated(d["gate"].shape).to(DT[gate_dtype])
    z = d["gate"].double()
    ref = Ref(d["x"], d["y"], d["post_w"], torch.sigmoid(z), False, 0.5, 1.25, d["next_w"], d["d_out"], d["d_h"])
    slope = torch.sigmoid(z) * torch.sigmoid(-z)
    got = grads(moe, d, True).d_gate
    want = ref.d_gate * slope
    fuzz = FUZZ + (T * 2.0 ** -24 if z.dim() == 1 else 0.0)
    within(got, want, half(got.dtype) * want.abs() + fuzz * ref.d_gate_m * slope, "d_gate")
    assert moe.moe_get_status() == 0


@pytest.mark.parametrize("gate,gate_dtype", [("channel", "bf16"), ("channel", "f32"), ("token", "f32"), ("full", "f32")])
def test_gradients_in_32_bits_take_the_gate_in_32_bits(moe, gate, gate_dtype):
    """A weight's gradient is fp32 beside bf16 rows too.  d_post_w = scale s(z) d_out n over one row of 64, in roundings of
    2^-24: the sum of y's squares takes 4 + 1 + 5, the mean and eps 2, half of each behind the root; the root 4; n, scale
    times d_out, the sum and the gate's product 5; the sigmoid's exponential 2, its sum 1, its quotient 4, their product 1.
    23 in all, below 2^5.  A full gate's exponential rounds its argument's product: 1.3 |z| more, below 2^7 at 80."""
    g = torch.Generator().manual_seed(5)
    H = 64
    for z in torch.linspace(-80.0, 80.0, 101).tolist():
        d = inputs(1, H, torch.bfloat16, torch.float32, g, True, gate, False, DT[gate_dtype])
        d["gate"] = torch.full_like(d["gate"], z)
        ref = Ref(d["x"], d["y"], d["post_w"], d["gate"], True, 0.5, 1.25, None, d["d_out"], None)
        got = grads(moe, d, True).d_post_w
        within(got, ref.d_post_w, (2.0 ** -17 if gate == "full" else 2.0 ** -19) * ref.d_post_w.abs(), f"d_post_w at {z}")


@pytest.mark.parametrize("gate", ["channel", "token", "full"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(9, 264), (700, 1024), (700, 2047), (5, 16384)])
def test_infinite_gates_are_saturated_ones(moe, T, H, dtype, gate):
    """exp(-10^4) is 0 in fp32: a gate of it and an infinite one are open or shut alike, bit for bit; a NaN is one."""
    g = torch.Generator().manual_seed(T + H)
    d = inputs(T, H, DT[dtype], torch.float32, g, True, gate, True)
    ends = [torch.where(torch.arange(d["gate"].numel()) % 2 == 0, v, -v).view(d["gate"].shape).to(DT[dtype])
            for v in (1e4, float("inf"))]
    for a, b in zip(*(grads(moe, {**d, "gate": v}, True) for v in ends)):
        assert bool(a.isfinite().all()) and torch.equal(a, b)
    kw = dict(post_w=d["post_w"].cuda(), sigmoid=True, next_w=d["next_w"].cuda())
    a, b = (moe.moe_postnorm(d["x"].cuda(), d["y"].cuda(), gate=v.cuda(), **kw) for v in ends)
    assert all(bool(u.isfinite().all()) and torch.equal(u, v) for u, v in zip(a, b))
    bad = d["gate"].clone()
    bad.view(-1)[0] = float("nan")
    out = moe.moe_postnorm(d["x"].cuda(), d["y"].cuda(), gate=bad.cuda(), **kw)[0]
    assert bool({"channel": out[:, 0], "token": out[0], "full": out[0, :1]}[gate].isnan().all())
    assert bool(grads(moe, {**d, "gate": bad}, True).d_gate.view(-1)[0].isnan())
    assert moe.moe_get_status() == 0
