"""Rows of the block-scaled experts' outputs between the second product and the combine.

Up to 64 tokens (swap-AB) they are fp32, above and on CTA pairs bf16.  What that costs is seen in the layer's bf16
output: its error against 64 bits over the error that rounding the 64-bit result to bf16 makes by itself.  Rows of
p significant bits add, in quadrature, 2^(8 - p) of that rounding's error (the terms of a token's sum are as large as
the sum, in the 2-norm): nothing for fp32, 1.41 in all for bf16.  Intermediates that take the other of two codes at a
border add at most 0.65 of it (2^-10 of the norm: one in 2^14, an eighth of its value each, is far above what sums in
another order do).  So the bars are sqrt(1 + 0.65^2) = 1.2 and sqrt(2 + 0.65^2) = 1.56.
"""
import numpy as np
import pytest
import torch

from test_gpu_block_fp8 import experts_reference, make_experts

pytestmark = pytest.mark.gpu

# T, E, k, options: fp32 rows, swap-AB with bf16 rows, CTA pairs (full tiles, tails, an odd number of column blocks)
FORMS = [(20, 8, 4, {}), (64, 32, 8, {}), (90, 32, 8, {}), (300, 16, 8, {"orientation": 1}), (300, 8, 8, {}),
         (700, 4, 3, {}), (40, 32, 8, {"orientation": 2})]


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


def run(moe, d, options, **over):
    c = {n: v.cuda() for n, v in dict(d, **over).items()}
    out = moe.moe_forward_routed(c["x"], c["tw"], c["ids"], c["w13"], c["w2"], c["s13"], c["s2"], options=options,
                                 w_format="e4m3_block")
    assert moe.moe_get_status() == 0
    return out.cpu()


@pytest.mark.parametrize("T,E,k,options", FORMS)
@pytest.mark.parametrize("H,I", [(384, 256), (256, 640)])
def test_error_over_that_of_one_rounding(moe, T, E, k, options, H, I):
    d = make_experts(T, H, I, E, k, torch.Generator().manual_seed(T + H))
    out = run(moe, d, options).double()
    ref = torch.from_numpy(experts_reference(d))
    ratio = float((out - ref).norm() / (ref.to(torch.bfloat16).double() - ref).norm())
    fp32_rows = T <= 64 and options.get("orientation") != 2
    assert ratio <= (1.2 if fp32_rows else 1.56), f"{ratio:.2f} times the error of one rounding"


@pytest.mark.parametrize("T,E,k,options", FORMS)
@pytest.mark.parametrize("shift", [-90, -30, 30, 100])
def test_a_power_of_two_in_the_weights_scales_comes_out_exactly(moe, T, E, k, options, shift):
    """Rows far from the usual size (2^-90 to 2^100 times)."""
    d = make_experts(T, 384, 256, E, k, torch.Generator().manual_seed(T))
    base = run(moe, d, options)
    out = run(moe, d, options, s2=d["s2"] * 2.0 ** shift)
    assert torch.equal(out.double(), base.double() * 2.0 ** shift)


@pytest.mark.parametrize("T,E,k,options", FORMS)
def test_column_blocks_of_different_size(moe, T, E, k, options):
    """Neighbouring blocks of 128 columns whose weights differ by 2^40: each keeps its own bits; a block of zero
    weights gives zeros."""
    d = make_experts(T, 384, 256, E, k, torch.Generator().manual_seed(T))
    f = torch.tensor([1.0, 2.0 ** 40, 2.0 ** -40])[None, :, None]
    base, out = run(moe, d, options), run(moe, d, options, s2=d["s2"] * f)
    assert torch.equal(out.double(), base.double() * f[:, :, 0].repeat_interleave(128, 1).double())
    w2 = d["w2"].clone()
    w2.view(torch.uint8)[:, 128:256] = 0
    out = run(moe, d, options, w2=w2)
    assert (out[:, 128:256] == 0).all() and torch.equal(out[:, :128], base[:, :128]) and torch.equal(out[:, 256:], base[:, 256:])


@pytest.mark.parametrize("T,E,k,options", FORMS)
def test_not_a_number_stays_with_its_token(moe, T, E, k, options):
    d = make_experts(T, 384, 256, E, k, torch.Generator().manual_seed(T))
    base = run(moe, d, options)
    x = d["x"].clone()
    x[3, 5], x[T - 2, 300] = float("nan"), float("inf")
    out = run(moe, d, options, x=x)
    bad = torch.zeros(T, dtype=torch.bool)
    bad[[3, T - 2]] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], base[~bad])


def test_wide_rows(moe):
    """H of 56 column blocks; every expert's weights of each block at a size of its own."""
    d = make_experts(80, 7168, 128, 4, 3, torch.Generator().manual_seed(1))
    d["s2"] = d["s2"] * 2.0 ** torch.randint(-40, 40, (4, 56, 1), generator=torch.Generator().manual_seed(2)).float()
    for options in ({"orientation": 1}, {"orientation": 2}):
        out = run(moe, d, options).double().numpy()
        ref = experts_reference(d)
        for b in range(56):  # (one block is as large as its largest expert's)
            o, r = out[:, 128 * b : 128 * b + 128], ref[:, 128 * b : 128 * b + 128]
            assert np.linalg.norm(o - r) <= 5e-3 * np.linalg.norm(r)
