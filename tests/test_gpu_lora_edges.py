"""Adapters whose numbers leave the ordinary: infinite weights, products near the end of fp32, results that need all of fp32.
The tensor cores and the path of a token at a time give the same answers."""
import pytest
import torch

from test_gpu_lora import DT, formula, make, sorts

pytestmark = pytest.mark.gpu

INF = float("inf")
# (tokens, K, N, rank, adapters), whether the tokens are sorted by adapter and multiplied on the tensor cores
PATHS = [((5, 64, 264, 16, 3), False), ((4000, 64, 1032, 16, 3), True), ((1030, 72, 520, 128, 2), True),
         ((3000, 64, 1032, 24, 6), True)]


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


def call(moe, d, base, dtype, **kw):
    c = {n: v.cuda() for n, v in d.items()}
    return moe.moe_lora(c["x"], c["a"], c["b"], c["ids"], scale=c["scale"], base=None if base is None else base.cuda(),
                        out_dtype=dtype, **kw).cpu()


@pytest.mark.parametrize("out_t", ["bf16", "f32"])
@pytest.mark.parametrize("size,tc", PATHS)
def test_infinite_weights_of_b(moe, size, tc, out_t):
    """An infinite element of b times h is infinite with h's sign, whatever h is made of; two of unlike signs, or one beside
    an h of exactly 0, give NaN; a NaN gives NaN; other columns are as the formula has them."""
    T, K, N, r, L = size
    assert sorts(moe, *size) == tc
    d = make(*size, seed=T)
    d["ids"][:4] = torch.tensor([0, 1, 0, -1], dtype=torch.int32)
    d["x"][2] = 0.0                                   # h = 0
    d["b"][:, 3, 1], d["b"][:, 70, 2], d["b"][0, N - 1, r - 1] = INF, -INF, INF
    d["b"][1, 8, 0], d["b"][1, 8, 5] = INF, -INF      # of h's unlike or like signs
    d["b"][0, 40, 4] = float("nan")
    d["a"][:, 7] = 0.0                                # an h of exactly 0 in every token
    d["b"][:, 100, 7] = INF
    d["x"][:, 1:] = torch.where(torch.arange(T)[:, None] % 5 == 4, 0.0, d["x"][:, 1:].float()).to(torch.bfloat16)
    d["x"][4::5, 0], d["a"][:, :7, 0] = 1.0, d["a"][:, :7, 0].abs() + 0.5  # every fifth token: h is one bf16 number
    d["scale"][:] = 1.0
    for base in (None, d["base"].to(DT[out_t])):
        ref, mag = formula(d, base, d["scale"])
        got = call(moe, d, base, DT[out_t]).double()
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(torch.where(got.isinf(), got.sign(), 0.0), torch.where(ref.isinf(), ref.sign(), 0.0))
        ok = ref.isfinite()
        # (the tolerance of ordinary values: bf16 parts of h, and fp32 sums)
        tol = torch.finfo(DT[out_t]).eps / 2 * ref.abs() + ((K + r + 4) * 2.0 ** -24 + 2.0 ** -16) * mag
        assert bool(((got - ref).abs() <= tol)[ok].all())
    assert moe.moe_get_status() == 0


@pytest.mark.parametrize("out_t", ["bf16", "f32"])
@pytest.mark.parametrize("size,tc", PATHS)
def test_product_between_the_largest_bf16_and_the_largest_fp32(moe, size, tc, out_t):
    """A x is finite in fp32 though it rounds to an infinite bf16; b brings it back into range.  h = 511.5 2^119 exactly,
    b a power of two: the result is h's, off by its type's rounding and by 2^-16 where a bf16 result takes h as two parts."""
    T, K, N, r, L = size
    assert sorts(moe, *size) == tc
    d = make(*size, seed=T, none=0.0)
    d["x"].zero_(), d["a"].zero_(), d["b"].zero_()
    d["x"][:, 0], d["x"][:, 1] = 2.0 ** 60, 2.0 ** 52
    d["a"][:, 1, 0], d["a"][:, 1, 1] = 255 * 2.0 ** 60, 192 * 2.0 ** 60  # (255 + 0.75) 2^120
    d["b"][:, :, 1] = 2.0 ** -100
    d["x"][1::2] = -d["x"][1::2]
    d["scale"][:] = 1.0
    want = 255.75 * 2.0 ** 20
    got = call(moe, d, None, DT[out_t]).double()
    sign = torch.where(torch.arange(T) % 2 == 1, -1.0, 1.0)[:, None].double()
    tol = (torch.finfo(DT[out_t]).eps / 2 + (2.0 ** -16 if out_t == "bf16" else 2.0 ** -23)) * want
    assert bool(((got - sign * want).abs() <= tol).all())
    assert moe.moe_get_status() == 0


@pytest.mark.parametrize("size,tc", PATHS)
def test_results_in_32_bits_hold_all_of_h(moe, size, tc):
    """h = c0 + c1 2^-8 + c2 2^-16 with odd c of 8 bits has 24, all of which reach an fp32 result: K sums without a
    rounding, one b of 1.  On the CUDA cores the result is h; the tensor cores may lose a unit (2^-23) when they add
    the parts of h.  h as two bf16 parts would not do, however they are rounded."""
    T, K, N, r, L = size
    assert sorts(moe, *size) == tc
    g = torch.Generator().manual_seed(T)
    d = make(*size, seed=T, none=0.0)
    d["x"].zero_(), d["a"].zero_(), d["b"].zero_()
    c = torch.randint(64, 128, (T, 3), generator=g) * 2 + 1
    x = c.double() * torch.tensor([1.0, 2.0 ** -8, 2.0 ** -16], dtype=torch.float64)
    at = [0, K // 2, K - 1]
    d["x"][:, at] = x.to(torch.bfloat16)
    assert torch.equal(d["x"][:, at].double(), x)
    row, col = r - 3, torch.arange(0, N, 3)
    d["a"][:, row, at] = 1.0
    for l in range(L):
        d["b"][l, col, row] = (-1.0) ** l
    d["scale"][:] = 1.0
    got = call(moe, d, None, torch.float32).double()
    want = (x.sum(1) * (1 - 2 * (d["ids"] % 2)))[:, None].expand(T, N).clone()
    want[:, torch.arange(N) % 3 != 0] = 0.0
    assert torch.equal(want.float().double(), want)
    h = x.sum(1)
    for first in (h.bfloat16().double(), (h.float().view(torch.int32) & -65536).view(torch.float32).double()):
        assert float(((h - first - (h - first).bfloat16().double()).abs() / h).max()) > 2.0 ** -20
    err = (got - want).abs() / x.sum(1)[:, None]
    assert float(err.max()) <= (2.0 ** -23 if tc else 0.0)
    assert moe.moe_get_status() == 0
