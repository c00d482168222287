"""Low-rank adapters of many requests against the formula in 64 bits.

Tolerances: half a step of the output's type, and with M = |base| + s |B| |A| |x| (the formula in absolute values):
(K + rank + 4) roundings of 2^-24 for fp32 sums in any order, and 2^-16 for the products h = A x taken as
two bf16 parts (2^-17 of h, for each of the two roundings)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


def make(T, K, N, r, L, seed, none=0.1, runs=False):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, L, (T,), generator=g)
    if runs:
        ids = ids.sort()[0][torch.randperm(T, generator=g).sort()[0]]
    ids[torch.rand(T, generator=g) < none] = -1
    return dict(x=torch.randn(T, K, generator=g).to(torch.bfloat16),
                a=(torch.randn(L, r, K, generator=g) / K ** 0.5).to(torch.bfloat16),
                b=(torch.randn(L, N, r, generator=g) / r ** 0.5).to(torch.bfloat16), ids=ids.to(torch.int32),
                scale=torch.rand(L, generator=g) + 0.5, base=torch.randn(T, N, generator=g))


def formula(d, base, scale):
    """(out, its magnitude) in 64 bits."""
    T, N = d["x"].shape[0], d["b"].shape[1]
    out = torch.zeros(T, N, dtype=torch.float64) if base is None else base.double()
    mag = out.abs()
    for l in range(d["a"].shape[0]):
        t = (d["ids"] == l).nonzero()[:, 0]
        if len(t):
            x, a, b = d["x"][t].double(), d["a"][l].double(), d["b"][l].double()
            s = 1.0 if scale is None else float(scale[l])
            out[t] += s * (x @ a.t() @ b.t())
            mag[t] += abs(s) * (x.abs() @ a.abs().t() @ b.abs().t())
    return out, mag


def check(moe, d, out_t="bf16", base=True, scale=True, out=None, ws=None):
    T, K = d["x"].shape
    dt = DT[out_t]
    bs = d["base"].to(dt) if base else None
    sc = d["scale"] if scale else None
    ref, mag = formula(d, bs, sc)
    got = moe.moe_lora(d["x"].cuda(), d["a"].cuda(), d["b"].cuda(), d["ids"].cuda(), scale=None if sc is None else sc.cuda(),
                       base=None if bs is None else bs.cuda(), out_dtype=dt, out=out, workspace=ws)
    tol = torch.finfo(dt).eps / 2 * ref.abs() + ((K + d["a"].shape[1] + 4) * 2.0 ** -24 + 2.0 ** -16) * mag
    bad = ~((got.double().cpu() - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off"
    assert moe.moe_get_status() == 0
    return got


# T, K, N, rank, L
SIZES = [(1, 8, 8, 8, 1), (1, 4096, 4096, 16, 4), (3, 72, 40, 24, 2), (16, 512, 1000, 64, 16), (48, 1024, 264, 16, 64),
         (65, 256, 2048, 128, 3), (130, 2040, 520, 32, 5), (300, 520, 136, 8, 40), (777, 328, 1032, 40, 7),
         (1030, 1024, 768, 64, 3), (2100, 136, 264, 128, 2), (257, 64, 8, 8, 200), (1500, 72, 4104, 16, 1)]


@pytest.mark.parametrize("out_t", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(moe, size, out_t):
    check(moe, make(*size, seed=sum(size)), out_t)


def sorts(moe, T, K, N, r, L):
    """Whether a call sorts its tokens by adapter (tensor cores): its workspace is then more than h [T,r] in fp32."""
    return moe.moe_lora_workspace_size(T, K, N, r, L) > -(-T * r * 4 // 256) * 256


# the same for what the tensor cores take: odd lengths of K, N and rank, a block of one token, adapters in one block
# each and in many, K in one piece and shared by clusters of 2, 4 and 8
LARGE = [(120000, 72, 40, 8, 3), (9000, 136, 264, 24, 5), (100001, 64, 8, 16, 1), (300, 2040, 4104, 128, 3),
         (129, 8192, 8200, 120, 1), (1000, 1032, 2056, 64, 40), (2500, 520, 1000, 40, 7), (30000, 8, 72, 32, 300),
         (900, 4096, 136, 72, 2)]


@pytest.mark.parametrize("out_t", ["bf16", "f32"])
@pytest.mark.parametrize("size", LARGE)
def test_tensor_core_sizes(moe, size, out_t):
    assert sorts(moe, *size)
    check(moe, make(*size, seed=sum(size), runs=size[0] % 2 == 0), out_t)


FORMS = [(2, 264, 520, 16, 6), (40, 264, 520, 16, 6), (3000, 264, 1032, 64, 6)]


@pytest.mark.parametrize("size", FORMS)
def test_forms(moe, size):
    """Without a base, without scales, one adapter for all, none at all, in place."""
    assert sorts(moe, *size) == (size[0] == 3000)
    T = size[0]
    d = make(*size, T)
    for out_t in ("bf16", "f32"):
        check(moe, d, out_t, base=False)
        check(moe, d, out_t, scale=False)
        check(moe, {**d, "ids": torch.full_like(d["ids"], 5)}, out_t)
        none = {**d, "ids": torch.full_like(d["ids"], -1)}
        got = check(moe, none, out_t)
        assert torch.equal(got.cpu(), d["base"].to(DT[out_t]))
        assert (check(moe, none, out_t, base=False) == 0).all()
    ref = check(moe, d, "bf16")
    buf = d["base"].to(torch.bfloat16).cuda()
    got = moe.moe_lora(d["x"].cuda(), d["a"].cuda(), d["b"].cuda(), d["ids"].cuda(), scale=d["scale"].cuda(), base=buf,
                       out=buf)
    assert got is buf and torch.equal(buf, ref)


@pytest.mark.parametrize("T", [7, 300, 12000])
def test_runs_and_single_tokens(moe, T):
    """Tokens of a request side by side, a request with one token, adapters that no token names (NaN there is not
    read into any result)."""
    d = make(T, 136, 264, 16, 9, T)
    d["ids"] = (torch.arange(T) * 3 // T).to(torch.int32) * 3
    d["ids"][0] = 8
    d["a"][1], d["b"][1], d["b"][4] = float("nan"), float("nan"), float("nan")
    check(moe, d)


@pytest.mark.parametrize("T", [5, 400, 12000])
def test_ids_out_of_range(moe, T):
    d = make(T, 136, 264, 16, 4, T)
    ids = d["ids"].clone()
    d["ids"][::3] = -1
    ids[::3] = torch.tensor([4, -2, 1 << 30, -(1 << 31)], dtype=torch.int32)[torch.arange(len(ids[::3])) % 4]
    ref = check(moe, d)
    c = {n: v.cuda() for n, v in d.items()}
    got = moe.moe_lora(c["x"], c["a"], c["b"], ids.cuda(), scale=c["scale"], base=c["base"].to(torch.bfloat16))
    assert moe.moe_get_status() == moe.MOE_ERR_DEVICE_INDEX
    assert torch.equal(got, ref)


def test_special_values(moe):
    """A NaN or an infinity in a token's input or base stays in that token's row."""
    for T in (9, 300, 12000):
        d = make(T, 136, 264, 16, 4, T, none=0.0)
        c = {n: v.cuda() for n, v in d.items()}
        ref = moe.moe_lora(c["x"], c["a"], c["b"], c["ids"], base=c["base"])
        x, base = c["x"].clone(), c["base"].clone()
        x[1, 3], x[2, 100], base[4, 7] = float("nan"), float("inf"), float("inf")
        got = moe.moe_lora(x, c["a"], c["b"], c["ids"], base=base)
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[[1, 2, 4]] = False
        assert torch.equal(got[keep], ref[keep])
        assert got[1].isnan().all() and not got[2].isfinite().any() and got[4, 7] == float("inf")
        assert torch.equal(got[4, :7], ref[4, :7])


def test_stale_workspace_graph_and_stream(moe):
    """A workspace with anything in it, shared by calls of other sizes; a captured call on new ids; another stream."""
    ws = torch.empty(max(moe.moe_lora_workspace_size(T, 520, 1032, 64, 8) for T in range(1, 601)), dtype=torch.uint8,
                     device="cuda").fill_(255)
    assert sorts(moe, 600, 520, 1032, 64, 8) and not sorts(moe, 200, 520, 1032, 64, 8)
    for T in (600, 3, 500, 200, 64, 601):
        check(moe, make(T, 520, 1032, 64, 8, T), ws=ws)
    assert sorts(moe, 9000, 264, 520, 16, 6)
    for T in (20, 500, 9000):
        sets = [{n: v.cuda() for n, v in make(T, 264, 520, 16, 6, s).items()} for s in range(3)]
        one = {n: v.clone() for n, v in sets[0].items()}
        call = lambda c, **k: moe.moe_lora(c["x"], c["a"], c["b"], c["ids"], scale=c["scale"], base=c["base"], **k)  # noqa: E731
        refs = [call(c).clone() for c in sets]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(one)
        for c, ref in zip(sets, refs):
            for n in one:
                one[n].copy_(c[n])
            graph.replay()
            assert torch.equal(out, ref)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)
        got = call(sets[1], stream=side)
        side.synchronize()
        with torch.cuda.stream(side):
            assert torch.equal(got, refs[1])
        torch.cuda.synchronize()
    assert moe.moe_get_status() == 0


def test_empty(moe):
    d = {n: v.cuda() for n, v in make(4, 64, 72, 8, 2, 1).items()}
    assert moe.moe_lora(d["x"][:0], d["a"], d["b"], d["ids"][:0]).shape == (0, 72)


@pytest.mark.parametrize("out_t", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 1030])
def test_product_that_overflows(moe, T, out_t):
    """A x beyond fp32 is infinite, and so is what it gives, with the formula's signs; other tokens are as they were."""
    d = make(T, 1024, 768, 16, 3, T)
    d["x"][::3] = d["x"][::3].abs() * 2.0 ** 66
    d["a"][:, 0] = 2.0 ** 66
    d["a"][:, 1:] = 0
    d["b"][:, :, 0] = torch.where(d["b"][:, :, 0] < 0, -1.0, 1.0)
    got = moe.moe_lora(*(d[n].cuda() for n in ("x", "a", "b", "ids")), out_dtype=DT[out_t]).cpu()
    on = (d["ids"] >= 0) & (torch.arange(T) % 3 == 0)
    sign = d["b"][d["ids"].clamp(min=0).long(), :, 0].float()
    assert torch.equal(got[on].float(), sign[on] * float("inf"))
    assert bool((got[d["ids"] < 0] == 0).all())
    rest = (d["ids"] >= 0) & (torch.arange(T) % 3 != 0)
    assert bool(got[rest].isfinite().all())


def test_two_streams_at_once(moe):
    """Calls in flight on two streams, each with its own workspace, beside a norm's gradient: as one after the other."""
    sets = [{n: v.cuda() for n, v in make(T, 1024, 2056, 64, 6, T).items()} for T in (3000, 1700)]
    assert all(sorts(moe, T, 1024, 2056, 64, 6) for T in (3000, 1700))
    h = torch.randn(2000, 1024, device="cuda").to(torch.bfloat16)
    w = torch.rand(1024, device="cuda")
    call = lambda c, **k: moe.moe_lora(c["x"], c["a"], c["b"], c["ids"], scale=c["scale"], base=c["base"], **k)  # noqa: E731
    refs, norm = [call(c) for c in sets], moe.moe_prenorm_backward(h, h, w)
    torch.cuda.synchronize()
    sides, got, norms = [torch.cuda.Stream() for _ in sets], ([], []), []
    for _ in range(10):
        for i, side in enumerate(sides):
            with torch.cuda.stream(side):
                got[i].append(call(sets[i]))
                norms.append(moe.moe_prenorm_backward(h, h, w))
    torch.cuda.synchronize()
    assert all(torch.equal(v, ref) for outs, ref in zip(got, refs) for v in outs)
    assert all(torch.equal(a, b) for n in norms for a, b in zip(n, norm))
    assert moe.moe_get_status() == 0
