"""Norms before and after a block and their gradients, against the formulas in 64 bits and against differences.

Tolerances: each fp32 step is one rounding of 2^-24; a row's sum takes at most 16 + 10 of them on positive terms, the
reciprocal root two, and a result three such sums at most, so each is within FUZZ = 2^-17 of the formula evaluated
with absolute values (times the cancellation of out, where its norm follows), plus half a step of its type."""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FUZZ = 2.0 ** -17
EPS = 1e-6


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


def within(got, ref, tol, what):
    got, ref, tol = got.double().cpu(), ref.detach().double().cpu(), tol.detach().double().cpu()
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got - ref).abs() - tol).max())}"


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rstd(v, eps=EPS):
    return ((v * v).mean(1, keepdim=True) + eps) ** -0.5


def mean(v):
    return v.mean(1, keepdim=True)


class Ref:
    """The formulas in 64 bits, each with its magnitude (absolute values through the same steps)."""

    def __init__(self, x, y, post_w, gate, sigmoid, scale, res, next_w, d_out, d_h):
        x, y, post_w, gate, next_w, d_out, d_h = (None if v is None else v.double()
                                                  for v in (x, y, post_w, gate, next_w, d_out, d_h))
        G = torch.ones(1, 1, dtype=torch.float64) if gate is None else torch.sigmoid(gate) if sigmoid else gate
        ry = rstd(y) if post_w is not None else torch.ones(1, 1, dtype=torch.float64)
        pw = post_w if post_w is not None else torch.ones(1, 1, dtype=torch.float64)
        n, v = y * ry, y * ry * pw
        self.out, mo = res * x + scale * G * v, (res * x).abs() + (scale * G * v).abs()
        self.out_m = mo
        D, mD = torch.zeros_like(x), torch.zeros_like(x)
        if d_out is not None:
            D, mD = D + d_out, mD + d_out.abs()
        self.d_next_w = self.d_next_w_m = self.h = None
        if next_w is not None:
            ro = rstd(self.out)
            # out's own error, relative to its row's norm
            amp = 1 + (mo.norm(dim=1, keepdim=True) / self.out.norm(dim=1, keepdim=True).clamp(min=1e-300))
            self.h = self.out * ro * next_w
            self.h_m = mo * ro * next_w.abs() * amp
            if d_h is not None:
                g, no, mn = d_h * next_w, self.out * ro, mo * ro
                D = D + ro * (g - no * mean(g * no))
                mD = mD + ro * amp * amp * (g.abs() + mn * mean(g.abs() * mn))
                self.d_next_w, self.d_next_w_m = (d_h * no).sum(0), (d_h.abs() * mn * amp).sum(0)
            else:
                self.d_next_w = self.d_next_w_m = torch.zeros_like(next_w)
        self.d_x, self.d_x_m = res * D, abs(res) * mD
        dv, mdv = scale * D * G, abs(scale) * mD * G.abs()
        dG, mdG = scale * D * v, abs(scale) * mD * v.abs()
        if sigmoid and gate is not None:
            dG, mdG = dG * G * (1 - G), mdG * G
        self.d_gate = self.d_gate_m = None
        if gate is not None:
            if gate.dim() == 1:
                self.d_gate, self.d_gate_m = dG.sum(0), mdG.sum(0)
            elif gate.shape[1] == 1:
                self.d_gate, self.d_gate_m = dG.sum(1, keepdim=True), mdG.sum(1, keepdim=True)
            else:
                self.d_gate, self.d_gate_m = dG, mdG
        self.d_post_w = self.d_post_w_m = None
        if post_w is not None:
            self.d_post_w, self.d_post_w_m = (dv * n).sum(0), (mdv * n.abs()).sum(0)
            g, mg = dv * pw, mdv * pw.abs()
            dv, mdv = ry * (g - n * mean(g * n)), ry * (mg + n.abs() * mean(mg * n.abs()))
        self.d_y, self.d_y_m = dv, mdv


def inputs(T, H, dt, wd, g, post, gate, nxt, gdt=None):
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gate]
    return dict(x=r(T, H).to(dt), y=(r(T, H) * 3).to(dt), post_w=(1 + r(H) / 4).to(wd) if post else None,
                gate=None if shape is None else r(*shape).to(gdt or dt), next_w=(1 + r(H) / 4).to(wd) if nxt else None,
                d_out=r(T, H).to(dt), d_h=r(T, H).to(dt) if nxt else None)


def cuda(v):
    return None if v is None else v.cuda()


def check_all(moe, d, sigmoid, scale, res, what, T, eps=EPS):
    args = {n: d[n] for n in ("x", "y", "post_w", "gate", "next_w")}
    ref = Ref(d["x"], d["y"], d["post_w"], d["gate"], sigmoid, scale, res, d["next_w"], d["d_out"], d["d_h"])
    dt = d["x"].dtype
    kw = dict(post_w=cuda(args["post_w"]), gate=cuda(args["gate"]), sigmoid=sigmoid, scale=scale, res_scale=res,
              next_w=cuda(args["next_w"]), eps=eps)
    out, h = moe.moe_postnorm(d["x"].cuda(), d["y"].cuda(), **kw)
    within(out, ref.out, half(dt) * ref.out.abs() + FUZZ * ref.out_m, what + " out")
    assert (h is None) == (d["next_w"] is None)
    if h is not None:
        within(h, ref.h, half(dt) * ref.h.abs() + FUZZ * ref.h_m, what + " h")
    gr = moe.moe_postnorm_backward(cuda(d["d_out"]), cuda(d["d_h"]), d["x"].cuda(), d["y"].cuda(), **kw)
    for name in ("d_x", "d_y", "d_post_w", "d_gate", "d_next_w"):
        got, r = getattr(gr, name), getattr(ref, name)
        assert (got is None) == (r is None), what + name
        if got is None:
            continue
        m = getattr(ref, name + "_m")
        # (sums over tokens: one fp32 addition more for each of them)
        fuzz = FUZZ + (T * 2.0 ** -24 if r.dim() == 1 else 0.0)
        within(got, r, half(got.dtype) * r.abs() + fuzz * m, f"{what} {name}")
    assert moe.moe_get_status() == 0


SIZES = [(1, 1), (2, 7), (5, 64), (3, 130), (33, 1000), (7, 2047), (4, 4096), (3, 4104), (2, 5001), (2, 8192), (2, 16384),
         (700, 96)]


@pytest.mark.parametrize("dtype,wide", [("bf16", False), ("bf16", True), ("f32", True), ("f32", False)])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(moe, size, dtype, wide):
    T, H = size
    g = torch.Generator().manual_seed(T * 7 + H)
    wd = torch.float32 if wide else torch.bfloat16
    d = inputs(T, H, DT[dtype], wd, g, True, "channel", True)
    check_all(moe, d, False, 0.5, 1.25, f"{size} {dtype}", T)
    x, w, dh = d["x"], d["next_w"], d["d_h"]
    h = moe.moe_prenorm(x.cuda(), w.cuda(), EPS)
    ref = x.double() * rstd(x.double()) * w.double()
    within(h, ref, (half(DT[dtype]) + FUZZ) * ref.abs(), "prenorm")
    d_x, d_w = moe.moe_prenorm_backward(dh.cuda(), x.cuda(), w.cuda(), EPS)
    r = rstd(x.double())
    n, gg = x.double() * r, dh.double() * w.double()
    ref = r * (gg - n * mean(gg * n))
    within(d_x, ref, half(DT[dtype]) * ref.abs() + FUZZ * r * (gg.abs() + n.abs() * mean((gg * n).abs())), "d_x")
    within(d_w, (dh.double() * n).sum(0), (FUZZ + T * 2.0 ** -24) * (dh.double() * n).abs().sum(0), "d_w")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post,nxt", list(itertools.product([False, True], [False, True])))
def test_forms(moe, post, nxt, gate, sigmoid):
    g = torch.Generator().manual_seed(3)
    for (T, H), (dt, gdt) in (((19, 264), (torch.bfloat16, torch.bfloat16)), ((6, 99), (torch.bfloat16, torch.float32)),
                              ((9, 520), (torch.float32, torch.bfloat16))):
        d = inputs(T, H, dt, torch.float32, g, post, gate, nxt, gdt)
        check_all(moe, d, sigmoid, 0.7, -1.5, f"{T} x {H} {dt}", T)
        for gone in ("d_out", "d_h"):  # a gradient that is not there is zero
            check_all(moe, {**d, gone: None}, sigmoid, 0.7, 1.0, f"{T} x {H} {dt} without {gone}", T)


def test_gradients_against_differences(moe):
    """Every gradient against differences of the 64-bit loss (central, step 1e-5: error about 1e-9 of the third
    derivative; the kernel's own is fp32)."""
    T, H = 3, 24
    g = torch.Generator().manual_seed(11)
    for gate, sigmoid in (("channel", True), ("token", False), ("full", True)):
        d = inputs(T, H, torch.float32, torch.float32, g, True, gate, True)

        def loss(v):
            r = Ref(v["x"], v["y"], v["post_w"], v["gate"], sigmoid, 0.7, 1.5, v["next_w"], None, None)
            return float((r.out * d["d_out"].double()).sum() + (r.h * d["d_h"].double()).sum())

        gr = moe.moe_postnorm_backward(cuda(d["d_out"]), cuda(d["d_h"]), cuda(d["x"]), cuda(d["y"]),
                                       post_w=cuda(d["post_w"]), gate=cuda(d["gate"]), sigmoid=sigmoid, scale=0.7,
                                       res_scale=1.5, next_w=cuda(d["next_w"]), eps=EPS)
        for leaf, grad in (("x", gr.d_x), ("y", gr.d_y), ("post_w", gr.d_post_w), ("gate", gr.d_gate),
                           ("next_w", gr.d_next_w)):
            flat = grad.flatten().cpu()
            for i in range(0, flat.numel(), 7):
                side = []
                for s in (1e-5, -1e-5):
                    v = {n: None if t is None else t.double().clone() for n, t in d.items()}
                    v[leaf].view(-1)[i] += s
                    side.append(loss(v))
                assert abs((side[0] - side[1]) / 2e-5 - float(flat[i])) < 2e-4, (gate, leaf, i)


def test_in_place_zero_rows_and_special_values(moe):
    T, H = 6, 512
    g = torch.Generator().manual_seed(2)
    d = {n: cuda(v) for n, v in inputs(T, H, torch.bfloat16, torch.bfloat16, g, True, "full", True).items()}
    kw = dict(post_w=d["post_w"], gate=d["gate"], next_w=d["next_w"], eps=EPS)
    out, h = moe.moe_postnorm(d["x"], d["y"], **kw)
    x, y = d["x"].clone(), d["y"].clone()
    o2, h2 = moe.moe_postnorm(x, y, out=x, h=y, **kw)
    assert o2 is x and h2 is y and torch.equal(x, out) and torch.equal(y, h)
    gr = moe.moe_postnorm_backward(d["d_out"], d["d_h"], d["x"], d["y"], **kw)
    d_out, d_h = d["d_out"].clone(), d["d_h"].clone()
    g2 = moe.moe_postnorm_backward(d_out, d_h, d["x"], d["y"], d_x=d_out, d_y=d_h, **kw)
    assert all(torch.equal(a, b) for a, b in zip(gr, g2))
    # rows of zeros: eps keeps the norm finite
    zero = torch.zeros(2, H, device="cuda")
    w = torch.ones(H, device="cuda")
    assert (moe.moe_prenorm(zero, w, EPS) == 0).all()
    d_x, _ = moe.moe_prenorm_backward(torch.ones_like(zero), zero, w, EPS)
    assert torch.allclose(d_x, torch.full_like(d_x, 1e3), rtol=1e-6)
    # a NaN or an infinity stays in its row
    x = torch.randn(4, H, generator=g).cuda()
    ref = moe.moe_prenorm(x, w, EPS)
    bad = x.clone()
    bad[1, 5], bad[2, 7] = float("nan"), float("inf")
    got = moe.moe_prenorm(bad, w, EPS)
    assert torch.equal(got[[0, 3]], ref[[0, 3]]) and got[1].isnan().all() and got[2, 7].isnan()
    assert (got[2, :7] == 0).all()


def test_empty_batch(moe):
    H = 64
    x, w = torch.zeros(0, H, device="cuda"), torch.ones(H, device="cuda")
    assert moe.moe_prenorm(x, w).shape == (0, H)
    out, h = moe.moe_postnorm(x, x, post_w=w, gate=w, next_w=w)
    assert out.shape == h.shape == (0, H)
    d_w = torch.full((H,), 3.0, device="cuda")
    d_x, got = moe.moe_prenorm_backward(x, x, w, d_w=d_w)
    assert got is d_w and (d_w == 0).all()
    gr = moe.moe_postnorm_backward(x, x, x, x, post_w=w, gate=w, next_w=w)
    assert all((v == 0).all() for v in (gr.d_post_w, gr.d_gate, gr.d_next_w)) and gr.d_y.shape == (0, H)
    assert moe.moe_get_status() == 0


@pytest.mark.parametrize("T,H", [(20000, 64), (5000, 4096)])
def test_long_batches_repeat(moe, T, H):
    """Many rows to a CTA; sums over them are the same bits on every call, and a captured call's too."""
    g = torch.Generator().manual_seed(T)
    d = inputs(T, H, torch.bfloat16, torch.float32, g, True, "token", True)
    check_all(moe, d, True, 1.0, 1.0, f"{T} x {H}", T)
    c = {n: cuda(v) for n, v in d.items()}
    kw = dict(post_w=c["post_w"], gate=c["gate"], sigmoid=True, next_w=c["next_w"], eps=EPS)
    ws = torch.empty(moe.moe_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda").fill_(255)
    a = moe.moe_postnorm_backward(c["d_out"], c["d_h"], c["x"], c["y"], workspace=ws, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = moe.moe_postnorm_backward(c["d_out"], c["d_h"], c["x"], c["y"], workspace=ws, **kw)
        o = moe.moe_postnorm(c["x"], c["y"], **kw)
    graph.replay()
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert all(torch.equal(u, v) for u, v in zip(o, moe.moe_postnorm(c["x"], c["y"], **kw)))


def test_other_stream(moe):
    g = torch.Generator().manual_seed(1)
    c = {n: cuda(v) for n, v in inputs(300, 1024, torch.bfloat16, torch.float32, g, True, "channel", True).items()}
    kw = dict(post_w=c["post_w"], gate=c["gate"], next_w=c["next_w"], eps=EPS)
    ref = moe.moe_postnorm_backward(c["d_out"], c["d_h"], c["x"], c["y"], **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(50_000_000)  # the current stream is busy: nothing of the call may wait there
    got = moe.moe_postnorm_backward(c["d_out"], c["d_h"], c["x"], c["y"], stream=side, **kw)
    side.synchronize()
    with torch.cuda.stream(side):
        assert all(bool(torch.equal(a, b)) for a, b in zip(got, ref))
    torch.cuda.synchronize()


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(6000, 512), (700, 1024), (500, 4096), (400, 8192), (700, 2047), (2500, 33), (6000, 8), (450, 4160)])
def test_rows_through_the_ring(moe, T, H, dtype, gate):
    """More rows than CTAs: rows that every thread holds whole vectors of, and others; rows that begin off a
    16-byte boundary; the last rows of a tensor."""
    g = torch.Generator().manual_seed(T + H)
    d = inputs(T, H, DT[dtype], torch.float32, g, True, gate, True)
    check_all(moe, d, gate == "full", 0.5, 1.25, f"{T} x {H} {dtype} {gate}", T)
    x, w, dh = d["x"].cuda(), d["next_w"].cuda(), d["d_h"].cuda()
    r = rstd(d["x"].double())
    n, gg = d["x"].double() * r, d["d_h"].double() * d["next_w"].double()
    within(moe.moe_prenorm(x, w, EPS), n * d["next_w"].double(), (half(DT[dtype]) + FUZZ) * (n * d["next_w"].double()).abs(), "h")
    d_x, d_w = moe.moe_prenorm_backward(dh, x, w, EPS)
    ref = r * (gg - n * mean(gg * n))
    within(d_x, ref, half(DT[dtype]) * ref.abs() + FUZZ * r * (gg.abs() + n.abs() * mean((gg * n).abs())), "d_x")
    within(d_w, (d["d_h"].double() * n).sum(0), (FUZZ + T * 2.0 ** -24) * (d["d_h"].double() * n).abs().sum(0), "d_w")


@pytest.mark.parametrize("T,H", [(3, 256), (900, 2048)])
def test_residual_that_cancels(moe, T, H):
    """Rows whose residual and branch nearly cancel: out is small beside them, and so is the sum of its squares."""
    g = torch.Generator().manual_seed(T)
    for small in (1e-1, 1e-3):
        d = inputs(T, H, torch.float32, torch.float32, g, False, "none", True)
        d["x"] = small * d["x"] - 0.5 * d["y"]
        check_all(moe, d, False, 0.5, 1.0, f"{small}", T, eps=EPS)
        d = inputs(T, H, torch.float32, torch.float32, g, True, "token", True)
        n = d["y"].double() * rstd(d["y"].double()) * d["post_w"].double()
        d["x"] = (small * d["x"].double() - d["gate"].double() * n).float()
        check_all(moe, d, False, 1.0, 1.0, f"normed {small}", T, eps=EPS)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(9, 16383), (170, 8190), (9, 8187), (330, 8179), (350, 4093), (5000, 5), (13, 3)])
def test_rows_that_share_units(moe, T, H, dtype):
    """Rows that begin and end inside a 16-byte unit, with the neighbours' elements around them: the longest, those at
    the turn from one form to the next, and rows of less than one unit."""
    g = torch.Generator().manual_seed(T + H)
    for gate in ("channel", "full"):
        check_all(moe, inputs(T, H, DT[dtype], torch.float32, g, True, gate, True), gate == "full", 0.5, 1.25, f"{T} x {H} {gate}", T)


@pytest.mark.parametrize("T,H", [(11, 1023), (700, 2045), (3000, 6)])
def test_bad_values_stay_in_their_row(moe, T, H):
    """NaN and infinities in every third row reach no other row's results."""
    g = torch.Generator().manual_seed(T)
    d = {n: cuda(v) for n, v in inputs(T, H, torch.bfloat16, torch.float32, g, True, "full", True).items()}
    kw = dict(post_w=d["post_w"], sigmoid=True, next_w=d["next_w"], eps=EPS)
    bad = {n: d[n].clone() for n in ("x", "y", "gate", "d_out", "d_h")}
    for i, n in enumerate(("x", "y", "d_out", "d_h")):
        bad[n][i % 3::3] = float("nan") if i % 2 else float("inf")
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[i % 3::3] = False
        new = {**{k: d[k] for k in bad}, n: bad[n]}
        for a, b in zip(moe.moe_postnorm(d["x"], d["y"], gate=d["gate"], **kw),
                        moe.moe_postnorm(new["x"], new["y"], gate=new["gate"], **kw)):
            assert torch.equal(a[keep], b[keep])
        ga = moe.moe_postnorm_backward(d["d_out"], d["d_h"], d["x"], d["y"], gate=d["gate"], **kw)
        gb = moe.moe_postnorm_backward(new["d_out"], new["d_h"], new["x"], new["y"], gate=new["gate"], **kw)
        for k in ("d_x", "d_y", "d_gate"):
            assert torch.equal(getattr(ga, k)[keep], getattr(gb, k)[keep]), (n, k)
    assert moe.moe_get_status() == 0


@pytest.mark.parametrize("T,H", [(3, 512), (400, 4096), (330, 2047)])
def test_block_output_of_any_size(moe, T, H):
    """out is of ordinary size, but y post_w gate, before its norm, is not: its squares leave fp32's range."""
    g = torch.Generator().manual_seed(T)
    d = inputs(T, H, torch.float32, torch.float32, g, True, "channel", True)
    d["y"], d["post_w"], d["gate"] = d["y"] * 2.0 ** 50, d["post_w"] * 2.0 ** 10, d["gate"] * 2.0 ** 10
    check_all(moe, d, False, 2.0 ** -20, 1.25, "large", T)
    # a norm without eps of a small output: squares below fp32's range (2^-149) where its own are not
    d = inputs(T, H, torch.float32, torch.float32, g, True, "channel", True)
    d["y"], d["post_w"] = d["y"] * 2.0 ** -56, d["post_w"] * 2.0 ** -30
    d["x"] = d["x"] * 2.0 ** -30
    out, h = moe.moe_postnorm(*(cuda(d[n]) for n in ("x", "y", "post_w", "gate")), next_w=cuda(d["next_w"]), eps=0.0)
    x, y = d["x"].double(), d["y"].double()
    branch = d["gate"].double() * d["post_w"].double() * y * rstd(y, 0.0)
    ref = x + branch
    mag = x.abs() + branch.abs()
    within(out, ref, half(torch.float32) * ref.abs() + FUZZ * mag, "small out")
    r = rstd(ref, 0.0) * d["next_w"].double()
    # (1 / rms moves with the sum of out^2: by its relative error, FUZZ times mean(mag^2) / mean(out^2))
    within(h, ref * r, half(torch.float32) * (ref * r).abs() + FUZZ * (mag * r.abs() + (ref * r).abs() * mean(mag * mag) / mean(ref * ref)), "small h")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(700, 5120), (400, 4104), (9, 5112), (330, 4128)])
def test_prenorm_gradient_of_two_ctas(moe, T, H, dtype):
    """Widths at which the prenorm's gradient holds its registers to two CTAs of an SM."""
    g = torch.Generator().manual_seed(T + H)
    x, w, dh = torch.randn(T, H, generator=g).to(DT[dtype]), 1 + torch.randn(H, generator=g) / 4, torch.randn(T, H, generator=g).to(DT[dtype])
    d_x, d_w = moe.moe_prenorm_backward(dh.cuda(), x.cuda(), w.cuda(), EPS)
    r = rstd(x.double())
    n, gg = x.double() * r, dh.double() * w.double()
    ref = r * (gg - n * mean(gg * n))
    within(d_x, ref, half(DT[dtype]) * ref.abs() + FUZZ * r * (gg.abs() + n.abs() * mean((gg * n).abs())), "d_x")
    within(d_w, (dh.double() * n).sum(0), (FUZZ + T * 2.0 ** -24) * (dh.double() * n).abs().sum(0), "d_w")
    assert moe.moe_get_status() == 0
