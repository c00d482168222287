"""Rows in expert order and back, and their gradients, against plain 64-bit forms.

Tolerances: a result rounded once is off by half a step (eps / 2 of its type, relative); a sum of n fp32 products in
any order by at most n + 1 more roundings of 2^-24, relative to the sum of the products' sizes."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


def ids_for(T, E, k, g, repeat=False):
    if repeat:
        return torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    return torch.rand(T, E, generator=g).topk(k, 1)[1].to(torch.int32)


def places(ids, E, block):
    """(row of each pair, padded length) by hand."""
    row, at = np.full(ids.shape, -1), 0
    for e in range(E):
        for t, j in zip(*np.nonzero(ids == e)):
            row[t, j] = at
            at += 1
        at = -(-at // block) * block
    return row, at


def within(got, ref, tol, what=""):
    got, ref = got.double().cpu(), ref.double().cpu()
    bad = (got - ref).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got - ref).abs() - tol).max())}"


def half(dtype):
    return torch.finfo(dtype).eps / 2


# T, H, E, k, block
SHAPES = [(1, 1, 1, 1, 1), (1, 128, 8, 2, 16), (3, 7, 4, 3, 1), (16, 2048, 128, 8, 16), (33, 66, 8, 2, 5),
          (64, 1000, 40, 6, 64), (129, 4096, 8, 2, 128), (700, 260, 64, 8, 1), (1500, 33, 300, 4, 16),
          (5, 16392, 16, 4, 1), (3, 64, 64, 40, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_permute(moe, shape, dtype):
    T, H, E, k, block = shape
    g = torch.Generator().manual_seed(T * H + k)
    x, ids = torch.randn(T, H, generator=g).to(DT[dtype]), ids_for(T, E, k, g)
    cap, _ = moe.moe_align_capacity(T, k, E, block)
    rows = torch.full((cap, H), 7.0, dtype=DT[dtype], device="cuda")
    p = moe.moe_permute(x.cuda(), ids.cuda(), E, block, rows=rows)
    assert moe.moe_get_status() == 0 and p.rows is rows
    row, n = places(ids.numpy(), E, block)
    assert np.array_equal(p.row_of.cpu().numpy(), row)
    ref = torch.zeros(cap, H, dtype=DT[dtype])
    ref[torch.from_numpy(row)] = x[:, None, :].expand(T, k, H)
    ref[n:] = 7.0
    assert torch.equal(rows.cpu(), ref)
    s, e, npp, c = moe.moe_align(ids.cuda(), E, block)
    assert int(p.num_post_pad) == int(npp) == n
    assert torch.equal(p.sorted_ids[:n], s[:n]) and torch.equal(p.expert_ids[: n // block], e[: n // block])
    assert torch.equal(p.expert_counts, c)


@pytest.mark.parametrize("T,k,E", [(40, 3, 8), (500, 4, 16), (3, 2, 4)])
def test_ids_out_of_range_and_repeated(moe, T, k, E):
    """Pairs without an expert have no row; a token that names an expert twice has two."""
    g = torch.Generator().manual_seed(T)
    x, ids = torch.randn(T, 96, generator=g), ids_for(T, E, k, g, repeat=True)
    bad = torch.rand(T, k, generator=g) < 0.2
    bad[0] = True  # (a token with no row at all)
    bad[1, 0] = False
    ids[bad] = torch.tensor([-1, E, -7, 1 << 30], dtype=torch.int32)[torch.arange(int(bad.sum())) % 4]
    cap = moe.moe_align_capacity(T, k, E, 4)[0]
    p = moe.moe_permute(x.cuda(), ids.cuda(), E, 4, rows=torch.full((cap, 96), 7.0, device="cuda"))
    assert moe.moe_get_status() == moe.MOE_ERR_DEVICE_INDEX
    row, n = places(ids.numpy(), E, 4)
    assert np.array_equal(p.row_of.cpu().numpy(), row) and int(p.num_post_pad) == n
    ref = torch.zeros(cap, 96)
    ref[n:] = 7.0
    ok = row >= 0
    ref[torch.from_numpy(row[ok])] = x[torch.from_numpy(np.nonzero(ok)[0])]
    assert torch.equal(p.rows.cpu(), ref)
    w = torch.rand(T, k, generator=g)
    rows = torch.randn(cap, 96, generator=g)
    out = moe.moe_unpermute(rows.cuda(), p.row_of, w.cuda())
    sel = torch.where(torch.from_numpy(ok), w, 0.0).double()
    terms = sel[:, :, None] * rows.double()[torch.from_numpy(row.clip(0))]
    within(out, terms.sum(1), (k + 2) * 2.0 ** -24 * terms.abs().sum(1))
    assert (out[0] == 0).all()
    d_out = torch.randn(T, 96, generator=g)
    buf = torch.full((cap, 96), 7.0, device="cuda")
    d_rows, d_w = moe.moe_unpermute_backward(d_out.cuda(), rows.cuda(), p.row_of, w.cuda(), sorted_ids=p.sorted_ids,
                                             num_post_pad=p.num_post_pad, d_rows=buf)
    assert (d_w.cpu()[~torch.from_numpy(ok)] == 0).all()
    used = torch.zeros(cap, dtype=torch.bool)
    used[torch.from_numpy(row[ok])] = True
    assert (d_rows.cpu()[:n][~used[:n]] == 0).all() and (d_rows.cpu()[n:] == 7.0).all()
    # row numbers past the buffer count as none as well: nothing is read or written there
    m = n // 2
    short = moe.moe_unpermute(rows[:m].contiguous().cuda(), p.row_of, w.cuda())
    sel = torch.where(torch.from_numpy(ok & (row < m)), w, 0.0).double()
    terms = sel[:, :, None] * rows.double()[torch.from_numpy(row.clip(0))]
    within(short, terms.sum(1), (k + 2) * 2.0 ** -24 * terms.abs().sum(1))
    assert moe.moe_get_status() == 0


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_back_and_gradients(moe, shape, dtype, weighted):
    T, H, E, k, block = shape
    dt = DT[dtype]
    g = torch.Generator().manual_seed(T * H + k + 1)
    ids = ids_for(T, E, k, g)
    row, n = places(ids.numpy(), E, block)
    at = torch.from_numpy(row)
    cap = moe.moe_align_capacity(T, k, E, block)[0]
    rows, d_out = torch.randn(cap, H, generator=g).to(dt), torch.randn(T, H, generator=g).to(dt)
    w = torch.randn(T, k, generator=g) if weighted else None
    w64 = (w.double() if weighted else torch.ones(T, k, dtype=torch.float64))[:, :, None]
    p = moe.moe_permute(d_out.cuda(), ids.cuda(), E, block)
    cw = w.cuda() if weighted else None
    out = moe.moe_unpermute(rows.cuda(), p.row_of, cw)
    terms = w64 * rows.double()[at]
    ref = terms.sum(1)
    fuzz = (k + 2) * 2.0 ** -24
    within(out, ref, half(dt) * ref.abs() + fuzz * terms.abs().sum(1), "out")
    d_x = moe.moe_permute_backward(rows.cuda(), p.row_of)
    terms = rows.double()[at]
    within(d_x, terms.sum(1), half(dt) * terms.sum(1).abs() + fuzz * terms.abs().sum(1), "d_x")
    buf = torch.full((cap, H), 7.0, dtype=dt, device="cuda")
    d_rows, d_w = moe.moe_unpermute_backward(d_out.cuda(), rows.cuda(), p.row_of, cw, sorted_ids=p.sorted_ids,
                                             num_post_pad=p.num_post_pad, d_rows=buf)
    ref = torch.zeros(cap, H, dtype=torch.float64)
    ref[n:] = 7.0
    ref[at] = w64 * d_out.double()[:, None, :]
    within(d_rows, ref, half(dt) * ref.abs(), "d_rows")  # (one product of fp32 weight and value, one rounding)
    terms = rows.double()[at] * d_out.double()[:, None, :]
    within(d_w, terms.sum(2), (H + 1) * 2.0 ** -24 * terms.abs().sum(2), "d_w")
    assert moe.moe_get_status() == 0
    # each gradient alone gives the same, and d_rows may take the place of rows
    lib, s = moe.lib(), moe._stream(None)
    only = torch.zeros_like(d_w)
    rr = rows.cuda()
    dd = d_out.cuda()
    assert lib.moe_unpermute_backward(dd.data_ptr(), rr.data_ptr(), cap, p.row_of.data_ptr(), moe._p(cw), None, None, T, H,
                                      k, moe._dt(rr), None, only.data_ptr(), s) == 0
    assert torch.equal(only, d_w)
    same, w2 = moe.moe_unpermute_backward(dd, rr, p.row_of, cw, d_rows=rr)
    assert torch.equal(same[at.cuda()], d_rows[at.cuda()]) and torch.equal(w2, d_w)


def test_gradients_against_differences(moe):
    """d_x, d_rows and d_w of permute, a product per expert and unpermute, against differences of a 64-bit form."""
    T, H, E, k = 6, 16, 4, 2
    g = torch.Generator().manual_seed(5)
    x, ids, w = torch.randn(T, H, generator=g), ids_for(T, E, k, g), torch.rand(T, k, generator=g)
    m, d_out = torch.randn(E, H, H, generator=g) / 4, torch.randn(T, H, generator=g)

    def loss(x, w):
        y = torch.einsum("tkhg,tg->tkh", m.double()[ids.long()], x)
        return float(((w[:, :, None] * y).sum(1) * d_out.double()).sum())

    p = moe.moe_permute(x.cuda(), ids.cuda(), E)
    e = p.expert_ids.long()
    y = torch.einsum("rhg,rg->rh", m.cuda()[e], p.rows)
    d_y, d_w = moe.moe_unpermute_backward(d_out.cuda(), y, p.row_of, w.cuda())
    d_x = moe.moe_permute_backward(torch.einsum("rhg,rh->rg", m.cuda()[e], d_y), p.row_of)
    for leaf, grad in ((x, d_x), (w, d_w)):
        for i in range(0, leaf.numel(), 5):
            step = torch.zeros(leaf.numel(), dtype=torch.float64)
            step[i] = 1e-4
            step = step.view(leaf.shape)
            args = [(x.double(), w.double()), (x.double(), w.double())]
            sides = [loss(*((v + s * step) if v.shape == leaf.shape else v for v in a)) for a, s in zip(args, (1, -1))]
            # (the loss is linear in each leaf: the difference is exact to 64 bits; the products are fp32)
            assert abs((sides[0] - sides[1]) / 2e-4 - float(grad.flatten()[i])) < 1e-4


def test_special_values_and_empty(moe):
    x = torch.tensor([[float("inf"), 1.0, -0.0, float("nan")], [1e-40, -float("inf"), 3e38, 2.0]], device="cuda")
    ids = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda")
    p = moe.moe_permute(x, ids, 2)
    assert torch.equal(p.rows.view(torch.int32), x.flip(0).view(torch.int32))
    back = moe.moe_unpermute(p.rows, p.row_of)
    assert torch.equal(back.nan_to_num(5.0), x.nan_to_num(5.0))
    # a row without a pair is not touched by a NaN elsewhere
    none = torch.full((2, 1), -1, dtype=torch.int32, device="cuda")
    assert (moe.moe_unpermute(torch.full((2, 4), float("nan"), device="cuda"), none) == 0).all()
    e = moe.moe_permute(x[:0], ids[:0], 2, 16)
    assert e.rows.shape == (0, 4) and int(e.num_post_pad) == 0 and (e.expert_counts == 0).all()
    assert moe.moe_unpermute(p.rows, ids[:0]).shape == (0, 4)
    assert (moe.moe_unpermute(p.rows[:0], none) == 0).all()
    d, w = moe.moe_unpermute_backward(x[:0], p.rows, ids[:0])
    assert d.shape == (2, 4) and w.shape == (0, 1)
    assert moe.moe_get_status() == 0


def test_rows_past_32_bits(moe):
    """Offsets of more than 2^32 bytes, and of more than 2^31 elements."""
    H, T, k = 16384, 70000, 2
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, ::4096] = torch.arange(T, device="cuda")[:, None].remainder(251).to(torch.bfloat16)
    ids = torch.stack([torch.arange(T, device="cuda") % 4, torch.full((T,), 5, device="cuda")], 1).to(torch.int32)
    p = moe.moe_permute(x, ids, 6)
    assert p.rows.numel() > 2 ** 31
    t = torch.tensor([0, 1, 34567, T - 1], device="cuda")
    assert torch.equal(p.rows[p.row_of[t].long()], x[t][:, None].expand(4, 2, H))
    back = moe.moe_unpermute(p.rows, p.row_of, torch.full((T, k), 0.5, device="cuda"))
    assert torch.equal(back, x)
    del back
    d, w = moe.moe_unpermute_backward(x, p.rows, p.row_of, None, d_rows=p.rows)
    assert torch.equal(d[p.row_of[t].long()], x[t][:, None].expand(4, 2, H))
    ref = (x[t].double() ** 2).sum(1, keepdim=True).expand(4, 2)
    assert ((w[t].double() - ref).abs() <= 2.0 ** -10 * ref).all()  # (16385 roundings of 2^-24)


def test_graph_replay_and_side_stream(moe):
    """A captured pass, replayed on new inputs, and a call on a stream beside the current one."""
    T, H, E, k = 200, 320, 16, 4
    g = torch.Generator().manual_seed(9)
    sets = [(torch.randn(T, H, generator=g).to(torch.bfloat16).cuda(), ids_for(T, E, k, g).cuda(),
             torch.rand(T, k, generator=g).cuda()) for _ in range(3)]

    def step(x, ids, w):
        p = moe.moe_permute(x, ids, E, 16)
        out = moe.moe_unpermute(p.rows, p.row_of, w)
        d_rows, d_w = moe.moe_unpermute_backward(x, p.rows, p.row_of, w, sorted_ids=p.sorted_ids,
                                                 num_post_pad=p.num_post_pad)
        return out, d_w, moe.moe_permute_backward(d_rows, p.row_of)

    refs = [[t.clone() for t in step(*s)] for s in sets]
    torch.cuda.synchronize()
    ins = [t.clone() for t in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*ins)
    for s, ref in zip(sets, refs):
        for a, b in zip(ins, s):
            a.copy_(b)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    x, ids, w = sets[1]
    p = moe.moe_permute(x, ids, E, 16, stream=side)
    out = moe.moe_unpermute(p.rows, p.row_of, w, stream=side)
    side.synchronize()
    assert torch.equal(out, refs[1][0]) and moe.moe_get_status() == 0


# short rows off the 16-byte grid in great number; few pairs of long rows; padding in plenty
MORE = [(900, 13, 16, 3, 4), (1300, 109, 64, 2, 16), (700, 235, 8, 4, 1), (2500, 1, 4, 1, 1), (30, 2056, 8, 4, 1),
        (9, 4133, 300, 8, 16), (1, 8195, 4, 1, 64), (20, 1028, 200, 3, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", MORE)
def test_forms_by_size(moe, shape, dtype):
    test_permute(moe, shape, dtype)
    test_back_and_gradients(moe, shape, dtype, True)
