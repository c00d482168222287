"""Block-scaled FP8 operators against plain 64-bit forms: quantisation by blocks, the matrix
product, and the expert layer on them.

Tolerances.
 Quantisation: the definition takes the scale, its reciprocal and the product as 32-bit numbers, so
 codes and scales of given values are compared bit for bit.  The SiLU form computes its values h in
 32 bits first (exp, a sum, a division, a product: a few 2^-23 together, under 1e-6), so its scales
 are within 1e-6 and every code stands within half a code step, plus 2e-6 of h, of h / scale.
 Products: products of e4m3 codes are exact.  A tensor-core instruction adds 32 of them to a 32-bit
 sum: at most 33 terms each cut at 2^-24 of the largest, four instructions a block: under 2^-17 of
 S = sum |a| |w|; scaling and adding the K / 128 blocks adds (K / 128 + 2) 2^-24 of S.  A bf16 output
 adds half an ulp.
 Expert layer: where an intermediate lies that close to the border of two codes it may take the
 other one.  Such a change moves an output by far less than the FP8 layer's bar (6e-2 of the RMS), and
 they are rare enough to stay inside 5e-3 in the 2-norm together with the bf16 rounding (2^-9).
"""
import numpy as np
import pytest
import torch

from helpers import assert_parity, bf16_half_ulp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_scan_gb300 as m

    assert torch.cuda.is_available()
    return m


# ---- plain forms ------------------------------------------------------------------------------------

TABLE = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)


def e4m3(v):
    """e4m3 codes of float64 v: the nearest of the 127 magnitudes, ties to the even code."""
    mags = TABLE[:127]
    a = np.minimum(np.abs(v), 448.0)
    hi = np.clip(np.searchsorted(mags, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up = (mags[hi] - a < a - mags[lo]) | ((mags[hi] - a == a - mags[lo]) & (hi % 2 == 0))
    code = np.where(up, hi, lo)
    return (code | (np.signbit(v) << 7)).astype(np.uint8)


def quant_reference(x):
    """Codes and scales of float32 x [T, K], each step of the definition one float32 rounding."""
    T, K = x.shape
    q, s = np.zeros((T, K), np.uint8), np.ones((T, -(-K // 128)), np.float32)
    for b in range(s.shape[1]):
        blk = x[:, b * 128 : (b + 1) * 128]
        a = np.abs(blk).max(1)
        sc = np.where(a == 0, np.float32(1), np.maximum(a * (np.float32(1) / np.float32(448)), np.float32(2.0 ** -126)))
        q[:, b * 128 : (b + 1) * 128] = e4m3((blk * (np.float32(1) / sc)[:, None]).astype(np.float64))
        s[:, b] = sc
    return q, s


def rows64(q, s):
    return q.float().double() * s.double().repeat_interleave(128, 1)[:, : q.shape[1]]


def weights64(q, s):
    N, K = q.shape
    return q.float().double() * s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def block_weights(N, K, gen):
    """Random e4m3 weights whose block scales differ by up to 16 times (a wrong block shows)."""
    q = (torch.randn(N, K, generator=gen) * 80).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = 2.0 ** (torch.rand(-(-N // 128), -(-K // 128), generator=gen) * 4 - 12)
    return q, s


# ---- quantisation -----------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K", [(1, 16), (1, 128), (3, 144), (7, 2000), (64, 4096), (333, 1040), (2, 20016)])
def test_quant_bit_exact(moe, T, K, dtype):
    gen = torch.Generator().manual_seed(T * K)
    x = torch.randn(T, K, generator=gen) * 2.0 ** (torch.rand(T, K // 16, generator=gen).repeat_interleave(16, 1) * 20 - 10)
    x = x.to(dtype)
    x[T // 2, : min(K, 128)] = 0  # a zero block
    q, s = moe.moe_quant_block(x.cuda())
    assert moe.moe_get_status() == 0
    rq, rs = quant_reference(x.float().numpy())
    assert np.array_equal(s.cpu().numpy().view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), rq)


def test_quant_extremes(moe):
    """Largest and smallest values, denormals, and blocks with an infinity or a NaN."""
    x = torch.zeros(6, 256)
    x[0, :128] = torch.finfo(torch.float32).max * torch.linspace(-1, 1, 128)
    x[1, :128] = 2.0 ** -140 * torch.arange(128)       # the scale is held at 2^-126
    x[2, 5] = 1e-45
    x[3, 7], x[3, 8] = float("inf"), 1.0
    x[4, 200] = float("nan")
    x[5, :] = torch.tensor([448.0, 1.0]).repeat(128)
    q, s = moe.moe_quant_block(x.cuda())
    q, s = q.float().cpu(), s.cpu()
    rq, rs = quant_reference(x[[0, 1, 2, 5]].numpy())
    assert np.array_equal(q[[0, 1, 2, 5]].numpy(), TABLE[rq].astype(np.float32))
    assert np.array_equal(s[[0, 1, 2, 5]].numpy(), rs)
    assert s[3, 0] == float("inf") and s[3, 1] == 1.0 and torch.isnan(q[3, 7])
    assert not torch.isfinite(q[3, :128] * s[3, 0]).any()
    assert torch.isnan(s[4, 1]) and torch.isnan(q[4, 128:]).all() and s[4, 0] == 1.0 and (q[4, :128] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,I", [(1, 16), (5, 128), (77, 768), (130, 1200)])
def test_silu_quant(moe, T, I, dtype):
    gen = torch.Generator().manual_seed(T + I)
    x = (torch.randn(T, 2 * I, generator=gen) * 3).to(dtype)
    q, s = moe.moe_silu_quant_block(x.cuda())
    g, u = x.double().split(I, 1)
    h = (g / (1 + torch.exp(-g)) * u).numpy()
    q, s = q.float().cpu().numpy().astype(np.float64), s.cpu().numpy().astype(np.float64)
    full = np.repeat(s, 128, 1)[:, :I]
    for b in range(s.shape[1]):
        a = np.abs(h[:, b * 128 : (b + 1) * 128]).max(1)
        assert np.allclose(s[:, b], a / 448, rtol=1e-6, atol=0)
    v = h / full
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    assert (np.abs(q - v) <= step / 2 + 2e-6 * np.abs(v)).all()


def test_silu_quant_of_large_values(moe):
    """The product is finite wherever its value is, gate and up of any size."""
    x = torch.zeros(4, 256)
    x[0, :128], x[0, 128:] = -20.0, 1e38  # g * u alone would overflow
    x[1, :128], x[1, 128:] = 1e30, 1e-30
    x[2, :128], x[2, 128:] = -200.0, 1e30  # SiLU is 0 in 32 bits
    x[3, :128], x[3, 128:] = 90.0, -3.0
    q, s = moe.moe_silu_quant_block(x.cuda())
    got = q.float().cpu().double() * s.cpu().double()
    g, u = x.double().split(128, 1)
    ref = g / (1 + torch.exp(-g)) * u
    ref[2] = 0
    assert torch.allclose(got, ref, rtol=2 ** -4, atol=0)


def test_quant_empty_and_far_offsets(moe):
    q, s = moe.moe_quant_block(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0, 2)
    # more than 2^31 elements: the last rows are right
    T, K = 70000, 32768
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, K, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    q, s = moe.moe_quant_block(x)
    rq, rs = quant_reference(x[-3:].float().cpu().numpy())
    assert np.array_equal(q[-3:].view(torch.uint8).cpu().numpy(), rq) and np.array_equal(s[-3:].cpu().numpy(), rs)
    assert (s[:-3] == 1).all() and (q[:4].float() == 0).all()


# ---- matrix product ---------------------------------------------------------------------------------

GEMMS = [
    # T, N, K
    (1, 1, 16), (1, 128, 128), (1, 4096, 2048), (2, 130, 144), (15, 257, 400), (16, 256, 1024), (17, 384, 128),
    (31, 100, 2064), (33, 640, 1152), (64, 512, 512), (65, 300, 272), (100, 2112, 2000), (127, 129, 640),
    (129, 513, 384), (200, 1000, 1168), (256, 512, 1024), (333, 777, 912), (511, 256, 4096), (700, 1537, 256),
    (1025, 2048, 768), (2049, 640, 528),
]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,K", GEMMS)
def test_gemm_against_64_bits(moe, T, N, K, out_dtype):
    gen = torch.Generator().manual_seed(T * 31 + N + K)
    a = (torch.randn(T, K, generator=gen) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    sa = 2.0 ** (torch.rand(T, -(-K // 128), generator=gen) * 4 - 8)
    w, sw = block_weights(N, K, gen)
    out = torch.full((T + 1, N), 7.0, dtype=out_dtype, device="cuda")  # a row behind the output stays as it is
    moe.moe_gemm_block(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), out=out[:T])
    assert moe.moe_get_status() == 0
    assert (out[T] == 7.0).all()
    A, W = rows64(a, sa), weights64(w, sw)
    ref, S = (A @ W.t()).numpy(), (A.abs() @ W.abs().t()).numpy()
    got = out[:T].double().cpu().numpy()
    tol = (2.0 ** -17 + (-(-K // 128) + 2) * 2.0 ** -24) * S
    if out_dtype == torch.bfloat16:
        tol = tol + bf16_half_ulp(np.maximum(np.abs(got), np.abs(ref)))
    assert (np.abs(got - ref) <= tol).all(), np.max((np.abs(got - ref)) / S)


@pytest.mark.parametrize("T", [40, 200])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_gemm_output_on_a_16_byte_boundary(moe, T, out_dtype):
    """An output that starts 16 bytes into a 256-byte boundary (the contract asks for no more)."""
    gen = torch.Generator().manual_seed(T)
    q, s = moe.moe_quant_block(torch.randn(T, 256, generator=gen).cuda())
    w, sw = (v.cuda() for v in block_weights(320, 256, gen))
    off = 16 // torch.empty(0, dtype=out_dtype).element_size()
    buf = torch.full((T * 320 + 2 * off,), 7.0, dtype=out_dtype, device="cuda")
    out = buf[off : off + T * 320].view(T, 320)
    moe.moe_gemm_block(q, s, w, sw, out=out)
    assert torch.equal(out, moe.moe_gemm_block(q, s, w, sw, out_dtype=out_dtype))
    assert (buf[:off] == 7.0).all() and (buf[-off:] == 7.0).all()


def test_gemm_sums_in_32_bits(moe):
    """A long sum with one large block: the small blocks' share survives (it would not in 16 bits)."""
    K = 8192
    a = torch.full((3, K), 1.0).to(torch.float8_e4m3fn)
    w = torch.full((5, K), 1.0).to(torch.float8_e4m3fn)
    sa, sw = torch.ones(3, K // 128), torch.ones(1, K // 128)
    sa[:, 0] = 2.0 ** 12
    out = moe.moe_gemm_block(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), out_dtype=torch.float32)
    assert (out.cpu() == 128 * 2.0 ** 12 + (K - 128)).all()


def test_gemm_nan_stays_in_its_row(moe):
    gen = torch.Generator().manual_seed(5)
    a = torch.randn(70, 256, generator=gen)
    a[9, 3] = float("nan")
    a[40, 200] = float("inf")
    q, s = moe.moe_quant_block(a.cuda())
    w, sw = block_weights(300, 256, gen)
    out = moe.moe_gemm_block(q, s, w.cuda(), sw.cuda(), out_dtype=torch.float32).cpu()
    bad = torch.isnan(out).all(1)
    assert bad[9] and bad[40] and torch.isfinite(out[~bad]).all() and int(bad.sum()) == 2


def test_gemm_repeats_bit_for_bit_and_on_another_stream(moe):
    gen = torch.Generator().manual_seed(6)
    for T, N, K in ((5, 1024, 2048), (300, 700, 1536)):
        a = torch.randn(T, K, generator=gen).cuda()
        q, s = moe.moe_quant_block(a)
        w, sw = (v.cuda() for v in block_weights(N, K, gen))
        ref = moe.moe_gemm_block(q, s, w, sw, out_dtype=torch.float32)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            got = moe.moe_gemm_block(q, s, w, sw, out_dtype=torch.float32, stream=side)
            side.synchronize()
            assert torch.equal(ref, got)


def test_dense_mlp_chain(moe):
    """quantise -> product -> SiLU quantise -> product, as a shared expert runs, against 64 bits."""
    gen = torch.Generator().manual_seed(8)
    T, H, I = 45, 640, 400
    x = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    w13, s13 = block_weights(2 * I, H, gen)
    w2, s2 = block_weights(H, I, gen)
    q, s = moe.moe_quant_block(x.cuda())
    gu = moe.moe_gemm_block(q, s, w13.cuda(), s13.cuda(), out_dtype=torch.float32)
    hq, hs = moe.moe_silu_quant_block(gu)
    out = moe.moe_gemm_block(hq, hs, w2.cuda(), s2.cuda())
    rq, rs = quant_reference(x.float().numpy())
    v = torch.from_numpy(TABLE[rq] * np.repeat(rs.astype(np.float64), 128, 1)[:, :H]) @ weights64(w13, s13).t()
    h = v[:, :I] / (1 + torch.exp(-v[:, :I])) * v[:, I:]
    hq, hs = quant_reference(h.float().numpy())
    ref = torch.from_numpy(TABLE[hq] * np.repeat(hs.astype(np.float64), 128, 1)[:, :I]) @ weights64(w2, s2).t()
    assert_parity(out.float().cpu().numpy(), ref.numpy(), "e4m3", "dense mlp")


# ---- expert layer -----------------------------------------------------------------------------------


def make_experts(T, H, I, E, k, gen, hot=False):
    x = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    score = torch.randn(T, E, generator=gen)
    if hot:
        score[:, E // 2] += 100
    v, ids = score.topk(k, 1)
    w13, s13 = zip(*(block_weights(2 * I, H, gen) for _ in range(E)))
    w2, s2 = zip(*(block_weights(H, I, gen) for _ in range(E)))
    return dict(x=x, ids=ids.to(torch.int32), tw=torch.softmax(v, 1), w13=torch.stack(w13), s13=torch.stack(s13),
                w2=torch.stack(w2), s2=torch.stack(s2))


def experts_reference(d):
    T, H = d["x"].shape
    k, I = d["ids"].shape[1], d["w2"].shape[2]
    q, s = quant_reference(d["x"].float().numpy())
    x = torch.from_numpy(TABLE[q] * np.repeat(s.astype(np.float64), 128, 1))
    out = torch.zeros(T, H, dtype=torch.float64)
    for e in range(d["w13"].shape[0]):
        t, j = (d["ids"] == e).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        gu = x[t] @ weights64(d["w13"][e], d["s13"][e]).t()
        g, u = gu.split(I, 1)
        q, s = quant_reference((g / (1 + torch.exp(-g)) * u).float().numpy())
        h = torch.from_numpy(TABLE[q] * np.repeat(s.astype(np.float64), 128, 1))
        y = h @ weights64(d["w2"][e], d["s2"][e]).t()
        out.index_add_(0, t, y * d["tw"][t, j].double()[:, None])
    return out.numpy()


def check(got, ref, label):
    got = got.float().cpu().numpy()
    assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref), label
    assert_parity(got, ref, "e4m3", label)


LAYERS = [
    # T, H, I, E, k, hot
    (1, 256, 128, 4, 2, False), (1, 2048, 768, 16, 8, False), (3, 384, 256, 8, 1, False), (16, 512, 384, 5, 3, False),
    (17, 640, 256, 8, 2, True), (33, 256, 512, 6, 6, False), (64, 1024, 256, 16, 4, True), (65, 256, 256, 8, 2, False),
    (130, 384, 384, 3, 2, False), (300, 512, 256, 40, 4, False), (700, 256, 640, 7, 2, True), (1500, 384, 128, 4, 4, False),
]


@pytest.mark.parametrize("T,H,I,E,k,hot", LAYERS)
def test_experts_against_64_bits(moe, T, H, I, E, k, hot):
    d = make_experts(T, H, I, E, k, torch.Generator().manual_seed(T + H), hot)
    c = {n: v.cuda() for n, v in d.items()}
    out = moe.moe_forward_routed(c["x"], c["tw"], c["ids"], c["w13"], c["w2"], c["s13"], c["s2"], w_format="e4m3_block")
    assert moe.moe_get_status() == 0
    check(out, experts_reference(d), f"experts {T}x{H}x{I} E{E} k{k}")
    again = moe.moe_forward_routed(c["x"], c["tw"], c["ids"], c["w13"], c["w2"], c["s13"], c["s2"], w_format="e4m3_block")
    assert torch.equal(out, again)


@pytest.mark.parametrize("T,hot", [(48, False), (90, True), (300, False), (400, True)])
def test_both_orientations_agree(moe, T, hot):
    d = make_experts(T, 512, 256, 8, 3, torch.Generator().manual_seed(2), hot)
    ref = experts_reference(d)
    c = {n: v.cuda() for n, v in d.items()}
    for o in (moe.ORIENT_SWAP_AB, moe.ORIENT_TOKEN_MAJOR):
        out = moe.moe_forward_routed(c["x"], c["tw"], c["ids"], c["w13"], c["w2"], c["s13"], c["s2"],
                                     options={"orientation": o}, w_format="e4m3_block")
        assert moe.moe_get_status() == 0
        check(out, ref, f"orientation {o}")


def test_forward_and_noalloc_route_themselves(moe):
    d = make_experts(20, 256, 256, 8, 2, torch.Generator().manual_seed(4))
    c = {n: v.cuda() for n, v in d.items()}
    wr = (torch.randn(8, 256, generator=torch.Generator().manual_seed(5)) / 16).to(torch.bfloat16).cuda()
    _, tw, ids = moe.moe_route(c["x"], wr, 2, True)
    ref = moe.moe_forward_routed(c["x"], tw, ids, c["w13"], c["w2"], c["s13"], c["s2"], w_format="e4m3_block")
    out = moe.moe_forward(c["x"], wr, c["w13"], c["w2"], 2, True, c["s13"], c["s2"], w_format="e4m3_block")
    assert torch.equal(out, ref)
    out = moe.moe_forward_noalloc(c["x"], wr, c["w13"], c["w2"], 2, True, c["s13"], c["s2"], w_format="e4m3_block")
    assert torch.equal(out, ref)
    out = moe.moe_forward_host(d["x"].pin_memory(), wr, c["w13"], c["w2"], 2, True, c["s13"], c["s2"],
                               w_format="e4m3_block")
    torch.cuda.synchronize()
    assert torch.equal(out, ref.cpu())


def test_short_batch_routes_itself(moe):
    d = make_experts(3, 512, 256, 8, 2, torch.Generator().manual_seed(6))
    c = {n: v.cuda() for n, v in d.items()}
    wr = (torch.randn(8, 512, generator=torch.Generator().manual_seed(7)) / 16).to(torch.bfloat16).cuda()
    _, tw, ids = moe.moe_route(c["x"], wr, 2, True)
    ref = moe.moe_forward_routed(c["x"], tw, ids, c["w13"], c["w2"], c["s13"], c["s2"], w_format="e4m3_block")
    for _ in range(5):
        out = moe.moe_forward(c["x"], wr, c["w13"], c["w2"], 2, True, c["s13"], c["s2"], w_format="e4m3_block")
        assert torch.equal(out, ref)


def test_expert_id_out_of_range_is_dropped_and_flagged(moe):
    for T in (9, 90):
        d = make_experts(T, 256, 128, 4, 2, torch.Generator().manual_seed(T))
        c = {n: v.cuda() for n, v in d.items()}
        c["ids"][3, 1] = 4
        c["ids"][5, 0] = -2
        d["ids"][3, 1], d["ids"][5, 0] = 4, -2
        moe.moe_forward_routed(c["x"], c["tw"], c["ids"], c["w13"], c["w2"], c["s13"], c["s2"], w_format="e4m3_block")
        assert moe.moe_get_status() == moe.MOE_ERR_DEVICE_INDEX
        assert moe.moe_get_status() == 0


@pytest.mark.parametrize("T", [1, 16, 20, 60, 100])
def test_an_expert_named_twice_for_a_token(moe, T):
    """A caller's routing may repeat an expert: its list is then longer than the batch."""
    d = make_experts(T, 256, 128, 4, 3, torch.Generator().manual_seed(T))
    d["ids"][:, 1] = d["ids"][:, 0]
    d["ids"][: T // 2 + 1] = 2
    c = {n: v.cuda() for n, v in d.items()}
    out = moe.moe_forward_routed(c["x"], c["tw"], c["ids"], c["w13"], c["w2"], c["s13"], c["s2"], w_format="e4m3_block")
    assert moe.moe_get_status() == 0
    check(out, experts_reference(d), f"repeated experts T={T}")


@pytest.mark.parametrize("T,k", [(32, 1), (16, 2), (17, 2), (10, 3), (11, 3), (4, 8), (5, 8), (1, 16)])
@pytest.mark.parametrize("one", [False, True])
def test_short_batches_around_32_pairs(moe, T, k, one):
    """Up to 32 pairs are sorted by the launch that quantises them; one: all pairs at a single expert."""
    d = make_experts(T, 384, 256, 19, k, torch.Generator().manual_seed(T * k))
    if one:
        d["ids"][:] = 7
    c = {n: v.cuda() for n, v in d.items()}
    out = moe.moe_forward_routed(c["x"], c["tw"], c["ids"], c["w13"], c["w2"], c["s13"], c["s2"], w_format="e4m3_block")
    assert moe.moe_get_status() == 0
    check(out, experts_reference(d), f"{T} x {k}")


def test_a_short_batch_depends_on_no_other_call(moe):
    """Calls of different batches back to back in one workspace: each reads its own routing."""
    ds = [make_experts(T, 256, 128, 12, 4, torch.Generator().manual_seed(T)) for T in (2, 8, 1, 5)]
    n = moe.moe_workspace_size(8, 256, 128, 12, 4, moe.MOE_BF16, moe.MOE_E4M3_B128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    cs = [{n: v.cuda() for n, v in d.items()} for d in ds]
    outs = [[moe.moe_forward_routed(c["x"], c["tw"], c["ids"], c["w13"], c["w2"], c["s13"], c["s2"], workspace=ws,
                                    w_format="e4m3_block") for c in cs] for _ in range(20)]
    assert moe.moe_get_status() == 0
    for i, d in enumerate(ds):
        check(outs[0][i], experts_reference(d), f"batch {i}")
        assert all(torch.equal(o[i], outs[0][i]) for o in outs)


def test_empty_batch(moe):
    d = make_experts(1, 256, 128, 4, 2, torch.Generator().manual_seed(1))
    c = {n: v.cuda() for n, v in d.items()}
    out = moe.moe_forward_routed(c["x"][:0], c["tw"][:0], c["ids"][:0], c["w13"], c["w2"], c["s13"], c["s2"],
                                 w_format="e4m3_block")
    assert out.shape == (0, 256)
