"""Cases for the operators of a block-scaled FP8 expert layer: routing by groups, quantisation by
blocks of 128, the FP8 matrix product with a scale per block, and the expert products built on them.

`run` computes each operator in plain form (elementary torch operations in 32 bits), or, where `own`
is true, through the package's entry points.
"""
import math

import torch

own = False

BLK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


def _route(name, T, E, k, groups, kept, group_sum, score, bias, renorm=True, scale=1.0):
    return dict(name=name, op="route", T=T, E=E, k=k, groups=groups, kept=kept, group_sum=group_sum, score=score,
                bias=bias, renorm=renorm, scale=scale)


def listed():
    return [
        # one token of a decode step: the call's latency
        _route("route decode 1", 1, 256, 8, 8, 4, 2, "sigmoid", True, True, 2.5),
        # a decode batch on the 160-expert form with softmax scores, the best expert standing for a group of 20
        _route("route batch softmax 160", 777, 160, 6, 8, 3, 1, "softmax", False, False, 16.0),
        # a long prefill chunk
        _route("route prefill 16384", 16384, 256, 8, 8, 4, 2, "sigmoid", True, True, 2.5),
        # the layer input of a decode batch
        dict(name="quant decode 64", op="quant", T=64, K=4096, dtype="bf16"),
        # the layer input of a prefill chunk
        dict(name="quant prefill 8192", op="quant", T=8192, K=4096, dtype="bf16"),
        # gate and up of a shared expert, an odd number of tokens
        dict(name="silu quant 4099", op="silu_quant", T=4099, K=2048, dtype="bf16"),
        # a projection at a small decode batch: streaming the weights
        dict(name="gemm decode 16", op="gemm", T=16, N=8192, K=4096, out="bf16"),
        # ragged in every direction: tokens, half a block of outputs, a last block of 80 inputs, fp32 out
        dict(name="gemm ragged 333", op="gemm", T=333, N=2112, K=2000, out="f32"),
        # a square projection of a prefill chunk
        dict(name="gemm prefill 8192", op="gemm", T=8192, N=4096, K=4096, out="bf16"),
        # one token through many small experts
        dict(name="experts decode fine 1", op="experts", T=1, H=2048, I=768, E=128, k=8, skew=1.1),
        # a decode batch over large experts: streaming the weights
        dict(name="experts decode 16", op="experts", T=16, H=4096, I=8192, E=64, k=8, skew=0.0),
        # a prefill chunk
        dict(name="experts prefill 8192", op="experts", T=8192, H=4096, I=2048, E=64, k=8, skew=0.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "quant", "silu_quant", "gemm", "gemm", "experts", "experts"])
    if op == "route":
        groups = rng.choice([1, 2, 4, 6, 8, 12, 16])
        per = rng.choice([g for g in (4, 8, 12, 16, 20, 32, 48, 64) if 8 <= g * groups <= 512])
        kept = rng.randint(max(1, groups // 4), groups)
        k = rng.randint(1, min(10, kept * per))
        score = rng.choice(["sigmoid", "softmax"])
        c = _route("", _log_int(rng, 1, 16384), groups * per, k, groups, kept, rng.choice([1, 2]), score,
                   rng.random() < 0.6, rng.random() < 0.7, rng.choice([1.0, 2.5, 16.0]))
        del c["name"]
        return c
    if op in ("quant", "silu_quant"):
        return dict(op=op, T=_log_int(rng, 1, 8192), K=16 * _log_int(rng, 8, 512), dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "gemm":
        return dict(op=op, T=_log_int(rng, 1, 8192), N=_log_int(rng, 64, 8192), K=16 * _log_int(rng, 8, 512),
                    out=rng.choice(["bf16", "bf16", "f32"]))
    E = rng.choice([8, 16, 40, 64, 128])
    return dict(op=op, T=_log_int(rng, 1, 4096), H=128 * rng.randint(4, 32), I=128 * _log_int(rng, 2, 16), E=E,
                k=rng.choice([1, 2, 4, 6, 8]), skew=rng.choice([0.0, 0.0, 1.1]))


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, T, K, dtype):
    """Hidden states: unit normal with a few outlier columns, as trained layers have them."""
    x = _randn(g, T, K)
    x *= torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    return x.to(dtype)


def _quant_rows(x):
    """Codes and scales of x [T, K] by rows and blocks of 128 columns."""
    T, K = x.shape
    nb = -(-K // BLK)
    xp = torch.nn.functional.pad(x.float(), (0, nb * BLK - K)).view(T, nb, BLK)
    amax = xp.abs().amax(2)
    s = torch.where(amax == 0, torch.ones_like(amax), (amax / E4M3_MAX).clamp(min=SCALE_MIN))
    q = (xp * (1.0 / s)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(T, nb * BLK)[:, :K].contiguous(), s


def _ranks64(c, logits, bias):
    """Scores, biased scores and group scores in 64 bits."""
    l64 = logits.double()
    s = torch.sigmoid(l64) if c["score"] == "sigmoid" else torch.softmax(l64, 1)
    r = s if bias is None else s + bias.double()
    top = r.view(len(r), c["groups"], -1).sort(2, descending=True)[0]
    return s, r, top[:, :, : c["group_sum"]].sum(2)


def _clear(c, logits, bias):
    """Rows whose ranking does not hang on the last bits of a 32-bit score."""
    s, r, gs = _ranks64(c, logits, bias)
    far = 1e-5 * r.abs().amax(1)
    ok = torch.ones(len(r), dtype=torch.bool, device=r.device)
    if c["kept"] < c["groups"]:
        g = gs.sort(1, descending=True)[0]
        ok &= g[:, c["kept"] - 1] - g[:, c["kept"]] > far
        keep = gs >= g[:, c["kept"] - 1 : c["kept"]]
        r = r.masked_fill(~keep.repeat_interleave(c["E"] // c["groups"], 1), -math.inf)
    t = r.sort(1, descending=True)[0][:, : c["k"] + 1]
    return ok & (t[:, :-1] - t[:, 1:] > far[:, None]).all(1)


def prepare(case, seed):
    c, g = case, _gen(seed)
    op, T = c["op"], c["T"]
    st = dict(case=c)

    def weights(lead, N, K):
        """Weights N(0, 0.02) as e4m3 codes [lead, N, K] with one scale per 128 x 128 block."""
        n, k = -(-N // BLK), -(-K // BLK)
        q = torch.empty(lead, N, K, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty(lead, n, k, dtype=torch.float32, device="cuda")
        for e in range(lead):
            w = torch.nn.functional.pad(_randn(g, N, K) * 0.02, (0, k * BLK - K, 0, n * BLK - N)).view(n, BLK, k, BLK)
            s[e] = w.abs().amax((1, 3)) / E4M3_MAX
            w = (w / s[e][:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            q[e] = w.view(n * BLK, k * BLK)[:N, :K]
        return q, s

    if op == "route":
        E = c["E"]
        st["bias"] = _randn(g, E) * 0.05 if c["bias"] else None
        if c["score"] == "softmax" and c["bias"]:
            st["bias"] = st["bias"] / E
        got = torch.empty(0, E, device="cuda")
        while len(got) < T:  # logits of a trained router: a common preference for some experts, and the token's own
            l = _randn(g, T + T // 4 + 64, E) * 1.2 + _randn(g, 1, E) * 0.5
            got = torch.cat([got, l[_clear(c, l, st["bias"])]])
        st["logits"] = got[:T].contiguous()
    elif op == "quant":
        st["x"] = _activations(g, T, c["K"], _DT[c["dtype"]])
    elif op == "silu_quant":
        st["x"] = (_activations(g, T, 2 * c["K"], torch.float32) * 1.5).to(_DT[c["dtype"]])
    elif op == "gemm":
        st["a"], st["sa"] = _quant_rows(_activations(g, T, c["K"], torch.bfloat16))
        w, s = weights(1, c["N"], c["K"])
        st["w"], st["sw"] = w[0], s[0]
    else:
        H, I, E, k = c["H"], c["I"], c["E"], c["k"]
        st["x"] = _activations(g, T, H, torch.bfloat16)
        like = _randn(g, T, E) - c["skew"] * torch.log(1.0 + torch.randperm(E, generator=g, device="cuda"))
        v, ids = like.topk(k, 1)
        st["ids"], st["tw"] = ids.to(torch.int32), torch.softmax(v, 1)
        st["w13"], st["s13"] = weights(E, 2 * I, H)
        st["w2"], st["s2"] = weights(E, H, I)
    return st


# ---- plain forms --------------------------------------------------------------------------------------


def _plain_route(c, logits, bias):
    e = torch.exp(-logits) if c["score"] == "sigmoid" else torch.exp(logits - logits.amax(1, keepdim=True))
    s = 1.0 / (1.0 + e) if c["score"] == "sigmoid" else e / e.sum(1, keepdim=True)
    r = s if bias is None else s + bias
    if c["kept"] < c["groups"]:
        grouped = r.view(len(r), c["groups"], -1)
        gs = grouped.sort(2, descending=True)[0][:, :, : c["group_sum"]].sum(2)
        best = gs.sort(dim=1, descending=True, stable=True)[1][:, : c["kept"]]
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, best, True)
        r = grouped.masked_fill(~keep[:, :, None], -math.inf).view_as(r)
    ids = r.sort(dim=1, descending=True, stable=True)[1][:, : c["k"]]
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return w * c["scale"], ids.to(torch.int32)


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _rows32(q, s, dtype=torch.float32):
    return q.to(dtype) * s.to(dtype).repeat_interleave(BLK, 1)[:, : q.shape[1]]


def _weights32(q, s, dtype=torch.float32):
    N, K = q.shape[-2:]
    return q.to(dtype) * s.to(dtype).repeat_interleave(BLK, -2)[..., :N, :].repeat_interleave(BLK, -1)[..., :K]


def _plain_experts(c, x, ids, tw, w13, s13, w2, s2):
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    xq = _rows32(*_quant_rows(x))
    flat = ids.reshape(-1).long()
    if T * k <= E:  # few pairs: each with its own expert's weights
        rows, pick = xq.repeat_interleave(k, 0)[:, None, :], flat
        place = None
    else:  # every expert's tokens side by side, padded to the longest list
        order = flat.sort(stable=True)[1]
        count = torch.bincount(flat, minlength=E)
        start = count.cumsum(0) - count
        e = flat[order]
        place = (e, torch.arange(T * k, device=x.device) - start[e])
        rows = torch.zeros(E, int(count.max()), H, device=x.device)
        rows[place] = xq[order // k]
        pick = slice(None)
    gu = rows @ _weights32(w13[pick], s13[pick]).transpose(1, 2)
    h = _silu(gu[..., :I]) * gu[..., I:]
    hq = _rows32(*_quant_rows(h.reshape(-1, I))).view(*h.shape)
    y = hq @ _weights32(w2[pick], s2[pick]).transpose(1, 2)
    if place is None:
        y = y[:, 0]
    else:
        y = torch.empty(T * k, H, device=x.device).index_copy_(0, order, y[place])
    return (y.view(T, k, H) * tw[:, :, None]).sum(1).to(torch.bfloat16)


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import mixture_experts_layer_scan_gb300 as moe

        if op == "route":
            return moe.moe_topk_grouped(state["logits"], c["k"], bias=state["bias"], score=c["score"], n_group=c["groups"],
                                        topk_group=c["kept"], group_sum=c["group_sum"], renorm=c["renorm"], scale=c["scale"])
        if op == "quant":
            return moe.moe_quant_block(state["x"])
        if op == "silu_quant":
            return moe.moe_silu_quant_block(state["x"])
        if op == "gemm":
            return moe.moe_gemm_block(state["a"], state["sa"], state["w"], state["sw"], out_dtype=_DT[c["out"]])
        if "ws" not in state:  # a program keeps the workspace of its layer
            n = moe.moe_workspace_size(c["T"], c["H"], c["I"], c["E"], c["k"], moe.MOE_BF16, moe.MOE_E4M3_B128)
            state["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return moe.moe_forward_routed(state["x"], state["tw"], state["ids"], state["w13"], state["w2"], state["s13"],
                                      state["s2"], workspace=state["ws"], w_format="e4m3_block")
    if op == "route":
        return _plain_route(c, state["logits"], state["bias"])
    if op == "quant":
        return _quant_rows(state["x"])
    if op == "silu_quant":
        x = state["x"].float()
        return _quant_rows(_silu(x[:, : c["K"]]) * x[:, c["K"] :])
    if op == "gemm":
        return (_rows32(state["a"], state["sa"]) @ _weights32(state["w"], state["sw"]).t()).to(_DT[c["out"]])
    return _plain_experts(c, *(state[n] for n in ("x", "ids", "tw", "w13", "s13", "w2", "s2")))


def work(case):
    c = case
    op, T = c["op"], c["T"]
    if op == "route":
        return {"bytes": 4 * T * c["E"] + 8 * T * c["k"] + (4 * c["E"] if c["bias"] else 0), "flops": 8 * T * c["E"]}
    if op in ("quant", "silu_quant"):
        K, two = c["K"], 2 if op == "silu_quant" else 1
        xb = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": T * (two * K * xb + K + 4 * -(-K // BLK)), "flops": 4 * two * T * K}
    if op == "gemm":
        N, K = c["N"], c["K"]
        nb, kb = -(-N // BLK), -(-K // BLK)
        ob = 2 if c["out"] == "bf16" else 4
        return {"bytes": T * K + N * K + 4 * T * kb + 4 * nb * kb + ob * T * N, "flops": 2 * T * N * K}
    H, I, E, k = c["H"], c["I"], c["E"], c["k"]
    active = E * (1.0 - (1.0 - k / E) ** T)  # experts that a batch reaches, on average
    return {"bytes": active * 3 * H * I * (1 + 4 / BLK ** 2) + 4 * T * H + 8 * T * k, "flops": 6 * T * k * H * I}


# ---- 64 bits ---------------------------------------------------------------------------------------------


def _codes64(v):
    """e4m3 values nearest to v (64 bits), ties to the even code, saturating at 448."""
    a = v.abs().clamp(max=E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _quant64(x):
    """Code values and scales by rows and blocks of 128, from 64-bit x.  The definition takes the scale, its
    reciprocal and the product as 32-bit numbers (16-bit inputs often lie on the border of two codes, which the
    last bit of these decides), so they are rounded here too."""
    T, K = x.shape
    s = torch.stack([b.abs().amax(1) for b in x.split(BLK, 1)], 1).float()
    s = torch.where(s == 0, 1.0, (s / E4M3_MAX).clamp(min=SCALE_MIN))
    r = (1.0 / s.double()).float().double()
    return _codes64((x.float().double() * r.repeat_interleave(BLK, 1)[:, :K]).float().double()), s.double()


def exact(case, seed):
    c, st = case, prepare(case, seed)
    op = c["op"]
    if op == "route":
        s, r, gs = _ranks64(c, st["logits"], st["bias"])
        best = gs.sort(1, descending=True)[1][:, : c["kept"]]
        member = torch.arange(c["E"], device=r.device) // (c["E"] // c["groups"])
        r = r.masked_fill(~(member[None, :, None] == best[:, None, :]).any(2), -math.inf)
        ids = r.topk(c["k"], 1)[1]
        w = s.gather(1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return w * c["scale"], ids.to(torch.int32)
    if op == "quant":
        return _quant64(st["x"].double())
    if op == "silu_quant":
        g, u = st["x"].double().split(c["K"], 1)
        return _quant64(g * torch.sigmoid(g) * u)
    if op == "gemm":
        a, sa, w, sw = (st[n].double() for n in ("a", "sa", "w", "sw"))
        out = torch.zeros(c["T"], c["N"], dtype=torch.float64, device=a.device)
        rows = torch.arange(c["N"], device=a.device) // BLK
        for b, (ab, wb) in enumerate(zip(a.split(BLK, 1), w.split(BLK, 1))):
            out += (ab @ wb.t()) * sa[:, b, None] * sw[rows, b]
        return out
    x, s = _quant64(st["x"].double())
    x = x * s.repeat_interleave(BLK, 1)
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=x.device)
    for e in range(c["E"]):
        t, j = (st["ids"] == e).nonzero(as_tuple=True)
        if len(t):
            gu = x[t] @ _weights32(st["w13"][e], st["s13"][e], torch.float64).t()
            g, u = gu.split(c["I"], 1)
            q, s = _quant64(g * torch.sigmoid(g) * u)
            y = (q * s.repeat_interleave(BLK, 1)) @ _weights32(st["w2"][e], st["s2"][e], torch.float64).t()
            out.index_add_(0, t, y * st["tw"][t, j].double()[:, None])
    return out
