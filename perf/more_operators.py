"""Cases for the operators around an expert layer: tokens sorted by expert and back with their
gradients, the norms before and after a block with its gate and residual scale, and low-rank adapters
of many requests beside a shared projection.

`run` computes each operator in plain form (elementary torch operations in 32 bits), or, where `own`
is true, through the package's entry points.
"""
import math

import torch

own = False

EPS = 1e-6


def _rows(name, op, T, H, E, k, dtype, block=1, weighted=True, skew=0.0):
    return dict(name=name, op=op, T=T, H=H, E=E, k=k, dtype=dtype, block=block, weighted=weighted, skew=skew)


def _norm(name, op, T, H, dtype, post=True, gate="none", sigmoid=False, nxt=True, scale=1.0, res_scale=1.0, wide=False):
    return dict(name=name, op=op, T=T, H=H, dtype=dtype, post=post, gate=gate, sigmoid=sigmoid, next=nxt, scale=scale,
                res_scale=res_scale, wide=wide)


def _lora(name, T, K, N, r, L, out, packed):
    return dict(name=name, op="lora", T=T, K=K, N=N, r=r, L=L, out=out, packed=packed)


def listed():
    return [
        # a decode batch over many small experts, blocks of 16 rows for a thin product
        _rows("permute decode 64", "permute", 64, 2048, 128, 8, "bf16", block=16, skew=1.1),
        # a prefill chunk or a training batch, padded to the tiles of a large product
        _rows("permute prefill 8192", "permute", 8192, 4096, 64, 8, "bf16", block=128),
        # the expert outputs of an odd batch back to token order, in 32 bits
        _rows("unpermute 4099 f32", "unpermute", 4099, 2048, 64, 6, "f32"),
        # the gradient of that step in training: rows and routing weights
        _rows("unpermute grad 8192", "unpermute_grad", 8192, 4096, 64, 8, "bf16", block=128),
        # one token of a decode step: the call's latency
        _norm("prenorm decode 1", "prenorm", 1, 4096, "bf16"),
        # gradient of the norm before a block, a row that is no multiple of a vector, 32-bit weights
        _norm("prenorm grad 4096 x 2047", "prenorm_grad", 4096, 2047, "bf16", wide=True),
        # a decode batch: norm after the block, channel gate, residual and the next block's norm at once
        _norm("postnorm decode 32", "postnorm", 32, 4096, "bf16", gate="channel", scale=0.22),
        # a long prefill chunk, the block's output gated per token
        _norm("postnorm prefill 16384", "postnorm", 16384, 4096, "bf16", gate="token", sigmoid=True, res_scale=1.5),
        # its gradient in a training step: both inputs, both weights, the gate's channels
        _norm("postnorm grad 8192", "postnorm_grad", 8192, 4096, "bf16", gate="channel", scale=0.22),
        # a decode batch of requests with adapters of their own
        _lora("lora decode 48", 48, 4096, 4096, 16, 64, "bf16", False),
        # a mixed batch, a few tokens for each adapter, odd sizes, 32-bit output
        _lora("lora mixed 777", 777, 2040, 5000, 32, 24, "f32", True),
        # a prefill chunk of several requests
        _lora("lora prefill 8192", 8192, 4096, 8192, 64, 16, "bf16", True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, most):
    """Row lengths: mostly whole vectors, some odd."""
    return _log_int(rng, 64, most) if rng.random() < 0.2 else 8 * _log_int(rng, 16, most // 8)


def draw(rng):
    op = rng.choice(["permute", "unpermute", "unpermute", "unpermute_grad", "prenorm", "prenorm_grad", "postnorm", "postnorm",
                     "postnorm_grad", "lora", "lora", "lora"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("permute", "unpermute", "unpermute_grad"):
        H, E = _width(rng, 8192), rng.choice([4, 8, 40, 64, 128, 256])
        k = rng.randint(1, min(8, E))
        T = _log_int(rng, 1, max(1, min(16384, 8192 * 8 * 4096 // (k * H * (2 if dtype == "f32" else 1)))))
        c = _rows("", op, T, H, E, k, dtype, rng.choice([1, 16, 64, 128]), op != "unpermute" or rng.random() < 0.6,
                  rng.choice([0.0, 0.0, 1.1]))
    elif op != "lora":
        H = _width(rng, 8192)
        T = _log_int(rng, 1, max(1, min(16384, 8192 * 4096 // (H * (2 if dtype == "f32" else 1)))))
        post = rng.random() < 0.7
        gate = rng.choice(["none", "channel", "token", "full"])
        c = _norm("", op, T, H, dtype, post, gate, gate != "none" and rng.random() < 0.5, rng.random() < 0.7,
                  rng.choice([1.0, 0.22]), rng.choice([1.0, 1.5]), rng.random() < 0.3)
    else:
        r, K, N = rng.choice([8, 16, 16, 24, 32, 64, 64, 128]), 8 * _log_int(rng, 16, 1024), 8 * _log_int(rng, 16, 1024)
        T = _log_int(rng, 1, max(1, min(8192, 8192 * 64 * 4096 * 3 // (r * (K + N)))))
        L = rng.randint(1, max(1, min(64, 8192 * 64 * 16 * 4096 * 3 // (T * r * (K + N)))))
        c = _lora("", T, K, N, r, L, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.6)
    del c["name"]
    return c


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


def _capacity(c):
    """Rows of a permutation: every pair, and up to block - 1 more for each expert that a batch can reach."""
    n = c["T"] * c["k"]
    return n + min(c["E"], n) * (c["block"] - 1)


def _places(ids, E, block):
    """Row of every pair in expert order, each expert's run padded to a multiple of block; pairs per expert."""
    flat = ids.reshape(-1).long()
    order = flat.sort(stable=True)[1]
    count = torch.bincount(flat, minlength=E)
    padded = (count + block - 1) // block * block
    start, first = count.cumsum(0) - count, padded.cumsum(0) - padded
    e = flat[order]
    row = torch.empty_like(flat).index_copy_(0, order, first[e] + torch.arange(len(flat), device=flat.device) - start[e])
    return row, count


def prepare(case, seed):
    c, g = case, _gen(seed)
    op, T = c["op"], c["T"]
    st = dict(case=c)
    if op in ("permute", "unpermute", "unpermute_grad"):
        H, E, k, dt = c["H"], c["E"], c["k"], _DT[c["dtype"]]
        like = _randn(g, T, E) - c["skew"] * torch.log(1.0 + torch.randperm(E, generator=g, device="cuda"))
        v, ids = like.topk(k, 1)
        ids = ids.to(torch.int32)
        if op == "permute":
            # (the buffer that a program keeps for its experts' rows: what lies behind the last row stays zero)
            st["x"], st["ids"] = _activations(g, T, H, dt), ids
            st["rows"] = torch.zeros(_capacity(c), H, dtype=dt, device="cuda")
            return st
        row, count = _places(ids, E, c["block"])
        # pair of every row, T * k for padding
        st["sorted_ids"] = torch.full((_capacity(c),), T * k, dtype=torch.int32, device="cuda")
        st["sorted_ids"][row] = torch.arange(T * k, dtype=torch.int32, device="cuda")
        st["num_post_pad"] = ((count + c["block"] - 1) // c["block"] * c["block"]).sum().to(torch.int32).view(1)
        st["rows"] = _activations(g, _capacity(c), H, dt) * (st["sorted_ids"] < T * k)[:, None]
        st["row_of"] = row.view(T, k).to(torch.int32)
        st["w"] = torch.softmax(v, 1) if c["weighted"] else None
        if op == "unpermute_grad":
            st["d_out"] = (_randn(g, T, H) * 0.1).to(dt)
            st["d_rows"] = torch.zeros(_capacity(c), H, dtype=dt, device="cuda")
    elif op == "lora":
        K, N, r, L = c["K"], c["N"], c["r"], c["L"]
        st["x"] = _activations(g, T, K, torch.bfloat16)
        st["a"] = (_randn(g, L, r, K) * K ** -0.5).to(torch.bfloat16)
        st["b"] = (_randn(g, L, N, r) * r ** -0.5).to(torch.bfloat16)
        st["scale"] = torch.rand(L, generator=g, device="cuda") * 1.5 + 0.5
        st["base"] = _randn(g, T, N).to(_DT[c["out"]])
        # popular adapters more often; one request in eight has none
        like = torch.rand(T, generator=g, device="cuda") ** 2 * L
        ids = torch.where(torch.rand(T, generator=g, device="cuda") < 0.125, -1, like.long().clamp(max=L - 1))
        if c["packed"]:  # prompts of several requests, one after another
            cut = torch.rand(T, generator=g, device="cuda") < min(1.0, 24.0 / T)
            at = torch.where(cut, torch.arange(T, device="cuda"), 0).cummax(0)[0]
            ids = ids[at]
        st["ids"] = ids.to(torch.int32)
    else:
        H, dt = c["H"], _DT[c["dtype"]]
        wd = torch.float32 if c["wide"] else dt
        weight = lambda: (1.0 + 0.2 * _randn(g, H)).to(wd)  # noqa: E731
        st["x"] = _activations(g, T, H, dt)
        st["w"] = weight()
        if op.startswith("postnorm"):
            st["y"] = _activations(g, T, H, dt)
            st["post_w"] = weight() if c["post"] else None
            shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[c["gate"]]
            gate = None if shape is None else _randn(g, *shape) + (0.0 if c["sigmoid"] else 1.0)
            st["gate"] = gate if gate is None else gate.to(wd if c["gate"] == "channel" else dt)
            if not c["next"]:
                st["w"] = None
        if op.endswith("grad"):
            st["d_h"] = None if st["w"] is None else (_randn(g, T, H) * 0.1).to(dt)
            st["d_out"] = (_randn(g, T, H) * 0.1).to(dt)
    return st


# ---- plain forms --------------------------------------------------------------------------------------


def _plain_permute(c, x, ids, rows):
    row, count = _places(ids, c["E"], c["block"])
    rows.zero_()
    rows[row] = x.repeat_interleave(c["k"], 0)
    return rows, row.view(ids.shape).to(torch.int32), count.to(torch.int32)


def _plain_unpermute(c, rows, row_of, w):
    y = rows[row_of.long()].float()
    if w is not None:
        y = y * w[:, :, None]
    return y.sum(1).to(rows.dtype)


def _plain_unpermute_grad(rows, row_of, w, d_out, d_rows):
    d = d_out.float()
    at = row_of.long()
    d_rows.zero_()
    d_rows[at] = (w[:, :, None] * d[:, None, :]).to(rows.dtype)
    return d_rows, (rows[at].float() * d[:, None, :]).sum(2)


def _rstd(x):
    return torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)


def _norm_grad(x, r, g):
    """Gradient of n = x r in x, from that in n."""
    n = x * r
    return r * (g - n * (g * n).mean(1, keepdim=True))


def _plain_post(st):
    """(x, y, r_y, v, G, out) in 32 bits."""
    c = st["case"]
    x, y = st["x"].float(), st["y"].float()
    ry = _rstd(y) if c["post"] else None
    v = y * ry * st["post_w"].float() if c["post"] else y
    gate = None if st["gate"] is None else st["gate"].float()
    if c["sigmoid"]:
        gate = 1.0 / (1.0 + torch.exp(-gate))
    out = x * c["res_scale"] + c["scale"] * (v if gate is None else gate * v)
    return x, y, ry, v, gate, out


def _plain_post_grad(st):
    c, dt = st["case"], st["x"].dtype
    x, y, ry, v, gate, out = _plain_post(st)
    d = st["d_out"].float()
    res = {}
    if c["next"]:
        r, dh = _rstd(out), st["d_h"].float()
        d = d + _norm_grad(out, r, dh * st["w"].float())
        res["d_next_w"] = (dh * out * r).sum(0)
    res["d_x"] = (d * c["res_scale"]).to(dt)
    dv = d * c["scale"] if gate is None else d * c["scale"] * gate
    if gate is not None:
        dg = d * c["scale"] * v
        if c["sigmoid"]:
            dg = dg * gate * (1.0 - gate)
        res["d_gate"] = {"channel": lambda: dg.sum(0), "token": lambda: dg.sum(1, keepdim=True),
                         "full": lambda: dg.to(dt)}[c["gate"]]()
    if c["post"]:
        res["d_post_w"] = (dv * y * ry).sum(0)
        dv = _norm_grad(y, ry, dv * st["post_w"].float())
    res["d_y"] = dv.to(dt)
    return res


def _plain_lora(c, x, a, b, ids, scale, base):
    T, L, r = c["T"], c["L"], c["r"]
    on = (ids >= 0).float()
    l = ids.long().clamp(min=0)
    s = (scale[l] * on)[:, None]
    if T <= L:  # few tokens: each with its own adapter's weights
        h = (a[l].float() @ x.float()[:, :, None])[:, :, 0] * s
        d = (b[l].float() @ h[:, :, None])[:, :, 0]
    else:  # every adapter on every token, and a token's own kept
        h = (x.float() @ a.view(L * r, -1).float().t()).view(T, L, r)
        h = h * (s * (l[:, None] == torch.arange(L, device=x.device)))[:, :, None]
        d = h.view(T, L * r) @ b.float().transpose(1, 2).reshape(L * r, -1)
    return (base.float() + d).to(base.dtype)


def run(state):
    c = state["case"]
    op = c["op"]
    st = state
    if own:
        import mixture_experts_layer_scan_gb300 as moe

        if op == "permute":
            p = moe.moe_permute(st["x"], st["ids"], c["E"], c["block"], rows=st["rows"])
            return p.rows, p.row_of, p.expert_counts
        if op == "unpermute":
            if c["weighted"]:
                return moe.moe_unpermute(st["rows"], st["row_of"], st["w"])
            return moe.moe_permute_backward(st["rows"], st["row_of"])
        if op == "unpermute_grad":
            return moe.moe_unpermute_backward(st["d_out"], st["rows"], st["row_of"], st["w"], sorted_ids=st["sorted_ids"],
                                              num_post_pad=st["num_post_pad"], d_rows=st["d_rows"])
        if op == "prenorm":
            return moe.moe_prenorm(st["x"], st["w"], EPS)
        if op == "prenorm_grad":
            return moe.moe_prenorm_backward(st["d_h"], st["x"], st["w"], EPS)
        kw = dict(post_w=st.get("post_w"), gate=st.get("gate"), sigmoid=c.get("sigmoid"), scale=c.get("scale"),
                  res_scale=c.get("res_scale"), next_w=st.get("w"), eps=EPS)
        if op == "postnorm":
            out, h = moe.moe_postnorm(st["x"], st["y"], **kw)
            return out if h is None else (out, h)
        if op == "postnorm_grad":
            g = moe.moe_postnorm_backward(st["d_out"], st["d_h"], st["x"], st["y"], **kw)
            return {n: v for n, v in g._asdict().items() if v is not None}
        if "ws" not in st:  # a program keeps the workspace of its adapters
            n = moe.moe_lora_workspace_size(c["T"], c["K"], c["N"], c["r"], c["L"])
            st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return moe.moe_lora(st["x"], st["a"], st["b"], st["ids"], scale=st["scale"], base=st["base"], workspace=st["ws"])
    if op == "permute":
        return _plain_permute(c, st["x"], st["ids"], st["rows"])
    if op == "unpermute":
        return _plain_unpermute(c, st["rows"], st["row_of"], st["w"])
    if op == "unpermute_grad":
        return _plain_unpermute_grad(*(st[n] for n in ("rows", "row_of", "w", "d_out", "d_rows")))
    if op == "prenorm":
        x = st["x"].float()
        return (x * _rstd(x) * st["w"].float()).to(st["x"].dtype)
    if op == "prenorm_grad":
        x, dh = st["x"].float(), st["d_h"].float()
        r = _rstd(x)
        return _norm_grad(x, r, dh * st["w"].float()).to(st["x"].dtype), (dh * x * r).sum(0)
    if op == "postnorm":
        dt = st["x"].dtype
        out = _plain_post(st)[-1]
        return (out.to(dt), (out * _rstd(out) * st["w"].float()).to(dt)) if c["next"] else out.to(dt)
    if op == "postnorm_grad":
        return _plain_post_grad(st)
    return _plain_lora(c, *(st[n] for n in ("x", "a", "b", "ids", "scale", "base")))


def work(case):
    c = case
    op, T = c["op"], c["T"]
    if op == "lora":
        K, N, r = c["K"], c["N"], c["r"]
        ob = 2 if c["out"] == "bf16" else 4
        used = min(c["L"], T)
        return {"bytes": 2 * T * K + 2 * used * r * (K + N) + 2 * ob * T * N, "flops": 2 * T * r * (K + N)}
    H, e = c["H"], 2 if c["dtype"] == "bf16" else 4
    if op == "permute":
        k = c["k"]
        return {"bytes": e * T * H * (k + 1) + 8 * T * k, "flops": 0}
    if op == "unpermute":
        k = c["k"]
        return {"bytes": e * T * H * (k + 1) + 8 * T * k, "flops": 2 * T * k * H}
    if op == "unpermute_grad":
        k = c["k"]
        return {"bytes": e * T * H * (2 * k + 1) + 12 * T * k, "flops": 3 * T * k * H}
    full = c["gate"] == "full"
    if op == "prenorm":
        return {"bytes": e * (2 * T * H + H), "flops": 4 * T * H}
    if op == "prenorm_grad":
        return {"bytes": e * (3 * T * H + H) + 4 * H, "flops": 12 * T * H}
    if op == "postnorm":
        return {"bytes": e * (T * H * (3 + c["next"] + full) + 3 * H), "flops": 12 * T * H}
    return {"bytes": e * (T * H * (5 + c["next"] + 2 * full) + 3 * H) + 12 * H, "flops": 30 * T * H}


# ---- 64 bits ---------------------------------------------------------------------------------------------


def _grads64(outputs, seeds, leaves):
    """Gradients of sum_i <outputs[i], seeds[i]> in the leaves, by torch's own differentiation."""
    return torch.autograd.grad(sum((o * s).sum() for o, s in zip(outputs, seeds)), leaves)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    op, T = c["op"], c["T"]
    if op == "permute":
        # a stable sort by expert, written out: pairs of smaller experts (padded) and earlier pairs of its own come first
        ids = st["ids"].reshape(-1).cpu()
        rows = torch.zeros(st["rows"].shape, dtype=torch.float64, device="cuda")
        row_of, counts, at = torch.empty(len(ids), dtype=torch.int32), [], 0
        for e in range(c["E"]):
            mine = (ids == e).nonzero()[:, 0]
            row_of[mine] = torch.arange(at, at + len(mine), dtype=torch.int32)
            if len(mine):
                rows[at : at + len(mine)] = st["x"][(mine // c["k"]).cuda()].double()
            counts.append(len(mine))
            at += -(-len(mine) // c["block"]) * c["block"]
        return rows, row_of.view(T, c["k"]).cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda")
    if op in ("unpermute", "unpermute_grad"):
        out = torch.zeros(T, c["H"], dtype=torch.float64, device="cuda")
        d_rows = torch.zeros(st["rows"].shape if op == "unpermute_grad" else 0, dtype=torch.float64, device="cuda")
        d_w = torch.zeros(T, c["k"], dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            at = st["row_of"][:, j].long()
            w = 1.0 if st["w"] is None else st["w"][:, j, None].double()
            if op == "unpermute":
                out += w * st["rows"][at].double()
            else:
                d = st["d_out"].double()
                d_rows[at] = w * d
                d_w[:, j] = torch.linalg.vecdot(st["rows"][at].double(), d)
        return out if op == "unpermute" else (d_rows, d_w)
    if op == "lora":
        out = st["base"].double()
        for l in range(c["L"]):
            t = (st["ids"] == l).nonzero()[:, 0]
            if len(t):
                h = st["x"][t].double() @ st["a"][l].double().t()
                out[t] += float(st["scale"][l]) * (h @ st["b"][l].double().t())
        return out
    grad = op.endswith("grad")
    leaf = lambda n: None if st.get(n) is None else st[n].double().requires_grad_(grad)  # noqa: E731
    x, w = leaf("x"), leaf("w")

    def normed(v, weight):
        return v / torch.linalg.vector_norm(torch.cat([v, torch.full_like(v[:, :1], math.sqrt(EPS * c["H"]))], 1), dim=1,
                                            keepdim=True) * math.sqrt(c["H"]) * weight

    if op.startswith("prenorm"):
        h = normed(x, w)
        return _grads64([h], [st["d_h"].double()], [x, w]) if grad else h
    y, post_w, gate = leaf("y"), leaf("post_w"), leaf("gate")
    z = c["scale"] * (y if post_w is None else normed(y, post_w))
    if gate is not None:
        z = z * (torch.sigmoid(gate) if c["sigmoid"] else gate)
    out = c["res_scale"] * x + z
    h = None if w is None else normed(out, w)
    if not grad:
        return out if h is None else (out, h)
    names = [("d_x", x), ("d_y", y), ("d_post_w", post_w), ("d_gate", gate), ("d_next_w", w)]
    names = [(n, v) for n, v in names if v is not None]
    outs, seeds = ([out], [st["d_out"].double()]) if h is None else ([out, h], [st["d_out"].double(), st["d_h"].double()])
    return dict(zip([n for n, _ in names], _grads64(outs, seeds, [v for _, v in names])))
