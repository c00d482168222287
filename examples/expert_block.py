"""An expert block from residual stream to residual stream: as a serving step runs it, and as a training step does.

  serving    the residual and its norm come in, the next residual and its norm go out:
             routing, block-scaled experts          moe_route_grouped, moe_forward_routed
             shared expert, an adapter per request  moe_quant_block, moe_gemm_block, moe_lora, moe_silu_quant_block
             norm, gate, residual, next norm        moe_postnorm
  training   the same frame around experts of one's own (here: a matrix each), forward and back:
             moe_prenorm, moe_permute, [experts], moe_unpermute, moe_postnorm and their gradients

Run it on a GB300 after the build:  python examples/expert_block.py [tokens]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mixture_experts_layer_scan_gb300 as moe  # noqa: E402

RULE = dict(score="sigmoid", n_group=8, topk_group=4, group_sum=2, renorm=True, scale=2.5)
TOPK = 8
EPS = 1e-6


class ServedBlock:
    """A layer's weights, its adapters (gate and up projection of the shared expert) and its norms."""

    def __init__(self, weights: dict, adapters: dict, norms: dict, scale: float = 1.0):
        self.w, self.a, self.n, self.scale = weights, adapters, norms, scale

    def first(self, x: torch.Tensor) -> torch.Tensor:
        """The norm that the first block of a stack needs before it."""
        return moe.moe_prenorm(x, self.n["pre"], EPS)

    def shared(self, h: torch.Tensor, requests: torch.Tensor):
        """The shared expert's output, and its gate and up projections with the requests' adapters."""
        w, a = self.w, self.a
        q, s = moe.moe_quant_block(h)
        gate_up = moe.moe_gemm_block(q, s, w["shared13"], w["shared13_scale"])
        moe.moe_lora(h, a["a"], a["b"], requests, scale=a["scale"], base=gate_up, out=gate_up)
        q, s = moe.moe_silu_quant_block(gate_up)
        return moe.moe_gemm_block(q, s, w["shared2"], w["shared2_scale"]), gate_up

    def experts(self, h: torch.Tensor) -> torch.Tensor:
        w = self.w
        _, topk_w, ids = moe.moe_route_grouped(h, w["router"], TOPK, bias=w["bias"], **RULE)
        return moe.moe_forward_routed(h, topk_w, ids, w["w13"], w["w2"], w["w13_scale"], w["w2_scale"],
                                      w_format="e4m3_block")

    def __call__(self, x: torch.Tensor, h: torch.Tensor, requests: torch.Tensor):
        """x [T,H]: the residual; h: its norm; requests int32 [T]: the adapter of each token (-1: none).
        The next residual (in x's place) and its norm."""
        y = self.experts(h)
        y += self.shared(h, requests)[0]
        return moe.moe_postnorm(x, y, post_w=self.n["post"], gate=self.n["gate"], scale=self.scale, next_w=self.n["next"],
                                eps=EPS, out=x)


def train_step(x, ids, topk_w, matrices, pre, post, gate, nxt, d_out, d_h, block: int = 16):
    """One block forward and back: (out, h, gradients by name).

    x [T,H]; ids, topk_w [T,k]: the routing; matrices [E,H,H]: an expert is h -> h . m^T; pre, post, nxt: the norms'
    weights; gate [H]; d_out, d_h: gradients of out and h."""
    E, H = matrices.shape[0], x.shape[1]
    n = moe.moe_prenorm(x, pre, EPS)
    # buffers of whole blocks: what lies behind the last block in use stays zero
    cap, _ = moe.moe_align_capacity(*ids.shape, E, block)
    blocks = -(-cap // block)
    inside, d_rows = (torch.zeros(blocks * block, H, dtype=x.dtype, device=x.device) for _ in range(2))
    p = moe.moe_permute(n, ids, E, block, rows=inside[:cap])
    used = torch.arange(blocks, device=x.device) < p.num_post_pad // block
    of = torch.zeros(blocks, dtype=torch.long, device=x.device)  # expert of each block
    of[: cap // block] = p.expert_ids.long()
    of = torch.where(used, of, 0)
    rows = torch.bmm(inside.view(-1, block, H), matrices[of].transpose(1, 2)).view(-1, H)[:cap]
    row_of = p.row_of
    y = moe.moe_unpermute(rows, row_of, topk_w)
    kw = dict(post_w=post, gate=gate, sigmoid=True, next_w=nxt, eps=EPS)
    out, h = moe.moe_postnorm(x, y, **kw)

    g = moe.moe_postnorm_backward(d_out, d_h, x, y, **kw)
    _, d_w = moe.moe_unpermute_backward(g.d_y, rows, row_of, topk_w, sorted_ids=p.sorted_ids,
                                        num_post_pad=p.num_post_pad, d_rows=d_rows[:cap])
    d_blocks = d_rows.view(-1, block, H)
    d_matrices = torch.zeros_like(matrices).index_add_(0, of, torch.bmm(d_blocks.transpose(1, 2), inside.view(-1, block, H)))
    d_in = torch.bmm(d_blocks, matrices[of]).view(-1, H)[:cap]
    d_n = moe.moe_permute_backward(d_in, row_of)
    d_x, d_pre = moe.moe_prenorm_backward(d_n, x, pre, EPS)
    grads = dict(x=g.d_x + d_x, topk_w=d_w, matrices=d_matrices, pre=d_pre, post=g.d_post_w, gate=g.d_gate, nxt=g.d_next_w)
    return out, h, grads


def main() -> None:
    from moe_synth import make_block_layer

    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 64
    H, I, E, I_shared, rank, requests = 2048, 768, 128, 1536, 16, 32
    dev = "cuda"
    weights = make_block_layer(H, I, E, I_shared=I_shared, device=dev)
    adapters = dict(a=(torch.randn(requests, rank, H, device=dev) * H ** -0.5).bfloat16(),
                    b=(torch.randn(requests, 2 * I_shared, rank, device=dev) * 0.1).bfloat16(),
                    scale=torch.ones(requests, device=dev))
    norms = {n: torch.ones(H, device=dev).bfloat16() for n in ("pre", "post", "gate", "next")}
    layer = ServedBlock(weights, adapters, norms, scale=0.25)
    x = torch.randn(tokens, H, device=dev).bfloat16()
    who = torch.randint(-1, requests, (tokens,), device=dev).int()
    h = layer.first(x)
    for _ in range(3):
        x, h = layer(x, h, who)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        x, h = layer(x, h, who)
    end.record()
    torch.cuda.synchronize()
    print(f"{tokens} tokens, {E} experts of {H} x {I}, {requests} adapters of rank {rank}: "
          f"{begin.elapsed_time(end) / 20 * 1e3:.1f} us a block, status {moe.strerror(moe.moe_get_status())}")


if __name__ == "__main__":
    main()
