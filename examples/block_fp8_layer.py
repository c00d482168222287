"""A fine-grained expert layer with block-scaled FP8 weights, as a serving step runs it.

  routing     sigmoid scores, a balance bias, 4 of 8 expert groups, top-8, weights scaled   moe_route_grouped
  experts     e4m3 weights with a scale per 128 x 128 block                                 moe_forward_routed
  shared      one dense expert beside them: quantise, product, SiLU product, product        moe_quant_block,
                                                                  moe_gemm_block, moe_silu_quant_block
  output      their sum

Run it on a GB300 after the build:  python examples/block_fp8_layer.py [tokens]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mixture_experts_layer_scan_gb300 as moe  # noqa: E402

RULE = dict(score="sigmoid", n_group=8, topk_group=4, group_sum=2, renorm=True, scale=2.5)
TOPK = 8


class BlockFp8Layer:
    """The weights of one layer and the workspace of its largest batch."""

    def __init__(self, weights: dict, max_tokens: int):
        self.w = weights
        E, two_i, H = weights["w13"].shape
        # (the plan, and with it the size, changes with the batch: a power of two covers those below it)
        sizes = [1 << b for b in range(max(1, max_tokens).bit_length())] + [max_tokens]
        need = max(moe.moe_workspace_size(T, H, two_i // 2, E, TOPK, moe.MOE_BF16, moe.MOE_E4M3_B128) for T in sizes)
        self.workspace = torch.empty(need, dtype=torch.uint8, device=weights["w13"].device)

    def shared(self, x: torch.Tensor) -> torch.Tensor:
        w = self.w
        q, s = moe.moe_quant_block(x)
        gate_up = moe.moe_gemm_block(q, s, w["shared13"], w["shared13_scale"])
        q, s = moe.moe_silu_quant_block(gate_up)
        return moe.moe_gemm_block(q, s, w["shared2"], w["shared2_scale"])

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        w = self.w
        _, topk_w, ids = moe.moe_route_grouped(x, w["router"], TOPK, bias=w["bias"], **RULE)
        T = x.shape[0]
        E, two_i, H = w["w13"].shape
        need = moe.moe_workspace_size(T, H, two_i // 2, E, TOPK, moe.MOE_BF16, moe.MOE_E4M3_B128)
        if need > self.workspace.numel():
            self.workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        y = moe.moe_forward_routed(x, topk_w, ids, w["w13"], w["w2"], w["w13_scale"], w["w2_scale"],
                                   workspace=self.workspace, w_format="e4m3_block")
        return y + self.shared(x)


def main() -> None:
    from moe_synth import make_block_layer

    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 64
    H, I, E = 2048, 768, 128
    layer = BlockFp8Layer(make_block_layer(H, I, E, I_shared=1536, device="cuda"), tokens)
    x = torch.randn(tokens, H, device="cuda").to(torch.bfloat16)
    for _ in range(3):
        out = layer(x)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        out = layer(x)
    end.record()
    torch.cuda.synchronize()
    status = moe.moe_get_status()
    print(f"{tokens} tokens, {E} experts of {H} x {I}: {begin.elapsed_time(end) / 20 * 1e3:.1f} us a layer, "
          f"output {tuple(out.shape)} rms {out.float().square().mean().sqrt().item():.3f}, status {moe.strerror(status)}")


if __name__ == "__main__":
    main()
