"""Refusals of the grouped-routing and block-scaled FP8 entry points (host checks: no call below
reaches the device)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__

    __graft_entry__._builder().build()
    import mixture_experts_layer_scan_gb300 as m

    return m


FAKE, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)


def rule(moe, **over):
    d = dict(score=1, n_group=8, topk_group=4, group_sum=2, renorm=1, scale=1.0)
    d.update(over)
    return ctypes.byref(moe.moe_route_rule(**d))


@pytest.mark.parametrize("over", [dict(score=2), dict(score=-1), dict(n_group=0), dict(n_group=33), dict(n_group=7),
                                  dict(topk_group=0), dict(topk_group=9), dict(group_sum=0), dict(group_sum=3),
                                  dict(n_group=32, topk_group=1)])
def test_rules_out_of_range(moe, over):
    lib = moe.lib()
    assert lib.moe_topk_grouped(FAKE, None, 4, 64, 8, rule(moe, **over), FAKE, FAKE, None) == moe.MOE_ERR_ARG
    assert lib.moe_route_grouped(FAKE, FAKE, None, 4, 64, 64, 8, rule(moe, **over), 1, FAKE, FAKE, FAKE,
                                 None) == moe.MOE_ERR_ARG


def test_grouped_routing_arguments(moe):
    lib, r = moe.lib(), rule(moe)
    assert lib.moe_topk_grouped(FAKE, None, 4, 64, 8, None, FAKE, FAKE, None) == moe.MOE_ERR_ARG
    for T, E, k in ((-1, 64, 8), (4, 0, 1), (4, 1032, 8), (4, 64, 0), (4, 64, 33), (4, 8, 9)):
        assert lib.moe_topk_grouped(FAKE, None, T, E, k, r, FAKE, FAKE, None) == moe.MOE_ERR_ARG
    for ptrs in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None)):
        assert lib.moe_topk_grouped(ptrs[0], None, 4, 64, 8, r, ptrs[1], ptrs[2], None) == moe.MOE_ERR_ARG
    assert lib.moe_topk_grouped(ODD, None, 4, 64, 8, r, FAKE, FAKE, None) == moe.MOE_ERR_ALIGNMENT
    assert lib.moe_topk_grouped(FAKE, ctypes.c_void_p(0x1002), 4, 64, 8, r, FAKE, FAKE, None) == moe.MOE_ERR_ALIGNMENT
    assert lib.moe_topk_grouped(None, None, 0, 64, 8, r, None, None, None) == moe.MOE_OK
    assert lib.moe_route_grouped(FAKE, FAKE, None, 4, 60, 64, 8, r, 1, FAKE, FAKE, FAKE, None) == moe.MOE_ERR_UNSUPPORTED
    assert lib.moe_route_grouped(FAKE, FAKE, None, 4, 64, 64, 8, r, 2, FAKE, FAKE, FAKE, None) == moe.MOE_ERR_UNSUPPORTED
    assert lib.moe_route_grouped(FAKE, FAKE, None, 4, 64, 64, 8, r, 1, None, FAKE, FAKE, None) == moe.MOE_ERR_ARG


def test_quant_arguments(moe):
    lib = moe.lib()
    for f in (lib.moe_quant_block, lib.moe_silu_quant_block):
        assert f(FAKE, -1, 128, 1, FAKE, FAKE, None) == moe.MOE_ERR_ARG
        assert f(FAKE, 4, 0, 1, FAKE, FAKE, None) == moe.MOE_ERR_ARG
        assert f(FAKE, 4, 120, 1, FAKE, FAKE, None) == moe.MOE_ERR_UNSUPPORTED
        assert f(FAKE, 4, 128, 2, FAKE, FAKE, None) == moe.MOE_ERR_UNSUPPORTED
        assert f(None, 4, 128, 1, FAKE, FAKE, None) == moe.MOE_ERR_ARG
        assert f(FAKE, 4, 128, 1, None, FAKE, None) == moe.MOE_ERR_ARG
        assert f(FAKE, 4, 128, 1, FAKE, None, None) == moe.MOE_ERR_ARG
        assert f(ODD, 4, 128, 1, FAKE, FAKE, None) == moe.MOE_ERR_ALIGNMENT
        assert f(FAKE, 4, 128, 1, FAKE, ctypes.c_void_p(0x1002), None) == moe.MOE_ERR_ALIGNMENT
        assert f(None, 0, 128, 1, None, None, None) == moe.MOE_OK


def test_gemm_arguments(moe):
    f = moe.lib().moe_gemm_block
    assert f(FAKE, FAKE, FAKE, FAKE, -1, 8, 128, 1, FAKE, None) == moe.MOE_ERR_ARG
    assert f(FAKE, FAKE, FAKE, FAKE, 4, 0, 128, 1, FAKE, None) == moe.MOE_ERR_ARG
    assert f(FAKE, FAKE, FAKE, FAKE, 4, 8, 0, 1, FAKE, None) == moe.MOE_ERR_ARG
    assert f(FAKE, FAKE, FAKE, FAKE, 4, 8, 136, 1, FAKE, None) == moe.MOE_ERR_UNSUPPORTED
    assert f(FAKE, FAKE, FAKE, FAKE, 4, 8, 128, 2, FAKE, None) == moe.MOE_ERR_UNSUPPORTED
    for i in range(4):
        p = [FAKE] * 4
        p[i] = None
        assert f(*p, 4, 8, 128, 1, FAKE, None) == moe.MOE_ERR_ARG
    assert f(FAKE, FAKE, FAKE, FAKE, 4, 8, 128, 1, None, None) == moe.MOE_ERR_ARG
    assert f(ODD, FAKE, FAKE, FAKE, 4, 8, 128, 1, FAKE, None) == moe.MOE_ERR_ALIGNMENT
    assert f(FAKE, FAKE, FAKE, FAKE, 4, 8, 128, 1, ODD, None) == moe.MOE_ERR_ALIGNMENT
    assert f(FAKE, ODD, FAKE, ctypes.c_void_p(0x1002), 4, 8, 128, 1, FAKE, None) == moe.MOE_ERR_ALIGNMENT
    assert f(None, None, None, None, 0, 8, 128, 1, None, None) == moe.MOE_OK


def test_python_checks(moe):
    """Shapes and types that the binding refuses before the library sees them (CPU tensors: nothing is launched)."""
    import torch

    f8, f32 = torch.float8_e4m3fn, torch.float32
    a, sa, w, sw = torch.zeros(4, 256, dtype=f8), torch.zeros(4, 2), torch.zeros(300, 256, dtype=f8), torch.zeros(3, 2)
    for bad in ((a, sa[:, :1], w, sw), (a, sa, w[:, :128], sw), (a, sa, w, sw[:2]), (a.float(), sa, w, sw),
                (a, sa.double(), w, sw)):
        with pytest.raises(ValueError):
            moe.moe_gemm_block(*bad)
    with pytest.raises(ValueError):
        moe.moe_gemm_block(a, sa, w, sw, out=torch.zeros(4, 256, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        moe.moe_quant_block(torch.zeros(4, 256), q=torch.zeros(4, 128, dtype=f8))
    with pytest.raises(ValueError):
        moe.moe_silu_quant_block(torch.zeros(4, 255))
    with pytest.raises(ValueError):
        moe.moe_topk_grouped(torch.zeros(4, 64, dtype=torch.bfloat16), 8)
    with pytest.raises(ValueError):
        moe.moe_topk_grouped(torch.zeros(4, 64), 8, bias=torch.zeros(32))
    x, tw, ids = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 2), torch.zeros(4, 2, dtype=torch.int32)
    w13, w2 = torch.zeros(8, 256, 256, dtype=f8), torch.zeros(8, 256, 128, dtype=f8)
    s13, s2 = torch.zeros(8, 2, 2), torch.zeros(8, 2, 1)
    for bad in ((x, tw, ids.long(), w13, w2, s13, s2), (x, tw[:2], ids, w13, w2, s13, s2),
                (x, tw, ids, w13, w2, s13[:, :1], s2), (x, tw, ids, w13, w2, s13, None),
                (x, tw, ids, w13.to(f32), w2, s13, s2), (x, tw, ids, w13, w2[:, :128], s13, s2)):
        with pytest.raises(ValueError):
            moe.moe_forward_routed(*bad, w_format="e4m3_block")


def test_block_weight_plans(moe):
    B = moe.MOE_E4M3_B128
    d = moe.moe_plan_info(64, 4096, 2048, 64, 8, moe.MOE_BF16, B)
    assert d["orientation"] == moe.ORIENT_SWAP_AB and d["block"] == 64
    assert moe.moe_plan_info(16, 4096, 2048, 64, 8, moe.MOE_BF16, B)["block"] == 16
    # above 64 tokens: blocks of 64 up to 32 pairs per expert, CTA pairs beyond
    s = moe.moe_plan_info(256, 4096, 2048, 64, 8, moe.MOE_BF16, B)
    assert s["orientation"] == moe.ORIENT_SWAP_AB and s["block"] == 64 and s["cta_pair"] == 0
    p = moe.moe_plan_info(257, 4096, 2048, 64, 8, moe.MOE_BF16, B)
    assert p["orientation"] == moe.ORIENT_TOKEN_MAJOR and p["block"] == 128 and p["cta_pair"] == 1
    assert moe.moe_plan_info(48, 4096, 2048, 64, 8, moe.MOE_BF16, B, {"orientation": 2})["cta_pair"] == 1
    for args, opts in (((64, 4000, 2048, 64, 8), None), ((64, 4096, 2000, 64, 8), None),
                       ((4096, 4096, 2048, 64, 8), {"cta_pair": 2})):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_plan_info(*args, moe.MOE_BF16, B, opts)
        assert e.value.code == moe.MOE_ERR_UNSUPPORTED
    with pytest.raises(moe.MoeError) as e:  # fp32 activations
        moe.moe_plan_info(64, 4096, 2048, 64, 8, moe.MOE_F32, B)
    assert e.value.code == moe.MOE_ERR_UNSUPPORTED
    with pytest.raises(moe.MoeError) as e:
        moe.moe_plan_info(64, 4096, 2048, 64, 8, moe.MOE_BF16, 5)
    assert e.value.code == moe.MOE_ERR_ARG
    lib, ws = moe.lib(), ctypes.c_void_p(0x100000)
    # no block scales: refused before anything is launched
    assert lib.moe_forward(FAKE, FAKE, FAKE, FAKE, 4, 512, 512, 8, 2, 1, 1, B, None, None, FAKE, ws, 1 << 30, None,
                           None) == moe.MOE_ERR_ARG
