"""Refusals of the row, norm and adapter entry points (host checks: no call below reaches the device)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__

    __graft_entry__._builder().build()
    import mixture_experts_layer_scan_gb300 as m

    return m


P, ODD4, ODD2 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), ctypes.c_void_p(0x10002)
BIG = (1 << 31) - 1


def each_refused(call, args, bad, code):
    """call(*args) with one argument replaced at a time."""
    for i, v in bad:
        a = list(args)
        a[i] = v
        assert call(*a) == code, (i, v)


def test_permute(moe):
    f = moe.lib().moe_permute
    args = [P, P, 4, 64, 8, 2, 16, 1, P, P, P, P, P, P, None]
    each_refused(f, args, [(2, -1), (3, 0), (3, BIG), (4, 0), (4, 1025), (5, 0), (6, 0), (6, 1025), (2, 1 << 30)],
                 moe.MOE_ERR_ARG)
    each_refused(f, args, [(i, None) for i in (0, 1, 8, 9, 10, 11, 12)], moe.MOE_ERR_ARG)
    each_refused(f, args, [(7, 2), (7, 3), (7, -1)], moe.MOE_ERR_UNSUPPORTED)
    each_refused(f, args, [(i, ODD4) for i in (0, 1, 8, 10, 11, 12, 13)] + [(9, ODD2)], moe.MOE_ERR_ALIGNMENT)
    assert f(None, None, 0, 64, 8, 2, 16, 1, None, None, None, None, None, None, None) == moe.MOE_OK


def test_unpermute(moe):
    f, b = moe.lib().moe_unpermute, moe.lib().moe_permute_backward
    args = [P, 8, P, P, 4, 64, 2, 1, P, None]
    each_refused(f, args, [(1, -1), (4, -1), (5, 0), (5, BIG), (6, 0), (4, BIG), (0, None), (2, None), (8, None)],
                 moe.MOE_ERR_ARG)
    each_refused(f, args, [(7, 2)], moe.MOE_ERR_UNSUPPORTED)
    each_refused(f, args, [(0, ODD4), (2, ODD2), (3, ODD2), (8, ODD4)], moe.MOE_ERR_ALIGNMENT)
    assert f(None, 0, None, None, 0, 64, 2, 1, None, None) == moe.MOE_OK
    args = [P, 8, P, 4, 64, 2, 1, P, None]
    each_refused(b, args, [(1, -1), (3, -1), (4, 0), (5, 0), (0, None), (2, None), (7, None)], moe.MOE_ERR_ARG)
    each_refused(b, args, [(0, ODD4), (2, ODD2), (7, ODD4)], moe.MOE_ERR_ALIGNMENT)


def test_unpermute_backward(moe):
    f = moe.lib().moe_unpermute_backward
    args = [P, P, 8, P, P, P, P, 4, 64, 2, 1, P, P, None]
    each_refused(f, args, [(2, -1), (7, -1), (8, 0), (9, 0), (0, None), (1, None), (3, None), (5, None), (6, None)],
                 moe.MOE_ERR_ARG)
    assert f(P, P, 8, P, P, P, P, 4, 64, 2, 1, None, None, None) == moe.MOE_ERR_ARG
    each_refused(f, args, [(10, 2)], moe.MOE_ERR_UNSUPPORTED)
    each_refused(f, args, [(i, ODD4) for i in (0, 1, 5, 6, 11)] + [(i, ODD2) for i in (3, 4, 12)], moe.MOE_ERR_ALIGNMENT)


def test_norms(moe):
    lib = moe.lib()
    args = [P, P, 4, 64, 1e-6, 1, 1, P, None]
    each_refused(lib.moe_prenorm, args, [(2, -1), (3, 0), (4, -1.0), (4, float("nan")), (0, None), (1, None), (7, None)],
                 moe.MOE_ERR_ARG)
    each_refused(lib.moe_prenorm, args, [(3, 16385), (5, 2), (6, 2)], moe.MOE_ERR_UNSUPPORTED)
    each_refused(lib.moe_prenorm, args, [(0, ODD4), (1, ODD4), (7, ODD4)], moe.MOE_ERR_ALIGNMENT)
    assert lib.moe_prenorm(None, None, 0, 64, 1e-6, 1, 1, None, None) == moe.MOE_OK
    need = moe.moe_norm_workspace_size(4, 64)
    args = [P, P, P, 4, 64, 1e-6, 1, 1, P, P, P, need, None]
    f = lib.moe_prenorm_backward
    each_refused(f, args, [(3, -1), (4, 0), (5, -1.0)] + [(i, None) for i in (0, 1, 2, 8, 10)], moe.MOE_ERR_ARG)
    each_refused(f, args, [(4, 16385), (6, 2), (7, 3)], moe.MOE_ERR_UNSUPPORTED)
    each_refused(f, args, [(i, ODD4) for i in (0, 1, 2, 8, 9, 10)], moe.MOE_ERR_ALIGNMENT)
    each_refused(f, args, [(11, need - 1)], moe.MOE_ERR_WORKSPACE)
    for bad in ((-1, 64), (4, 0)):
        with pytest.raises(moe.MoeError):
            moe.moe_norm_workspace_size(*bad)


def test_postnorms(moe):
    lib = moe.lib()

    def rule(**over):
        d = dict(eps=1e-6, scale=1.0, res_scale=1.0, gate=1, gate_sigmoid=0, gate_dtype=1, w_dtype=1)
        return ctypes.byref(moe.moe_postnorm_rule(**{**d, **over}))

    f, args = lib.moe_postnorm, [P, P, P, P, P, 4, 64, 1, rule(), P, P, None]
    each_refused(f, args, [(i, None) for i in (0, 1, 3, 4, 8, 9, 10)] + [(5, -1), (6, 0)], moe.MOE_ERR_ARG)
    each_refused(f, args, [(8, rule(gate=4)), (8, rule(gate=-1)), (8, rule(gate=0)), (8, rule(eps=-1.0))],
                 moe.MOE_ERR_ARG)
    each_refused(f, args, [(8, rule(w_dtype=2)), (8, rule(gate_dtype=3)), (7, 2), (6, 16385)], moe.MOE_ERR_UNSUPPORTED)
    each_refused(f, args, [(i, ODD4) for i in (0, 1, 2, 3, 4, 9, 10)], moe.MOE_ERR_ALIGNMENT)
    need = moe.moe_norm_workspace_size(4, 64)
    f = lib.moe_postnorm_backward
    args = [P, P, P, P, P, P, P, 4, 64, 1, rule(), P, P, P, P, P, P, need, None]
    # (2: x, 3: y, 5: gate, 6: next_w beside d_h, 4: post_w beside its gradient)
    each_refused(f, args, [(i, None) for i in (2, 3, 4, 5, 6, 10, 11, 12, 16)] + [(7, -1), (8, 0)], moe.MOE_ERR_ARG)
    each_refused(f, args, [(i, ODD4) for i in (0, 1, 2, 3, 4, 5, 6, 11, 12, 13, 14, 15, 16)], moe.MOE_ERR_ALIGNMENT)
    each_refused(f, args, [(17, need - 1)], moe.MOE_ERR_WORKSPACE)
    each_refused(f, args, [(10, rule(gate=2, gate_dtype=2)), (9, 4)], moe.MOE_ERR_UNSUPPORTED)


def test_lora(moe):
    f = moe.lib().moe_lora
    need = moe.moe_lora_workspace_size(4, 64, 72, 16, 3)
    args = [P, P, P, P, P, P, 4, 64, 72, 16, 3, 1, P, P, need, None]
    each_refused(f, args, [(6, -1), (7, 0), (8, 0), (9, 0), (10, 0), (10, 1024), (6, BIG), (7, BIG), (8, BIG)] +
                 [(i, None) for i in (0, 1, 2, 3, 12, 13)], moe.MOE_ERR_ARG)
    each_refused(f, args, [(7, 60), (8, 70), (9, 12), (9, 136), (11, 2)], moe.MOE_ERR_UNSUPPORTED)
    each_refused(f, args, [(i, ODD4) for i in (0, 1, 2, 5, 12, 13)] + [(3, ODD2), (4, ODD2)], moe.MOE_ERR_ALIGNMENT)
    each_refused(f, args, [(14, need - 1)], moe.MOE_ERR_WORKSPACE)
    assert f(None, None, None, None, None, None, 0, 64, 72, 16, 3, 1, None, None, 0, None) == moe.MOE_OK


def test_python_checks(moe):
    """Shapes, types and devices that the binding refuses before the library sees them (CPU tensors: nothing is
    launched, and no host address reaches a kernel)."""
    x, w = torch.zeros(4, 64), torch.zeros(64)
    ids, rows = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, 64)
    tw = torch.zeros(4, 2)
    calls = [
        lambda: moe.moe_permute(x.half(), ids, 8), lambda: moe.moe_permute(x, ids.long(), 8),
        lambda: moe.moe_permute(x, ids[:3], 8), lambda: moe.moe_permute(x, ids, 8),
        lambda: moe.moe_unpermute(rows, ids.long()), lambda: moe.moe_unpermute(rows, ids, tw.double()),
        lambda: moe.moe_unpermute(rows, ids, tw[:, :1]), lambda: moe.moe_unpermute(rows, ids, tw),
        lambda: moe.moe_permute_backward(rows.half(), ids), lambda: moe.moe_permute_backward(rows, ids),
        lambda: moe.moe_unpermute_backward(x[:3], rows, ids), lambda: moe.moe_unpermute_backward(x.half(), rows, ids),
        lambda: moe.moe_unpermute_backward(x, rows, ids, sorted_ids=ids[0]), lambda: moe.moe_unpermute_backward(x, rows, ids),
        lambda: moe.moe_prenorm(x, w[:32]), lambda: moe.moe_prenorm(x.half(), w), lambda: moe.moe_prenorm(x, w),
        lambda: moe.moe_prenorm_backward(x[:2], x, w), lambda: moe.moe_prenorm_backward(x, x, w),
        lambda: moe.moe_postnorm(x, x[:2]), lambda: moe.moe_postnorm(x, x, gate=w[:5]),
        lambda: moe.moe_postnorm(x, x, post_w=w, next_w=w.bfloat16()), lambda: moe.moe_postnorm(x, x),
        lambda: moe.moe_postnorm_backward(x, x, x, x), lambda: moe.moe_postnorm_backward(x[:2], None, x, x),
        lambda: moe.moe_postnorm_backward(x, None, x, x),
    ]
    xb, a, b = x.bfloat16(), torch.zeros(3, 8, 64).bfloat16(), torch.zeros(3, 16, 8).bfloat16()
    one = ids[:, 0].contiguous()
    calls += [
        lambda: moe.moe_lora(x, a, b, one), lambda: moe.moe_lora(xb, a, b[:2], one),
        lambda: moe.moe_lora(xb, a[:, :, :32], b, one), lambda: moe.moe_lora(xb, a, b, one.long()),
        lambda: moe.moe_lora(xb, a, b, one[:3]), lambda: moe.moe_lora(xb, a, b, one, base=torch.zeros(4, 8)),
        lambda: moe.moe_lora(xb, a, b, one, scale=torch.zeros(2)), lambda: moe.moe_lora(xb, a, b, one),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()


def test_row_widths(moe):
    """Rows too wide for the kernels' 32-bit offsets in a row."""
    wide = 1 << 25
    for f, args, at in ((moe.lib().moe_permute, [P, P, 1, 64, 8, 2, 16, 1, P, P, P, P, P, P, None], 3),
                        (moe.lib().moe_unpermute, [P, 8, P, P, 1, 64, 2, 1, P, None], 5),
                        (moe.lib().moe_permute_backward, [P, 8, P, 1, 64, 2, 1, P, None], 4),
                        (moe.lib().moe_unpermute_backward, [P, P, 8, P, P, P, P, 1, 64, 2, 1, P, P, None], 8)):
        each_refused(f, args, [(at, wide), (at, wide + 1)], moe.MOE_ERR_ARG)


def test_postnorm_rule_follows_its_numbers(moe):
    """A scale that is a tensor: its present value counts, not its identity."""
    x, scale = torch.zeros(4, 64), torch.tensor(0.5)
    rule = lambda: moe._postnorm(x, x, None, None, False, scale, 1.0, None, 1e-6)[-1]._obj.scale  # noqa: E731
    assert rule() == 0.5
    scale.fill_(2.0)
    assert rule() == 2.0
