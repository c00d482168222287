"""After a bounded wait gives up, the block-scaled products still end: what each lane learnt of its own wait must
not decide which lanes of a warp meet a warp-wide instruction.  A wait that runs out cannot be brought about on a
GPU without breaking a kernel, so this is read from the source."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_scan_gb300", "csrc")


def body(text: str, head: str) -> str:
    """The braces' content that follows the first place of `head`."""
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at : i + 1]
    raise AssertionError(f"{head}: no end")


def source(name: str) -> str:
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_swap_ab_rows_are_stored_by_whole_warps():
    text = source("moe_gemm_block.cu")
    assert "__shfl_xor_sync" in body(text, "void bg_store_row(")  # the store needs all lanes of its warp
    epilogue = body(text, "k_gemm_block(const __grid_constant__")
    epilogue = epilogue[epilogue.index("float2 acc[NT / 2]"):]
    last_wait = max(m.end() for m in re.finditer(r"ok = mbar_wait_one\(", epilogue))
    stores = [m.start() for m in re.finditer(r"bg_store_row<", epilogue)]
    assert len(stores) == 2
    vote = epilogue.find("ok = __all_sync(0xffffffffu, ok);", last_wait)
    assert last_wait < vote < min(stores), "the stores hang on one lane's own wait"


def test_pair_rows_are_stored_by_whole_warps():
    text = source("moe_gemm_block.cu")
    kernel = body(text, "k_gemm_block_pair(const __grid_constant__")
    assert "f.ok = " not in kernel[kernel.index("setmaxnreg_inc<"):].replace("f.ok = true;", "")
    for name in ("tma_store_2d(", "bp_store_box<"):  # both meet __syncwarp: under a vote, never under f.ok alone
        for m in re.finditer(re.escape(name), kernel):
            guard = kernel.rfind("f.ok", 0, m.start())
            assert kernel[:guard].endswith("__all_sync(0xffffffffu, ")
