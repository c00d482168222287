"""What a GPU run of the adapters' kernels could not show without a fault, read from their source: counters that stay
in range, the order of tensor memory's readers and writers, and what is read before a kernel's dependency wait."""
import re

from test_block_bounded_waits_cpu import body, source


def constants(text: str) -> dict:
    """The file's integer constants, those made of others too."""
    known = {}
    for name, expr in re.findall(r"constexpr (?:int|long long) (\w+) = ([^;]+);", text):
        try:
            known[name] = int(eval(re.sub(r"(?<=\d)ll\b", "", expr).replace("/", "//"), {}, dict(known)))
        except (NameError, SyntaxError):
            pass
    return known


def test_columns_of_few_tokens_stay_below_2_31():
    """The column counter of a token at a time is 32 bits wide, and a CTA goes gridDim.y runs of columns further at each
    step: from the last column that a call may have, the sum has to stay in range, the order of tensor memory's readers and writers, and what is read before a kernel's dependency wait."""
    text = source("moe_lora.cu")
    limit = constants(source("moe_api.cu"))["kBlockMaxDim"]
    known = constants(text)
    assert re.search(r"for \(int n0 = blockIdx\.y \* kRun \+ .*; n0 \+= gridDim\.y \* kRun\)", body(text, "k_lora_expand(const LoraDev p)"))
    launch = body(text, "cudaError_t launch_few(const LoraDev& p, cudaStream_t s)")
    assert "MOE_LAUNCH((k_lora_expand<T, G>), dim3(rows, runs), " in launch
    grid = re.search(r"const int runs = (.*);", launch).group(1)
    grid = grid.replace("std::min", "min").replace("/", "//").replace("p.N", "N")
    for G in (1, 2, 4, 8, 16):
        run = 8 * (32 // G) * known["kExpandUnroll"]
        for N in (8, 4096, 1 << 30, limit - 1):
            runs = eval(grid, {"min": min}, {**known, "kRun": run, "N": N})
            assert 1 <= runs <= 65535
            # the furthest start of a step, the step behind it, and the columns of a run
            assert (N - 1) + runs * run + run < 1 << 31, (G, N, runs)


def test_new_h_is_written_behind_the_products_with_the_old():
    """An epilogue warp that puts the next block's h into tensor memory has waited for the products that read the
    last one's; its stores are ordered behind that wait by a fence of their own."""
    kernel = body(source("moe_lora.cu"), "k_lora_expand_tc(const __grid_constant__")
    stores = [m.start() for m in re.finditer(r"tmem_st4\(", kernel)]
    assert len(stores) == 2
    wait = kernel.rfind("mbar_wait_one(b.tfull", 0, stores[0])
    assert 0 < wait < kernel.find("tc_fence_after();", wait) < stores[0]
    ready = kernel.index("mbar_arrive(b.done)", stores[1])
    assert stores[1] < kernel.find("tmem_wait_st();", stores[1]) < kernel.find("tc_fence_before();", stores[1]) < ready


def test_nothing_of_an_earlier_kernel_is_read_ahead_of_the_wait():
    """The wait for the preceding kernel is what makes the memory of all before it visible, to the thread that waits:
    every thread of the tensor-core kernels passes it before it reads anything but the launch's own arguments."""
    text = source("moe_lora.cu")
    for name in ("k_lora_shrink_tc(const __grid_constant__", "k_lora_expand_tc(const __grid_constant__"):
        kernel = body(text, name)
        assert kernel.count("pdl_wait();") == 1
        before = kernel[: kernel.index("pdl_wait();")]
        assert "if (" not in before and "lora_blocks" not in before and "p." not in before.replace("p.bar_off", "")
