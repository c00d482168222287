"""What a GPU run of the norms' kernels could not show without a race, read from their source."""
from test_block_bounded_waits_cpu import body, source


def test_a_single_warp_orders_its_reads_before_the_refill():
    """The ring's oldest row is overwritten behind the row's sums: with one warp to a CTA the sums have no barrier of the CTA,
    so the warp's own stands there (a shuffle orders no memory)."""
    text = source("moe_norm.cuh")
    sums = body(text, "void block_sums(")
    alone = sums[sums.index("if (warps == 1)"): sums.index("if (lane == 0)")]
    assert alone.index("__syncwarp();") < alone.index("return;")
    for name, kernel in (("moe_norm.cu", "k_norm(const __grid_constant__"), ("moe_norm_grad.cu", "k_norm_grad(const __grid_constant__")):
        k = body(source(name), kernel)
        refills = k.count("rows.refill(t);")
        assert refills == 2 and all(part.rstrip().endswith("block_sums(v, s2[0]);") for part in k.split("rows.refill(t);")[:-1])
