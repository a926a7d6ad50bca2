"""What the experts' operators promise beyond values, shown on the CPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_rank_b200", "csrc")


@pytest.mark.parametrize("name,N,h,M,k", [
    ("moe_layer", 64, 4096, 512, 8), ("moe_layer_int8", 64, 4096, 512, 8), ("moe_layer", 64, 7168, 64, 8),
    ("moe_layer_int8", 64, 131072, 64, 16), ("experts", 64, 4096, 512, 8), ("experts_int8", 64, 4096, 512, 8),
    ("experts", 16, 131072, 64, 16), ("experts_int8", 16, 131072, 64, 16)])
def test_few_tokens_of_any_h_keep_no_rows_in_memory(name, N, h, M, k):
    """Up to 64 tokens (16 of the experts alone, more with few shared experts) take the few-token kernel whatever their h:
    the sums over their selections are its shared memory's, so the scratch holds the middles (s values a selection) and
    no rows of h values."""
    import mixture_experts_rank_b200 as m
    assert 0 < getattr(m, name + "_scratch_bytes")(N, h, 16, M, k) < N * k * h * 2


def function(source, name):
    """The text of a function from its name to the brace that closes it."""
    at = source.index("{", source.index(name))
    depth = 0
    for i in range(at, len(source)):
        depth += {"{": 1, "}": -1}.get(source[i], 0)
        if depth == 0:
            return source[at:i + 1]
    raise ValueError(name)


def test_epilogue_of_the_grouped_products_waits_with_a_limit():
    """Once a wait has run out its warp leaves the tiles.  What another warp waits for meanwhile has to run out too, and
    lanes must not leave their warp behind: no named barrier in the roles of the kernel, and every wait of the epilogue a
    whole warp's.  Shown in the source: on a GPU the failure would be a hang."""
    with open(os.path.join(CSRC, "experts_tc.cu")) as f:
        source = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"\bbar\.sync|barrier\.(cta\.)?sync|__barrier_sync", source)
    waits = re.findall(r"\w*wait\w*\s*\(", function(source, "__device__ void epilogue("))
    limited = {"warp_wait(", "warp_poll(", "tmem_wait_ld("}
    stores = {"bulk_wait_group_read<0>(", "bulk_wait_group("}  # for the thread's own copies
    assert waits and set(waits) <= limited | stores
    for name in ("bool warp_wait(", "bool warp_poll("):
        assert "__all_sync(0xffffffffu" in function(source, name)
