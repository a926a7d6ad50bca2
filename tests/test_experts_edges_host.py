"""What the experts' operators promise beyond values, shown on the CPU."""
import pytest


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
