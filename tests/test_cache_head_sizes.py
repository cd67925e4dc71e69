"""The head sizes of a new paged cache (no GPU)."""
import pytest

from block_sparse_gqa_topk_gb300 import ops


@pytest.mark.parametrize("kind", [{}, {"fp8": True}, {"fp4": True}])
@pytest.mark.parametrize("d", [0, 1, 16, 63, 65, 96, 127, 129, 256])
def test_others_are_refused(d, kind):
    """In 4 bits an odd d is no cache of the even one below it."""
    with pytest.raises(ValueError, match="d must be 64 or 128"):
        ops.new_paged_cache(2, 1, page_size=16, d=d, d_idx=0, device="cpu", **kind)
