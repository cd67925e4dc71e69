"""The bounded waits of the whole-cache decode over 4 bits, where four groups come together by TMA: a wait that
runs out ends the call with the device status, and the next call is right."""
import pytest
import torch

from block_sparse_gqa_topk_gb300 import _lib, ops
from test_gpu_decode_e2m1 import Batch4, tables  # noqa: F401
from test_gpu_decode_paged import query

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,G", [(64, 2), (128, 4), (128, 16)])  # two stages, and three for 16 heads
def test_a_wait_that_runs_out(d, G):
    """The first unit's copies of every span are left out, the next ones (of three stages) are on their way:
    every CTA gives up after its first wait and gives those their time to land."""
    lens, H = [90001, 0, 33000], 8
    batch = Batch4(lens, 128, H, d, 0, seed=101)
    q = query(len(lens), H * G, d, 102)
    call = lambda: ops.msa_decode_paged_dense(q, batch.cache, batch.table, batch.lens_t)  # noqa: E731
    want = call()
    assert ops.device_status() == 0
    for _ in range(2):
        _lib.msa_debug_set(20_000_000, _lib.MSA_DEBUG_WITHHOLD_LOAD)  # waits of 20 ms
        try:
            call()
            assert ops.device_status() == _lib.MSA_ERR_DEVICE_TIMEOUT
        finally:
            _lib.msa_debug_set(0, 0)
        o, lse = call()
        assert ops.device_status() == 0
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    batch.check_dense(q, d ** -0.5, *want)
