"""Which wait the status names when a rank of the fused combine + all-reduce gives up, whatever the order in which
its waits begin."""

import pytest
import torch

from moe_layer_top_b200 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_layer_top_b200 import build
    build.build()


@pytest.mark.parametrize("timeout_us", [1, 5, 200])
def test_status_names_the_wait_for_the_peers_although_others_run_out_earlier(timeout_us):
    """Rank 0 of sixteen alone, one token per chunk.  Its chunks belong to the blocks that have two chunks to add up
    first, so the other blocks' waits for the finished chunks begin, and with a short limit run out, before a wait
    for a peer has begun."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    world, topk, H = 16, 8, 16384
    T = sms + sms // world + 1                # chunks 0, 16, 32 .. belong to rank 0: to its first T / 16 blocks
    dev = torch.device("cuda")
    y = torch.ones((T * topk, H), dtype=torch.bfloat16, device=dev)
    ranks = [dict(y=y, partial=torch.zeros((T, H), dtype=torch.bfloat16, device=dev),
                  out=torch.zeros((T, H), dtype=torch.bfloat16, device=dev),
                  flags=torch.zeros(ops.combine_allreduce_flag_count(T, world), dtype=torch.int32, device=dev),
                  status=torch.zeros((1,), dtype=torch.int32, device=dev)) for _ in range(world)]
    for epoch in (1, 2, 3):
        ranks[0]["status"].zero_()
        ops.combine_allreduce(T, topk, H, 0, ranks, epoch=epoch, timeout_us=timeout_us)
        torch.cuda.synchronize()
        assert int(ranks[0]["status"]) == ops.MOE_STATUS_WAIT_TIMEOUT | 0x31
        assert int(ranks[0]["flags"][-1]) == epoch
        assert (ranks[0]["partial"] == topk).all()
    assert not any(int(r["status"]) for r in ranks[1:])
