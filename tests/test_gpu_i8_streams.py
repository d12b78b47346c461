"""moe_layer with 8-bit experts on a stream other than the current one."""
import pytest
import torch

from mxfp4_mixture_experts_route_amd import _lib as moe
from test_gpu_i8 import busy, layer, same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,tile_m", [(5, 1), (40, 8)])
def test_layer_takes_nothing_that_the_current_stream_still_writes(T, tile_m):
    """Blocks let go on the current stream with writes to them still in flight (their values are
    valid everywhere: expert 1, row 1) are not what the layer on the other stream works in."""
    E, k, D, F = 8, 2, 200, 96
    logits, x, GU, DN = layer(5, T, E, k, D, F)
    want = moe.moe_layer(x, logits, GU[3], DN[3], k, tile_m, projection="i8")
    side = torch.cuda.Stream()
    side_pool = moe.moe_layer(x, logits, GU[3], DN[3], k, tile_m, projection="i8", stream=side)
    torch.cuda.synchronize()
    del side_pool
    keep = busy(torch.cuda.current_stream())
    late = [torch.empty_like(t).fill_(1) for t in want.values() if torch.is_tensor(t)
            for _ in range(3)]
    del late
    got = moe.moe_layer(x, logits, GU[3], DN[3], k, tile_m, projection="i8", stream=side)
    torch.cuda.synchronize()
    for key in ("ids", "w", "counts", "basep", "pos", "y"):
        same_bits(got[key], want[key], key)
    del keep
