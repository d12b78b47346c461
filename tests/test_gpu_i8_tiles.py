"""Every tile of the dense 8-bit products against 64 bits: each output type, rows and channels that
end inside a tile, K from one step to many (fewer steps than the groups that split K, odd numbers of
chunks), outputs that start and step off 16 bytes. Which tile a shape gets is checked on the host
(test_i8_tiles_host.py). Tolerances are those of test_gpu_i8.py."""
import pytest
import torch

from mxfp4_mixture_experts_route_amd import _lib as moe
from test_gpu_i8 import BF16, F16, F32, assert_out, log, rand_stack, ref_project, rng, same_bits

pytestmark = pytest.mark.gpu

# tile: [(rows, channels)]
DENSE = {
    "I8Few": [(17, 517), (45, 2047)],
    "I8Low": [(64, 5760), (63, 5761), (33, 6011)],
    "I8Half": [(128, 5760), (127, 5777), (65, 5701)],
    "I8Pair": [(250, 5701), (256, 5760)],
    "I8Mid": [(511, 5701)],
    "I8Wide": [(2045, 5701)],
    "I8Big": [(4090, 4085)],
}
SHAPES = [(tile, rows, N, K) for tile, sizes in DENSE.items() for rows, N in sizes
          for K in ((1, 64, 129, 200, 1003, 2880) if rows <= 256 else (1, 129, 200))]


@pytest.mark.parametrize("tile,rows,N,K", SHAPES)
def test_every_tile_in_every_type(tile, rows, N, K):
    log(f"{tile}: i8_gemm {rows}x{K} -> {N}")
    bias = (rows + K) % 2 == 0
    q, s, b, W = rand_stack(rows + N + K, 1, N, K, bias=bias)
    x = torch.randn(rows, K, generator=rng(rows), device="cuda").to(BF16)
    x[rows // 2] = 0.0
    aq, as_ = moe.i8_quantize(x)
    p, ref = ref_project(aq[:, :K], as_, q[0], s[0], None if b is None else b[0])
    for dt in (F32, BF16, F16):
        out = moe.i8_gemm(aq, as_, W, out_dtype=dt)
        assert_out(out, p, ref, f"{dt}")
        big = torch.full((rows, N + 5), 55.0, device="cuda", dtype=dt)
        moe.i8_gemm(aq, as_, W, out=big[:, 3:3 + N])
        same_bits(big[:, 3:3 + N], out, f"{dt}, strided")
        assert bool((big[:, :3] == 55).all()) and bool((big[:, 3 + N:] == 55).all())
        same_bits(moe.i8_linear(x, W, out_dtype=dt), out, f"{dt}, linear")
