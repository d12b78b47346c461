"""The 8-bit products where the product of a row's and a channel's scale leaves the normal range of
f32: its value times the sum may be an ordinary number all the same.

The bound is that of test_gpu_i8.py, |out - ref| <= 2 * 2^-24 (2 |p| + |ref|) and one smallest step,
p being the product without bias: relative to p itself, whatever the size of the scales. Values that
the output type does not hold become infinite; a sum of zero stays zero (the bias alone).
"""
import pytest
import torch

from mxfp4_mixture_experts_route_amd import _lib as moe
from test_gpu_i8 import (ALPHA, BF16, F16, F32, LIMIT, NONE, SWIGLU, TINY, assert_out, csr, log,
                         rand_stack, ref_project, rng, same_bits)
from test_gpu_i8_tiles import DENSE

pytestmark = pytest.mark.gpu


def scales(seed, n, lo=-149, hi=127):
    """n f32 values over every exponent from 2^lo on, below 2^(hi + 1)."""
    g = rng(seed)
    e = torch.randint(lo, hi + 1, (n,), generator=g, device="cuda").double()
    return (torch.exp2(e) * (1 + torch.rand(n, generator=g, device="cuda").double())).float().clamp(
        max=torch.finfo(F32).max)


def assert_out_range(out, p, ref, what):
    """assert_out where the type holds the value, infinities where it does not (what lies within one
    rounding of the border is left out)."""
    top = torch.finfo(out.dtype).max
    eps = torch.finfo(out.dtype).eps
    past = ref.abs() > top * (1 + eps)
    inside = ref.abs() < top * (1 - eps)
    assert torch.equal(out[past].double(), torch.sign(ref[past]) * float("inf")), f"{what}: past the type"
    z = torch.zeros_like(ref)
    assert_out(torch.where(inside, out, torch.zeros_like(out)), torch.where(inside, p, z),
               torch.where(inside, ref, z), what)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("tile", list(DENSE))
def test_gemm_over_every_scale(tile, bias):
    K = 200
    rows, N = DENSE[tile][-1]
    log(f"{tile}: i8_gemm {rows}x{K} -> {N}, bias {bias}")
    q, _, _, _ = rand_stack(rows, 1, N, K)
    q[0, N // 3] = 0                                        # sums of zero: a channel, a row
    s = scales(1, N)
    b = (torch.randn(N, generator=rng(2), device="cuda").double() *
         scales(3, N, -140, 120).double()).float() if bias else None
    W = moe.I8Experts(q[0], s, b)
    aq, _ = moe.i8_quantize(torch.randn(rows, K, generator=rng(4), device="cuda").to(BF16))
    aq[rows // 2] = 0
    as_ = scales(5, rows)
    p, ref = ref_project(aq[:, :K], as_, q[0], s, b)
    p = torch.where(p == 0, torch.zeros_like(p), p)
    for dt in (F32, BF16, F16):
        out = moe.i8_gemm(aq, as_, W, out_dtype=dt)
        assert_out_range(out, p, ref, f"{dt}")
        nothing = b.to(dt) if bias else torch.zeros(N, device="cuda", dtype=dt)
        assert torch.equal(out[rows // 2], nothing), f"{dt}: a row of zeros"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 3, 8, 40])
def test_linear_over_every_scale(rows, dtype):
    """The one-launch kernel of few rows and the two launches of more."""
    N, K = 700, 333
    q, _, _, _ = rand_stack(rows, 1, N, K)
    s = scales(6, N)
    W = moe.I8Experts(q[0], s)
    x = torch.randn(rows, K, generator=rng(7), device="cuda").double()
    x = (x * scales(8, rows, -125, 119).double()[:, None]).to(dtype)
    aq, as_ = moe.i8_quantize(x)
    p, ref = ref_project(aq[:, :K], as_, q[0], s, None)
    out = moe.i8_linear(x, W, out_dtype=F32)
    assert_out_range(out, p, ref, "linear")
    same_bits(out, moe.i8_gemm(aq, as_, W, out_dtype=F32), "gemm")


@pytest.mark.parametrize("F,D", [(24, 100), (700, 131), (2049, 328)])
def test_moe_gemm_over_every_scale(F, D):
    counts, tile_m, tokens = [15, 130, 0, 63, 1], 16, 320
    cnt, basep, row_tok, mpad = csr(counts, tile_m, 1, tokens)
    q, _, _, _ = rand_stack(F, len(counts), 2 * F, D, glu=True)
    s = scales(9, len(counts) * 2 * F).reshape(len(counts), 2 * F)
    W = moe.I8Experts(q, s, glu=True)
    aq, _ = moe.i8_quantize(torch.randn(tokens, D, generator=rng(2), device="cuda").to(BF16))
    as_ = scales(10, tokens)
    out = moe.i8_moe_gemm(aq, as_, row_tok, W, cnt, basep, tile_m, mpad, NONE)
    h = moe.i8_moe_gemm(aq, as_, row_tok, W, cnt, basep, tile_m, mpad, SWIGLU, ALPHA, LIMIT)
    for e, c in enumerate(counts):
        span = slice(int(basep[e]), int(basep[e]) + c)
        t = row_tok[span].long()
        p, ref = ref_project(aq[t, :D], as_[t], q[e], s[e], None)
        assert_out_range(out[span], p, ref, f"expert {e}")
        # SwiGLU of small pairs, from the definition: gate and up carry 2^-22 of their size each, the
        # rest as in test_gpu_i8.test_moe_gemm
        g, u = ref[:, :F], ref[:, F:]
        small = (g.abs() < 4) & (u.abs() < LIMIT)
        gate, up = torch.where(small, g, torch.zeros_like(g)), torch.where(small, u, torch.zeros_like(u))
        want = gate * torch.sigmoid(ALPHA * gate) * (up + 1.0)
        tol = want.abs() * (2.0 ** -8 + (16 + (ALPHA * gate).abs() * 4) * 2.0 ** -23) + \
            gate.abs() * 2.0 ** -20 + TINY[BF16]
        bad = small & ~((h[span].double() - want).abs() <= tol)
        assert not bool(bad.any()), f"expert {e}: {int(bad.sum())} SwiGLU values outside"


@pytest.mark.parametrize("T,E,k,D,F", [(1, 8, 4, 200, 144), (3, 4, 2, 100, 96), (9, 8, 4, 130, 70)])
def test_decode_over_small_scales_is_the_chain_bit_for_bit(T, E, k, D, F):
    """Hidden values around 2^-110 from scales whose products are below 2^-126, and outputs of the
    same kind."""
    g = rng(T)
    logits = torch.randn(T, E, generator=g, device="cuda")
    x = (torch.randn(T, D, generator=g, device="cuda") * 2.0 ** -60).to(BF16)
    gq, _, _, _ = rand_stack(1, E, 2 * F, D, glu=True)
    dq, _, _, _ = rand_stack(2, E, D, F)
    gs = scales(11, E * 2 * F, -70, -62).reshape(E, 2 * F)
    gs[:, F:] = 2.0 ** 40                                     # up values of their own size
    GU = moe.I8Experts(gq, gs, glu=True)
    DN = moe.I8Experts(dq, scales(12, E * D, -22, -12).reshape(E, D))
    o = moe.i8_moe_decode(logits, x, GU, DN, k, ALPHA, LIMIT, want_d=True)
    c = moe.moe_layer(x, logits, GU, DN, k, 1, ALPHA, LIMIT, projection="i8")
    at = c["pos"].long().reshape(-1)
    same_bits(o["h"], c["h"][at], "h")
    same_bits(o["d"], c["d"][at], "d")
    same_bits(o["y"], c["y"], "y")
    hq, hs = moe.i8_quantize(o["h"])
    ids = o["ids"].reshape(-1)
    for r in range(T * k):
        e = int(ids[r])
        p, ref = ref_project(hq[r:r + 1, :F], hs[r:r + 1], dq[e], DN.s[e], None)
        assert float(p.abs().max()) > 2.0 ** -126
        assert_out(o["d"][r:r + 1], p, ref, f"d of row {r}")
