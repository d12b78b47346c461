"""The 8-bit integer projections against plain implementations in 64 bits.

Codes and scales of quantized rows are compared bit for bit (both sides round the exact
quotient). Products are exact integers on both sides, so an fp32 output carries three roundings
(the sum to f32, the product of the scales, the fused multiply-add): |out - ref| <=
2^-24 (2 |p| + |ref|) with p the product without bias, doubled here for second-order terms; an
output of fewer bits adds half a step, eps / 2 * |ref|. The results of one call and of another
that computes the same rows in another way are compared bit for bit.
"""
import numpy as np
import pytest
import torch

import oracle
from mxfp4_mixture_experts_route_amd import _lib as moe

pytestmark = pytest.mark.gpu

ALPHA, LIMIT = 1.702, 7.0
NONE, SWIGLU = moe.MOE_ACT_NONE, moe.MOE_ACT_SWIGLU_OAI
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TINY = {BF16: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -149}   # half the smallest step (f32: one)


def log(*a):
    print(*a, flush=True)


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand_rows(seed, rows, K, dtype):
    """Rows over many magnitudes with a row of zeros and one of the type's smallest values."""
    g = rng(seed)
    x = torch.randn(rows, K, generator=g, device="cuda")
    lo, hi = (-10, 10) if dtype == F16 else (-60, 60)
    x = x * torch.exp2(torch.randint(lo, hi, (rows, 1), generator=g, device="cuda").float())
    if rows > 2:
        x[1] = 0.0
        x[2] = torch.randn(K, generator=g, device="cuda") * torch.finfo(dtype).smallest_normal / 8
    return x.to(dtype)


def rand_stack(seed, E, N, K, bias=True, glu=False):
    g = rng(seed)
    q = torch.randint(-127, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    q[:, :1] = -128            # the quantizer never makes it; a weight may hold it
    s = torch.rand(E, N, generator=g, device="cuda") * (2.0 / 73.0 / K ** 0.5) + 1e-6
    b = torch.randn(E, N, generator=g, device="cuda") if bias else None
    return q, s, b, moe.I8Experts(q, s, b, glu=glu)


def ref_quantize(x):
    """(codes int64, scale f32): the definition in 64 bits."""
    v = x.double()
    top = v.abs().amax(dim=1)
    bad = ~torch.isfinite(top)
    top = torch.where(bad, torch.zeros_like(top), top)
    safe = torch.where(top > 0, top, torch.ones_like(top))[:, None]
    q = torch.round(127.0 * torch.where(bad[:, None], torch.zeros_like(v), v) / safe)
    s = (top / 127.0).float()
    s[bad] = float("nan")
    return q.long(), s


def ref_project(aq, as_, q, s, b):
    """(p, p + bias) in f64 of codes aq [rows][K], scales, and one matrix."""
    p = (aq.double() @ q.double().t().contiguous()) * as_.double()[:, None] * s.double()
    return p, p if b is None else p + b.double()


def assert_out(out, p, ref, what):
    o = out.double()
    eps = torch.finfo(out.dtype).eps / 2
    tol = 2.0 * 2.0 ** -24 * (2.0 * p.abs() + ref.abs()) + TINY[out.dtype]
    if out.dtype != F32:
        tol = tol + eps * ref.abs() * (1 + 2.0 ** -20)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(o), nan), f"{what}: NaN elsewhere"
    bad = ~nan & ~((o - ref).abs() <= tol)
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: "
                             f"{float(o[i])!r} for {float(ref[i])!r}, tolerance {float(tol[i])!r}")


def same_bits(a, b, what):
    assert a.dtype == b.dtype and a.shape == b.shape, what
    it = {2: torch.int16, 4: torch.int32, 1: torch.int8}[a.element_size()]
    assert torch.equal(a.contiguous().view(it), b.contiguous().view(it)), what


# ---------------------------------------------------------------------------------------------
# rows
# ---------------------------------------------------------------------------------------------

def check_quantize(x, q, s, what):
    K = x.shape[1]
    rq, rs = ref_quantize(x)
    assert torch.equal(q[:, :K].long(), rq), what
    assert not bool(q[:, K:].any()), f"{what}: padding"
    assert torch.equal(torch.isnan(s), torch.isnan(rs)), what
    assert torch.equal(torch.nan_to_num(s), torch.nan_to_num(rs)), what


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 63), (5, 64), (4, 65), (7, 1003), (9, 2880),
                                    (1030, 2880), (1025, 100), (3, 8200), (1024, 4100), (2, 65536),
                                    (2051, 2880), (2049, 100), (2050, 4096), (2050, 4097)])
def test_quantize_bit_exact(rows, K, dtype):
    log(f"i8_quantize {rows}x{K} {dtype}")
    x = rand_rows(rows * 7 + K, rows, K, dtype)
    q, s = moe.i8_quantize(x)
    check_quantize(x, q, s, f"{rows}x{K}")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_quantize_ties_and_near_ties(dtype):
    """Rows whose quotients 127 x / m are exact ties (m = 127 * 2^j: every half step of the code
    is a value of the type), and all the significands of bf16 against each other."""
    half = torch.arange(-254, 255, device="cuda").float() / 2.0            # ..., j / 2, ...
    rows = [half * 2.0 ** e for e in (-8, 0, 5)]
    rows.append(torch.nextafter(half, torch.full_like(half, 1e9)))
    rows.append(torch.nextafter(half, torch.full_like(half, -1e9)))
    x = torch.stack(rows).to(dtype)
    q, s = moe.i8_quantize(x)
    check_quantize(x, q, s, "ties")
    m = torch.arange(128, 256, device="cuda").float()[:, None]
    v = torch.arange(0, 256, device="cuda").float()[None, :]
    for e in (0, 1, 2, 6, 8):
        x = torch.where(v * 2.0 ** -e <= m, v * 2.0 ** -e, m)
        x = torch.cat([x, m], dim=1).to(dtype)
        q, s = moe.i8_quantize(x)
        check_quantize(x, q, s, f"significands at 2^-{e}")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_quantize_extremes_and_non_finite_rows(dtype):
    fi = torch.finfo(dtype)
    K = 130
    x = torch.randn(9, K, generator=rng(3), device="cuda").to(dtype)
    x[0] = fi.max
    x[1] = -fi.max
    x[2, 5] = float("inf")
    x[3, 129] = float("-inf")
    x[4, 0] = float("nan")
    x[5] = float("nan")
    x[6] = 0.0
    x[7] = 0.0
    x[7, 64] = fi.smallest_normal * (fi.eps)          # the smallest value of the type
    q, s = moe.i8_quantize(x)
    check_quantize(x, q, s, "extremes")
    assert torch.isnan(s[2:6]).all() and not bool(q[2:6].any())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_strides_alignment_and_live_rows(dtype):
    g = rng(11)
    big = torch.randn(50, 211, generator=g, device="cuda").to(dtype)
    for x in (big[:, 3:104], big[::2, :211], big[5:6, 1:200], big[:, 8:208]):
        q, s = moe.i8_quantize(x)
        check_quantize(x, q, s, f"view {tuple(x.shape)} {x.stride()}")
    live = torch.arange(50, device="cuda", dtype=torch.int32)
    live[::3] = -1
    q, s = moe.i8_row_buffers(50, 211)
    q.fill_(77)
    s.fill_(-5.0)
    moe.i8_quantize(big, live=live, out=(q, s))
    on = live >= 0
    assert bool((q[~on] == 77).all()) and bool((s[~on] == -5.0).all())
    check_quantize(big[on], q[on], s[on], "live rows")


# ---------------------------------------------------------------------------------------------
# weights
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("E,N,K,glu", [(1, 1, 1, False), (2, 37, 100, False), (3, 34, 130, True),
                                       (1, 64, 64, True), (2, 33, 64, False)])
def test_pack_is_the_documented_layout(E, N, K, glu):
    q, s, b, W = rand_stack(E + N + K, E, N, K, glu=glu)
    src = q.cpu().numpy()
    halves = [src[:, :N // 2], src[:, N // 2:]] if glu else [src]
    KP = (K + 63) // 64 * 64
    rows = []
    for h in halves:
        pad = np.zeros((E, (h.shape[1] + 15) // 16 * 16, KP), dtype=np.int8)
        pad[:, :h.shape[1], :K] = h
        rows.append(pad)
    full = np.concatenate(rows, axis=1)                                # [E][NT*16][KP]
    NT = full.shape[1] // 16
    want = full.reshape(E, NT, 16, KP // 64, 4, 16).transpose(0, 3, 1, 4, 2, 5)
    assert np.array_equal(W.q.cpu().numpy(), want.reshape(-1))


def test_quantized_stack_from_plain_weights():
    w = torch.randn(3, 20, 150, generator=rng(5), device="cuda").to(BF16)
    W = moe.I8Experts.quantized(w)
    rq, rs = ref_quantize(w.reshape(-1, 150))
    V = moe.I8Experts(rq.to(torch.int8).reshape(3, 20, 150), rs.reshape(3, 20))
    same_bits(W.q, V.q, "codes")
    same_bits(W.s, V.s, "scales")


# ---------------------------------------------------------------------------------------------
# dense
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 33, 64, 65, 127, 130, 257, 300])
@pytest.mark.parametrize("N,K", [(1, 1), (48, 64), (37, 100), (517, 1003), (260, 2880)])
def test_gemm_dense(rows, N, K):
    log(f"i8_gemm {rows}x{K} -> {N}")
    q, s, b, W = rand_stack(N + K, 1, N, K)
    x = rand_rows(rows + N, rows, K, BF16)
    aq, as_ = moe.i8_quantize(x)
    p, ref = ref_project(aq[:, :K], as_, q[0], s[0], b[0])
    for dt in (F32, BF16, F16):
        # f16 rows of large magnitude leave its range: to infinity, on both sides
        r = ref
        o = moe.i8_gemm(aq, as_, W, out_dtype=dt)
        if dt == F16:
            inside = ref.abs() < 65000
            assert torch.isinf(o[ref.abs() > 65600]).all()
            o, r, pp = torch.where(inside, o, 0), torch.where(inside, ref, 0), torch.where(inside, p, 0)
            assert_out(o, pp, r, f"{dt}")
        else:
            assert_out(o, p, r, f"{dt}")


@pytest.mark.parametrize("rows,N,K", [(5003, 5003, 129), (5003, 4999, 328), (4090, 4090, 65),
                                      (4090, 4085, 712), (1030, 2051, 200), (2, 60000, 70),
                                      (250, 5700, 64), (250, 5701, 130), (130, 8001, 1000)])
def test_gemm_dense_many_rows_and_channels(rows, N, K):
    """The tiles of large products (their sums are exact in f32 too: K 2^14 < 2^24)."""
    log(f"i8_gemm {rows}x{K} -> {N}")
    q, s, b, W = rand_stack(N + K, 1, N, K)
    aq, as_ = moe.i8_quantize(torch.randn(rows, K, generator=rng(rows), device="cuda").to(BF16))
    sums = aq[:, :K].float() @ q[0].float().t().contiguous()
    p = sums.double() * as_.double()[:, None] * s[0].double()
    out = moe.i8_gemm(aq, as_, W, out_dtype=F32)
    assert_out(out, p, p + b[0].double(), "f32")
    same_bits(moe.i8_gemm(aq, as_, W, out_dtype=BF16), out.to(BF16), "bf16")


def test_rows_and_outputs_behind_32_bits():
    """More rows than one launch takes, their codes past 4 GB; an output past 2^31 elements."""
    rows, N = (1 << 25) + 5, 9
    x = torch.randn(rows, 1, generator=rng(1), device="cuda").to(BF16)
    live = torch.ones(rows, dtype=torch.int32, device="cuda")
    live[-2] = -1
    aq, as_ = moe.i8_row_buffers(rows, 1)
    aq[-2], as_[-2] = 5, 0.5
    moe.i8_quantize(x, live=live, out=(aq, as_))
    assert int(aq[-2, 7]) == 5 and float(as_[-2]) == 0.5
    aq[-2], as_[-2] = 0, 0.0
    sign = torch.sign(x[:, 0].float())
    sign[-2] = 0.0
    assert torch.equal(aq[:, 0], (127 * sign).to(torch.int8)) and not bool(aq[-100:, 1:].any())
    top = torch.where(sign != 0, x[:, 0].float().abs(), 0.0)
    same_bits(as_, (top.double() / 127).float(), "scales")
    w = torch.arange(-4, 5, device="cuda", dtype=torch.int8)[:, None].contiguous()
    sc = torch.full((N,), 0.5, device="cuda")
    out = moe.i8_gemm(aq, as_, moe.I8Experts(w, sc))
    for i in range(N):
        want = (127 * (i - 4)) * sign.double() * (as_ * 0.5).double()
        same_bits(out[:, i].contiguous() + 0.0, want.float().to(BF16) + 0.0, f"channel {i}")
    del x, aq, as_, out, live, sign, top, want
    rows, N, K = 70001, 32771, 64
    q, s, b, W = rand_stack(1, 1, N, K)
    aq, as_ = moe.i8_quantize(torch.randn(rows, K, generator=rng(2), device="cuda").to(BF16))
    out = moe.i8_gemm(aq, as_, W)
    tail = moe.i8_gemm(aq[-3:, :].contiguous(), as_[-3:].contiguous(), W)
    same_bits(out[-3:], tail, "last rows")
    same_bits(out[:3], moe.i8_gemm(aq[:3].contiguous(), as_[:3].contiguous(), W), "first rows")


def test_experts_behind_4_gb_and_the_longest_sums():
    E, N, K, tokens = 3, 24000, 65536, 5
    g = rng(4)
    q = torch.randint(-128, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand(E, N, generator=g, device="cuda") * 1e-4
    W = moe.I8Experts(q, s)
    aq, as_ = moe.i8_quantize(torch.randn(tokens, K, generator=g, device="cuda").to(BF16))
    cnt, basep, row_tok, mpad = csr([2, 0, 4], 1, 1, tokens)
    out = moe.i8_moe_gemm(aq, as_, row_tok, W, cnt, basep, 1, mpad)
    for e, span in ((0, slice(0, 2)), (2, slice(2, 6))):
        t = row_tok[span].long()
        for n0 in (0, 11008, N - 992):
            n = slice(n0, n0 + 992)
            p, ref = ref_project(aq[t, :K], as_[t], q[e, n], s[e, n], None)
            assert_out(out[span, n], p, ref, f"expert {e} channels {n0}..")


@pytest.mark.parametrize("rows,N,K", [(1, 517, 1003), (3, 64, 64), (16, 100, 200), (17, 100, 200),
                                      (70, 300, 520), (300, 130, 2880), (256, 4099, 129), (4, 40, 4095),
                                      (2, 40, 4097), (3, 50, 5), (4, 33, 15001), (5, 33, 15001),
                                      (8, 40, 3000), (8, 40, 3100), (7, 70, 2001), (5, 33, 4097),
                                      (6, 33, 4095), (9, 40, 64), (1, 20, 24576), (1, 20, 24577)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_linear_is_quantize_then_gemm(rows, N, K, dtype):
    q, s, b, W = rand_stack(N + K, 1, N, K, bias=rows != 16)
    x = torch.randn(rows, K, generator=rng(rows), device="cuda").to(dtype)
    aq, as_ = moe.i8_quantize(x)
    for odt in (BF16, F16, F32):
        want = moe.i8_gemm(aq, as_, W, out_dtype=odt)
        same_bits(moe.i8_linear(x, W, out_dtype=odt), want, f"{odt}")
    assert moe.i8_linear(x, W).dtype == dtype
    p, ref = ref_project(*[t.to("cuda") for t in ref_quantize(x)], q[0], s[0],
                         None if b is None else b[0])
    assert_out(moe.i8_linear(x, W, out_dtype=F32), p, ref, "linear")


@pytest.mark.parametrize("rows", [1, 16, 40, 300])
def test_linear_strided_rows_in_and_out(rows):
    N, K = 100, 333
    q, s, b, W = rand_stack(1, 1, N, K)
    x = torch.randn(rows, K + 31, generator=rng(9), device="cuda").to(BF16)
    big = torch.full((rows, N + 7), 55.0, device="cuda", dtype=BF16)
    out = moe.i8_linear(x[:, 5:5 + K], W, out=big[:, 2:2 + N])
    same_bits(out, moe.i8_linear(x[:, 5:5 + K].contiguous(), W), "strided")
    assert bool((big[:, :2] == 55).all()) and bool((big[:, 2 + N:] == 55).all())


@pytest.mark.parametrize("rows", [5, 40, 300])
def test_linear_rows_without_a_value_stay_alone(rows):
    N, K = 70, 190
    q, s, b, W = rand_stack(2, 1, N, K)
    x = torch.randn(rows, K, generator=rng(4), device="cuda").to(BF16)
    clean = moe.i8_linear(x, W)
    y = x.clone()
    y[1, 7] = float("nan")
    y[3] = float("-inf")
    out = moe.i8_linear(y, W)
    keep = [r for r in range(rows) if r not in (1, 3)]
    assert torch.isnan(out[[1, 3]]).all()
    same_bits(out[keep], clean[keep], "other rows")


def test_gemm_largest_sums_are_exact():
    """Every product of the largest size and one sign, at the longest K: the 32-bit sums hold."""
    K, N = moe.MOE_I8_MAX_K, 20
    q = torch.full((1, N, K), -128, dtype=torch.int8, device="cuda")
    q[0, 1] = 127
    W = moe.I8Experts(q, torch.ones(1, N, device="cuda"))
    x = torch.ones(3, K, device="cuda")
    x[1] = -1.0
    aq, as_ = moe.i8_quantize(x)
    as_.fill_(1.0)
    out = moe.i8_gemm(aq, as_, W, out_dtype=F32)
    want = aq.double() @ q[0].double().t().contiguous()
    assert torch.equal(out.double(), want)


def test_glu_stack_in_a_dense_product_keeps_channel_order():
    q, s, b, _ = rand_stack(6, 1, 2 * 21, 77)
    x = torch.randn(9, 77, generator=rng(6), device="cuda").to(BF16)
    same_bits(moe.i8_linear(x, moe.I8Experts(q, s, b, glu=True)), moe.i8_linear(x, moe.I8Experts(q, s, b)), "glu")


# ---------------------------------------------------------------------------------------------
# routed
# ---------------------------------------------------------------------------------------------

def csr(counts, tile_m, seed, tokens):
    """A CSR with the given rows per expert, tokens drawn per expert without repetition."""
    g = np.random.default_rng(seed)
    basep, row_tok = [0], []
    for c in counts:
        tok = np.sort(g.choice(tokens, c, replace=False))
        pad = -c % tile_m
        row_tok += tok.tolist() + [-1] * pad
        basep.append(basep[-1] + c + pad)
    row_tok += [-1] * 21                                   # ghost rows
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    return dev(counts), dev(basep), dev(row_tok), len(row_tok)


ROUTED = {
    "few": ([0, 3, 1, 0, 5, 16, 17], 1), "tiles": ([15, 16, 17, 0, 64, 63, 65, 1], 16),
    "one": ([0, 0, 300, 0], 7), "tall": ([135, 136, 257, 2], 32), "empty": ([0, 0, 0], 16),
    "many": ([(7 * i) % 5 for i in range(80)], 4), "ends": ([130] + [0] * 40 + [40], 1),
}


@pytest.mark.parametrize("name", list(ROUTED))
@pytest.mark.parametrize("F,D", [(24, 100), (176, 520), (161, 64), (700, 131), (1500, 65),
                                 (2049, 328)])
def test_moe_gemm(name, F, D):
    counts, tile_m = ROUTED[name]
    log(f"i8_moe_gemm {name} F={F} D={D}")
    E, tokens = len(counts), 320
    cnt, basep, row_tok, mpad = csr(counts, tile_m, 1, tokens)
    x = torch.randn(tokens, D, generator=rng(2), device="cuda").to(BF16)
    aq, as_ = moe.i8_quantize(x)
    q, s, b, W = rand_stack(E + F, E, 2 * F, D, glu=True)
    b *= 3.0
    live = torch.zeros(mpad, dtype=torch.bool, device="cuda")
    ref = torch.zeros(mpad, 2 * F, dtype=torch.float64, device="cuda")
    p = torch.zeros_like(ref)
    for e, c in enumerate(counts):
        span = slice(int(basep[e]), int(basep[e]) + c)
        live[span] = True
        t = row_tok[span].long()
        p[span], ref[span] = ref_project(aq[t, :D], as_[t], q[e], s[e], b[e])
    # plain
    out = torch.full((mpad, 2 * F), -77.0, device="cuda")
    moe.i8_moe_gemm(aq, as_, row_tok, W, cnt, basep, tile_m, mpad, NONE, ALPHA, LIMIT, out=out)
    assert bool((out[~live] == -77.0).all()), "rows that are not live were written"
    assert_out(out[live], p[live], ref[live], "plain")
    # SwiGLU: the activation of the fp32 pair, its own f32 evaluation (a few units) and the rounding
    h = torch.full((mpad, F), -77.0, device="cuda", dtype=BF16)
    moe.i8_moe_gemm(aq, as_, row_tok, W, cnt, basep, tile_m, mpad, SWIGLU, ALPHA, LIMIT, out=h)
    assert bool((h[~live] == -77.0).all()), "rows that are not live were written"
    g64 = out.double()
    gate, up = g64[:, :F].clamp(max=LIMIT), g64[:, F:].clamp(-LIMIT, LIMIT)
    want = gate * torch.sigmoid(ALPHA * gate) * (up + 1.0)
    # z = alpha g is rounded, and so its multiple of log2 e: the sigmoid is off by |z| 2^-22 at most
    tol = want.abs() * (2.0 ** -8 + (8 + (ALPHA * gate).abs() * 2) * 2.0 ** -23) + \
        gate.abs() * 2.0 ** -23 + TINY[BF16]
    bad = live[:, None] & ~((h.double() - want).abs() <= tol)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} SwiGLU values outside"
    # the same rows in CSR order, without indices
    rows = row_tok.long().clamp(min=0)
    same_bits(moe.i8_moe_gemm(aq[rows].contiguous(), as_[rows].contiguous(), None, W, cnt, basep,
                              tile_m, mpad, NONE)[live], out[live], "without a_row")


def test_moe_gemm_row_indices_out_of_range_are_left_unwritten():
    E, D, N, tokens = 3, 96, 40, 50
    cnt, basep, row_tok, mpad = csr([20, 0, 70 % 50], 8, 3, tokens)
    q, s, b, W = rand_stack(1, E, N, D)
    aq, as_ = moe.i8_quantize(torch.randn(tokens, D, generator=rng(1), device="cuda").to(BF16))
    clean = moe.i8_moe_gemm(aq, as_, row_tok, W, cnt, basep, 8, mpad,
                            out=torch.full((mpad, N), -7.0, device="cuda"))
    bad = row_tok.clone()
    bad[2], bad[5] = tokens, -4
    out = moe.i8_moe_gemm(aq, as_, bad, W, cnt, basep, 8, mpad,
                          out=torch.full((mpad, N), -7.0, device="cuda"))
    assert bool((out[[2, 5]] == -7.0).all())
    keep = [r for r in range(mpad) if r not in (2, 5)]
    same_bits(out[keep], clean[keep], "other rows")


# ---------------------------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------------------------

def layer(seed, T, E, k, D, F, popular=0.0):
    g = rng(seed)
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[:, 0] += popular
    x = torch.randn(T, D, generator=g, device="cuda").to(BF16)
    GU = rand_stack(seed + 1, E, 2 * F, D, glu=True)
    DN = rand_stack(seed + 2, E, D, F)
    return logits, x, GU, DN


DECODE = {
    "one": (1, 8, 4, 200, 144), "top1": (3, 4, 1, 64, 64), "all": (2, 4, 4, 100, 33),
    "popular": (16, 32, 4, 130, 70), "most": (16, 16, 8, 96, 80), "wide": (5, 1024, 8, 65, 17),
    "single": (4, 1, 1, 70, 50), "e65": (7, 65, 3, 333, 95), "large": (2, 8, 2, 2880, 2880),
    "long": (16, 6, 2, 8000, 40), "deep": (3, 5, 2, 40, 9000),
    "odd1": (1, 27, 4, 1737, 179), "odd3": (3, 30, 5, 619, 946), "odd13": (13, 37, 8, 261, 110),
    "tiny": (1, 3, 2, 3, 5), "one_wide": (1, 200, 8, 97, 4095),
}


@pytest.mark.parametrize("name", list(DECODE))
def test_decode_is_the_chain_bit_for_bit(name):
    T, E, k, D, F = DECODE[name]
    log(f"i8_moe_decode {name} T={T} E={E} k={k} D={D} F={F}")
    logits, x, GU, DN = layer(len(name) + T, T, E, k, D, F, 3.0 if name == "popular" else 0.0)
    o = moe.i8_moe_decode(logits, x, GU[3], DN[3], k, ALPHA, LIMIT, want_d=True)
    c = moe.moe_layer(x, logits, GU[3], DN[3], k, 1, ALPHA, LIMIT, projection="i8")
    at = c["pos"].long().reshape(-1)
    assert torch.equal(o["ids"], c["ids"])
    same_bits(o["w"], c["w"], "w")
    same_bits(o["h"], c["h"][at], "h")
    same_bits(o["d"], c["d"][at], "d")
    same_bits(o["y"], c["y"], "y")
    # without d, and y in 16 bits: the same sum, rounded once
    o2 = moe.i8_moe_decode(logits, x, GU[3], DN[3], k, ALPHA, LIMIT, y_dtype=BF16)
    same_bits(o2["y"], o["y"].to(BF16), "bf16 y")
    assert "d" not in o2


@pytest.mark.parametrize("T", [1, 6, 16])
@pytest.mark.parametrize("E", [7, 64, 65, 128, 129, 300])
def test_decode_routes_ties_and_odd_logits_as_the_router(T, E):
    """Equal logits, zeros of both signs, infinities and NaN: fewer numbers than picks among them.
    The experts that are computed are those that are written."""
    k, D, F = 6, 64, 32
    g = rng(E + T)
    logits = torch.randint(-2, 3, (T, E), generator=g, device="cuda").float()
    logits[logits == 0] *= -1.0
    odd = torch.tensor([float("nan"), float("inf"), float("-inf"), 0.0, -0.0, float("nan")],
                       device="cuda")
    logits[:, :6] = odd
    logits[0, 3:] = float("nan")
    if T > 2:
        logits[1] = float("-inf")
        logits[2] = float("nan")
    x = torch.randn(T, D, generator=g, device="cuda").to(BF16)
    GU, DN = rand_stack(1, E, 2 * F, D, glu=True), rand_stack(2, E, D, F)
    o = moe.i8_moe_decode(logits, x, GU[3], DN[3], k)
    ids, _ = moe.moe_route_topk(logits, k)
    assert torch.equal(o["ids"], ids)
    aq, as_ = moe.i8_quantize(x)
    for t in range(T):
        for r in range(k):
            e = int(ids[t, r])
            one = moe.I8Experts(GU[0][e], GU[1][e].contiguous(), GU[2][e].contiguous(), glu=True)
            want = moe.i8_moe_gemm(aq[t:t + 1].contiguous(), as_[t:t + 1].contiguous(), None, one,
                                   torch.ones(1, dtype=torch.int32, device="cuda"),
                                   torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1, 1,
                                   SWIGLU, ALPHA, LIMIT)
            same_bits(o["h"][t * k + r], want[0], f"token {t} slot {r} expert {e}")


@pytest.mark.parametrize("T,E,k,D,F,tile_m", [(1, 4, 2, 64, 64, 1), (9, 8, 3, 100, 70, 4),
                                             (200, 6, 2, 130, 90, 16), (600, 3, 2, 96, 48, 16)])
def test_layer_against_the_definition(T, E, k, D, F, tile_m):
    logits, x, (gq, gs, gb, GU), (dq, ds, db, DN) = layer(T, T, E, k, D, F)
    c = moe.moe_layer(x, logits, GU, DN, k, tile_m, ALPHA, LIMIT, projection="i8")
    ids, w = oracle.route_topk(logits.cpu().numpy(), k)
    assert np.array_equal(c["ids"].cpu().numpy(), ids)
    at = c["pos"].long()
    xq, xs = ref_quantize(x)
    hq, hs = ref_quantize(c["h"][at.reshape(-1)])
    for t in range(0, T, max(1, T // 40)):
        y = torch.zeros(D, dtype=torch.float64, device="cuda")
        size = torch.zeros(D, dtype=torch.float64, device="cuda")
        for slot in range(k):
            e = int(ids[t, slot])
            _, g = ref_project(xq[t:t + 1], xs[t:t + 1], gq[e], gs[e], gb[e])
            gate, up = g[:, :F].clamp(max=LIMIT), g[:, F:].clamp(-LIMIT, LIMIT)
            want = (gate * torch.sigmoid(ALPHA * gate) * (up + 1.0))[0]
            h = c["h"][at[t, slot]].double()
            # fp32 gate and up (2^-22 of their sizes carries, slopes below 9), then bf16
            tol = want.abs() * 2.0 ** -8 * (1 + 2.0 ** -8) + 16 * 2.0 ** -22 * (g.abs().max() + 4)
            assert bool(((h - want).abs() <= tol).all()), f"h of token {t} slot {slot}"
            r = t * k + slot
            p, d = ref_project(hq[r:r + 1], hs[r:r + 1], dq[e], ds[e], db[e])
            y += float(w[t, slot]) * d[0]
            size += float(w[t, slot]) * (2 * p[0].abs() + d[0].abs())
        assert bool(((c["y"][t].double() - y).abs() <= (k + 3) * 2.0 ** -23 * size).all()), t


def test_layer_with_a_token_without_values():
    T, E, k, D, F = 6, 5, 2, 80, 48
    logits, x, GU, DN = layer(1, T, E, k, D, F)
    clean = moe.i8_moe_decode(logits, x, GU[3], DN[3], k)
    bad = x.clone()
    bad[2, 3] = float("nan")
    out = moe.i8_moe_decode(logits, bad, GU[3], DN[3], k)
    assert torch.isnan(out["y"][2]).all()
    keep = [0, 1, 3, 4, 5]
    same_bits(out["y"][keep], clean["y"][keep], "other tokens")
    lg = logits.clone()
    lg[4] = float("nan")                     # routes to valid experts, weights without a value
    out = moe.i8_moe_decode(lg, x, GU[3], DN[3], k)
    assert torch.isnan(out["y"][4]).all()
    keep = [0, 1, 2, 3, 5]
    same_bits(out["y"][keep], clean["y"][keep], "other tokens")


# ---------------------------------------------------------------------------------------------
# streams, graphs, repetition
# ---------------------------------------------------------------------------------------------

def test_on_another_stream():
    logits, x, GU, DN = layer(8, 3, 8, 2, 200, 96)
    want = moe.i8_moe_decode(logits, x, GU[3], DN[3], 2)["y"]
    lin = moe.i8_linear(x, DN_dense(DN))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = moe.i8_moe_decode(logits, x, GU[3], DN[3], 2, stream=side)["y"]
    with torch.cuda.stream(side):
        got2 = moe.i8_linear(x, DN_dense(DN))
    torch.cuda.synchronize()
    same_bits(got, want, "decode")
    same_bits(got2, lin, "linear")


def busy(stream):
    """Some milliseconds of work on the stream."""
    with torch.cuda.stream(stream):
        a = torch.randn(4096, 4096, device="cuda")
        for _ in range(8):
            a = a @ a * 1e-3
    return a


def test_stream_argument_covers_everything_a_call_does():
    """What a call allocates, copies or packs on the way stays behind the work of its stream, not of
    the current one: scratch is not handed out again while the stream still needs it."""
    K, N, rows = 520, 96, 40
    wts = torch.randn(N, K, generator=rng(1), device="cuda").to(BF16)
    x = torch.randn(rows, K, generator=rng(2), device="cuda").to(BF16)
    W = moe.I8Experts.quantized(wts)
    want = moe.i8_linear(x, W)
    aq, as_ = moe.i8_quantize(x)
    logits, xt, GU, DN = layer(3, 9, 8, 2, 200, 96)
    want_y = moe.i8_moe_decode(logits, xt, GU[3], DN[3], 2)["y"]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    keep = [busy(side)]
    W2 = moe.I8Experts.quantized(wts, stream=side)
    got = moe.i8_linear(x, W2, stream=side)
    aq2, as2 = moe.i8_quantize(x, stream=side)
    got_gemm = moe.i8_gemm(aq2, as2, W2, stream=side)
    y = moe.i8_moe_decode(logits, xt, GU[3], DN[3], 2, stream=side)["y"]
    for n in (rows * moe.i8_pitch(K), N * K, N * moe.i8_pitch(K), 18 * 128):   # the sizes let go
        keep += [torch.full((n,), 85, dtype=torch.int8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    same_bits(W2.q, W.q, "packed")
    same_bits(aq2, aq, "quantized")
    same_bits(got, want, "linear")
    same_bits(got_gemm, want, "gemm")
    same_bits(y, want_y, "decode")
    assert all(bool((t == 85).all()) for t in keep[1:])


def test_two_streams_at_once():
    """Two calls of every entry point in flight together, each with scratch of its own."""
    sets = []
    for i in range(2):
        logits, x, GU, DN = layer(20 + i, 16, 8, 4, 520, 176)
        sets.append((logits, x, GU[3], DN[3], torch.cuda.Stream()))
    want = [(moe.moe_layer(x, lo, gu, dn, 4, 8, projection="i8")["y"],
             moe.i8_moe_decode(lo, x, gu, dn, 4)["y"]) for lo, x, gu, dn, _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for lo, x, gu, dn, st in sets:
            with torch.cuda.stream(st):
                got.append((moe.moe_layer(x, lo, gu, dn, 4, 8, projection="i8")["y"],
                            moe.i8_moe_decode(lo, x, gu, dn, 4)["y"]))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            same_bits(a[0], b[0], "layer")
            same_bits(a[1], b[1], "decode")


def DN_dense(DN):
    q, s, b, _ = DN
    return moe.I8Experts(q[0].t().contiguous().repeat(1, 3)[:, :q.shape[1]].contiguous(),
                         s[0][:q.shape[2]].contiguous())


def test_captured_and_replayed():
    T, E, k, D, F = 4, 8, 2, 300, 110
    logits, x, GU, DN = layer(12, T, E, k, D, F)
    q, s, b, W = rand_stack(1, 1, 150, D)
    many = torch.randn(300, D, generator=rng(1), device="cuda").to(BF16)
    ws = moe.i8_row_buffers(300, D)
    out = torch.empty(300, 150, device="cuda", dtype=BF16)
    o = {"ids": torch.empty(T, k, dtype=torch.int32, device="cuda"),
         "w": torch.empty(T, k, device="cuda"),
         "h": torch.empty(T * k, F, dtype=BF16, device="cuda"),
         "y": torch.empty(T, D, device="cuda")}

    def both():
        moe.i8_moe_decode(logits, x, GU[3], DN[3], k, out=o)
        moe.i8_linear(many, W, out=out, ws=ws)
        return moe.moe_layer(x, logits, GU[3], DN[3], k, 16, projection="i8")["y"]

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y_layer = both()
    for i in range(4):
        logits.copy_(torch.randn(T, E, generator=rng(100 + i), device="cuda"))
        x.copy_(torch.randn(T, D, generator=rng(200 + i), device="cuda"))
        many.copy_(torch.randn(300, D, generator=rng(300 + i), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = {key: t.clone() for key, t in o.items()}
        got_out, got_layer = out.clone(), y_layer.clone()
        want = moe.i8_moe_decode(logits, x, GU[3], DN[3], k)
        for key in got:
            same_bits(got[key], want[key], f"replay {i}: {key}")
        same_bits(got_out, moe.i8_linear(many, W), f"replay {i}: linear")
        same_bits(got_layer, want["y"], f"replay {i}: layer")


def test_refusals_before_any_launch():
    q, s, b, W = rand_stack(1, 1, 32, 64)
    x = torch.randn(4, 64, device="cuda").to(BF16)
    with pytest.raises(TypeError):
        moe.i8_quantize(x.double())
    with pytest.raises(ValueError):
        moe.i8_quantize(x.t())
    with pytest.raises(moe.MoeError):
        moe.i8_quantize(x[:0])
    with pytest.raises(ValueError):
        moe.i8_linear(x[:, :63], W)
    with pytest.raises(ValueError):
        moe.i8_linear(x, W, out=torch.empty(4, 31, device="cuda", dtype=BF16))
    with pytest.raises(TypeError):
        moe.i8_linear(x, W, out=torch.empty(4, 32, device="cuda"), out_dtype=BF16)
    with pytest.raises(ValueError):
        moe.i8_linear(x, W, ws=moe.i8_row_buffers(3, 64))
    with pytest.raises(ValueError):
        moe.I8Experts(q, s[:, :31].contiguous())
    with pytest.raises(moe.MoeError):
        moe.I8Experts(q[:, :31].contiguous(), s[:, :31].contiguous(), glu=True)
    with pytest.raises(TypeError):
        moe.I8Experts(q.to(torch.uint8), s)
    aq, as_ = moe.i8_quantize(x)
    with pytest.raises(ValueError):
        moe.i8_gemm(aq[:, :32].contiguous(), as_, W)
    with pytest.raises(ValueError):
        moe.i8_moe_decode(torch.randn(3, 4, device="cuda"), x, W, W, 1)


@pytest.mark.parametrize("rows", [2, 40])
def test_outputs_are_rounded_over_the_whole_range(rows):
    """A one-channel-per-value projection whose outputs cover every bf16 exponent, subnormals, ties
    and both signs among them: the stored value is torch's rounding of the fp32 one."""
    N, K = 2048, 64
    q = torch.zeros(1, N, K, dtype=torch.int8, device="cuda")
    q[0, :, 0] = 1
    g = rng(3)
    s = torch.exp2(torch.randint(-140, 120, (1, N), generator=g, device="cuda").double()) * \
        (1 + torch.randint(0, 512, (1, N), generator=g, device="cuda").double() / 512)
    W = moe.I8Experts(q, s.float())
    x = torch.zeros(rows, K, device="cuda")
    x[:, 0] = 127.0                                     # code 127, scale 1
    x[1] = -x[1]
    full = moe.i8_linear(x, W, out_dtype=F32)
    assert torch.equal(full[0], (s[0] * 127.0).float())
    assert torch.equal(moe.i8_linear(x, W, out_dtype=BF16), full.to(BF16))
    half = moe.i8_linear(x, W, out_dtype=F16)
    assert torch.equal(half, full.to(F16))
