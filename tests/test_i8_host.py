"""The 8-bit integer entry points on the host (no GPU): sizes, argument checks of the C ABI and of
the binding. Fake (never dereferenced) device addresses, so only where no GPU is visible."""
import ctypes

import pytest
import torch

from mxfp4_mixture_experts_route_amd import _lib

no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="host-only validation tests use fake device addresses")
FAKE = ctypes.c_void_p(0x1000)
OFF = {n: ctypes.c_void_p(0x1000 + n) for n in (1, 2, 4, 8)}
EINVAL, ESHAPE, EALIGN = _lib.MOE_EINVAL, _lib.MOE_ESHAPE, _lib.MOE_EALIGN
BF16, F32 = _lib.MOE_BF16, _lib.MOE_F32


def stack(q=0x1000, s=0x2000, bias=None, E=1, N=48, K=100, glu=0):
    return _lib.I8ExpertsC(q, s, bias, E, N, K, glu)


def ref(w):
    return None if w is None else ctypes.byref(w)


@pytest.mark.parametrize("E,N,K,glu,tiles,chunks", [
    (1, 1, 1, 0, 1, 1), (1, 16, 64, 0, 1, 1), (3, 17, 65, 0, 2, 2), (2, 34, 100, 1, 4, 2),
    (2, 32, 64, 1, 2, 1), (32, 5760, 2880, 1, 360, 45), (1, 48, 65536, 0, 3, 1024)])
def test_packed_bytes(E, N, K, glu, tiles, chunks):
    assert _lib.lib().i8_packed_bytes(E, N, K, glu) == E * tiles * chunks * 1024


def test_packed_bytes_refuses():
    f = _lib.lib().i8_packed_bytes
    for args in [(0, 16, 64, 0), (1, 0, 64, 0), (1, 16, 0, 0), (1, 15, 64, 1),
                 (1, 16, _lib.MOE_I8_MAX_K + 1, 0)]:
        assert f(*args) == -1


def test_pitch():
    assert [_lib.i8_pitch(k) for k in (1, 127, 128, 129, 2880, 1003)] == [128, 128, 128, 256, 2944, 1024]


@no_gpu
def test_pack_argument_checks():
    f = _lib.lib().i8_pack_experts
    assert f(None, 1, 16, 64, 0, FAKE, None) == EINVAL
    assert f(FAKE, 1, 16, 64, 0, None, None) == EINVAL
    assert f(FAKE, 0, 16, 64, 0, FAKE, None) == EINVAL
    assert f(FAKE, _lib.MOE_MAX_E + 1, 16, 64, 0, FAKE, None) == ESHAPE
    assert f(FAKE, 1, 15, 64, 1, FAKE, None) == ESHAPE
    assert f(FAKE, 1, 16, 65537, 0, FAKE, None) == ESHAPE
    assert f(FAKE, 1, 16, 64, 0, OFF[8], None) == EALIGN


@no_gpu
def test_quantize_argument_checks():
    f = _lib.lib().i8_quantize

    def call(x=FAKE, dt=BF16, ld=100, rows=4, K=100, q=FAKE, s=FAKE):
        return f(x, dt, ld, None, rows, K, q, s, None)

    assert call(x=None) == EINVAL
    assert call(q=None) == EINVAL
    assert call(s=None) == EINVAL
    assert call(rows=0) == EINVAL
    assert call(K=0) == EINVAL
    assert call(dt=3) == EINVAL
    assert call(dt=-1) == EINVAL
    assert call(ld=99) == ESHAPE
    assert call(K=65537, ld=65537) == ESHAPE
    assert call(rows=1 << 31) == ESHAPE
    assert call(q=OFF[8]) == EALIGN
    assert call(s=OFF[2]) == EALIGN
    assert call(x=OFF[1]) == EALIGN
    assert call(x=OFF[2], dt=F32) == EALIGN
    assert f(FAKE, BF16, 100, OFF[2], 4, 100, FAKE, FAKE, None) == EALIGN


@no_gpu
def test_gemm_argument_checks():
    f = _lib.lib().i8_gemm

    def call(aq=FAKE, as_=FAKE, rows=3, w=stack(), out=FAKE, dt=BF16, ld=48):
        return f(aq, as_, rows, ref(w), out, dt, ld, None)

    assert call(aq=None) == EINVAL
    assert call(as_=None) == EINVAL
    assert call(w=None) == EINVAL
    assert call(w=stack(q=None)) == EINVAL
    assert call(w=stack(s=None)) == EINVAL
    assert call(w=stack(K=0)) == EINVAL
    assert call(w=stack(glu=2)) == EINVAL
    assert call(out=None) == EINVAL
    assert call(rows=0) == EINVAL
    assert call(dt=7) == EINVAL
    assert call(w=stack(E=2)) == ESHAPE
    assert call(w=stack(N=47, glu=1)) == ESHAPE
    assert call(w=stack(K=65537)) == ESHAPE
    assert call(w=stack(N=1 << 20, K=1 << 12), ld=1 << 20) == ESHAPE   # 4 GB of one matrix
    assert call(ld=47) == ESHAPE
    assert call(aq=OFF[8]) == EALIGN
    assert call(w=stack(q=0x1008)) == EALIGN
    assert call(w=stack(s=0x2002)) == EALIGN
    assert call(w=stack(bias=0x2002)) == EALIGN
    assert call(out=OFF[1]) == EALIGN
    assert call(out=OFF[2], dt=F32) == EALIGN


@no_gpu
def test_linear_argument_checks():
    f = _lib.lib().i8_linear

    def call(x=FAKE, dt=BF16, ld=100, rows=3, w=stack(), q=FAKE, s=FAKE, out=FAKE, odt=BF16,
             ldo=48):
        return f(x, dt, ld, rows, ref(w), q, s, out, odt, ldo, None)

    assert call(x=None) == EINVAL
    assert call(q=None) == EINVAL
    assert call(s=None) == EINVAL
    assert call(out=None) == EINVAL
    assert call(w=None) == EINVAL
    assert call(rows=0) == EINVAL
    assert call(dt=5) == EINVAL
    assert call(odt=5) == EINVAL
    assert call(ld=99) == ESHAPE
    assert call(ldo=47) == ESHAPE
    assert call(w=stack(E=2)) == ESHAPE
    assert call(x=OFF[1]) == EALIGN
    assert call(q=OFF[4]) == EALIGN
    assert call(s=OFF[1]) == EALIGN
    assert call(out=OFF[1]) == EALIGN


@no_gpu
def test_moe_gemm_argument_checks():
    f = _lib.lib().i8_moe_gemm
    NONE, SW = _lib.MOE_ACT_NONE, _lib.MOE_ACT_SWIGLU_OAI

    def call(aq=FAKE, as_=FAKE, a_row=FAKE, a_rows=8, w=stack(E=4), counts=FAKE, basep=FAKE,
             tile_m=16, mpad=64, act=NONE, out=FAKE):
        return f(aq, as_, a_row, a_rows, ref(w), counts, basep, tile_m, mpad, act, 1.702, 7.0,
                 out, None)

    assert call(aq=None) == EINVAL
    assert call(as_=None) == EINVAL
    assert call(w=None) == EINVAL
    assert call(counts=None) == EINVAL
    assert call(basep=None) == EINVAL
    assert call(out=None) == EINVAL
    assert call(a_rows=0) == EINVAL
    assert call(mpad=0) == EINVAL
    assert call(act=_lib.MOE_ACT_SWIGLU_OAI_MX8) == EINVAL
    assert call(act=SW) == ESHAPE                                  # not packed for SwiGLU
    assert call(tile_m=0) == ESHAPE
    assert call(tile_m=257) == ESHAPE
    assert call(w=stack(E=1025)) == ESHAPE
    assert call(a_row=None) == ESHAPE                              # fewer rows than the CSR
    assert call(mpad=1 << 31) == ESHAPE
    assert call(a_rows=1 << 25) == ESHAPE                          # 4 GB of rows of 128 bytes
    assert call(aq=OFF[4]) == EALIGN
    assert call(as_=OFF[2]) == EALIGN
    assert call(out=OFF[2]) == EALIGN
    assert call(out=OFF[1], act=SW, w=stack(E=4, glu=1)) == EALIGN
    for name in ("a_row", "counts", "basep"):
        assert call(**{name: OFF[2]}) == EALIGN, name


@no_gpu
def test_decode_argument_checks():
    f = _lib.lib().i8_moe_decode
    gu, dn = stack(E=4, N=96, K=100, glu=1), stack(E=4, N=100, K=48)

    def call(logits=FAKE, x=FAKE, T=2, E=4, k=2, gu=gu, dn=dn, ids=FAKE, w=FAKE, h=FAKE, q=FAKE,
             s=FAKE, d=None, y=FAKE, dt=F32):
        return f(logits, x, T, E, k, ref(gu), ref(dn), 1.702, 7.0, ids, w, h, q, s, d, y, dt, None)

    for name in ("logits", "x", "gu", "dn", "ids", "w", "h", "y"):
        assert call(**{name: None}) == EINVAL, name
    assert call(T=0) == EINVAL
    assert call(k=0) == EINVAL
    assert call(k=5) == EINVAL
    assert call(dt=4) == EINVAL
    assert call(T=17) == ESHAPE
    assert call(E=16, k=9, gu=stack(E=16, N=96, glu=1), dn=stack(E=16, N=100, K=48)) == ESHAPE
    assert call(gu=stack(E=4, N=96, K=100)) == ESHAPE              # gate_up not packed for SwiGLU
    assert call(dn=stack(E=4, N=100, K=48, glu=1)) == ESHAPE
    assert call(dn=stack(E=3, N=100, K=48)) == ESHAPE
    assert call(dn=stack(E=4, N=99, K=48)) == ESHAPE
    assert call(dn=stack(E=4, N=100, K=47)) == ESHAPE
    assert call(T=16, gu=stack(E=4, N=96, K=10000, glu=1), dn=stack(E=4, N=10000, K=48)) == ESHAPE
    assert call(T=9, q=None) == EINVAL                             # 18 rows of h need scratch
    assert call(T=9, s=None) == EINVAL
    assert call(T=9, q=OFF[8]) == EALIGN
    assert call(T=9, s=OFF[2]) == EALIGN
    assert call(x=OFF[8]) == EALIGN
    assert call(h=OFF[8]) == EALIGN
    assert call(logits=OFF[2]) == EALIGN
    assert call(d=OFF[2]) == EALIGN
    assert call(y=OFF[2]) == EALIGN
    assert call(y=OFF[1], dt=BF16) == EALIGN
    for name in ("ids", "w"):
        assert call(**{name: OFF[2]}) == EALIGN, name
    assert call(gu=stack(bias=0x3002, E=4, N=96, K=100, glu=1)) == EALIGN
    assert call(dn=stack(bias=0x3002, E=4, N=100, K=48)) == EALIGN


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        _lib.i8_quantize(x)                                        # not on the device
    with pytest.raises(TypeError):
        _lib.I8Experts(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(TypeError):
        _lib._i8_dtype(torch.float64, "x")
    with pytest.raises(TypeError):
        _lib.moe_layer(x, torch.zeros(2, 4), None, None, 1, 1, projection="i8")
    with pytest.raises(ValueError):
        _lib.moe_layer(x, torch.zeros(2, 4), None, None, 1, 1, projection="i4")
    w = object.__new__(_lib.I8Experts)
    for projection, stacks in (("i8", (w, None)), ("i8", (None, w)), ("gemm", (w, None)),
                               ("gemv", (None, w)), ("gemm_mx8", (w, w))):
        with pytest.raises(TypeError):
            _lib.moe_layer(x, torch.zeros(2, 4), *stacks, 1, 1, projection=projection)
