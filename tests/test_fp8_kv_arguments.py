"""Host-side argument checks of the 8-bit layer and the cache, at made-up addresses that lie apart:
a call that passes every check ends with GPTQ_ERR_CUDA where there is no device, so a refusal
below comes from the one argument that is wrong. Skipped where a device could run such a call."""

import pytest
import torch

if torch.cuda.is_available():
    pytest.skip("made-up addresses are used without a device only", allow_module_level=True)

ERR_ARG, ERR_CUDA = -1, -4
MB = 1 << 20
A, B, C, D, E, F = ((i + 1) * MB for i in range(6))


@pytest.fixture(scope="module")
def L():
    from post_weight_quantization_24_b200 import build, gptq
    build.build()
    return gptq.lib()


def _linear(L, X=A, sx=B, n=4, d=128, W=C, sw=D, o=40, R=None, Y=E, dt=0, st=None):
    return L.fp8_linear(X, sx, n, d, W, sw, o, R, Y, dt, st, None)


def _write(L, K=A, V=B, dt=0, n=4, ks=256, vs=256, H=2, D_=128, slots=C, ns=64, bits=8, g=64, c=D,
           s=E, z=F, st=None):
    return L.kv_cache_write(K, V, dt, n, ks, vs, H, D_, slots, ns, bits, g, c, s, z, st, None)


def _read(L, c=A, s=B, z=C, npg=4, ps=16, H=2, D_=128, bits=8, g=64, tab=D, ns=2, mp=3,
          cu=D + 4096, total=7, K=E, V=F, dt=0, st=None):
    return L.kv_cache_read(c, s, z, npg, ps, H, D_, bits, g, tab, ns, mp, cu, total, K, V, dt, st,
                           None)


def test_calls_with_arguments_apart_pass_the_checks(L):
    assert L.fp8_quantize_act(A, 0, 4, 128, B, C, None) == ERR_CUDA
    assert L.fp8_quantize_weight(A, 2, 4, 128, B, C, None) == ERR_CUDA
    assert _linear(L) == _linear(L, R=F) == ERR_CUDA
    assert _write(L) == ERR_CUDA
    assert _read(L) == ERR_CUDA


@pytest.mark.parametrize("name", ["fp8_quantize_act", "fp8_quantize_weight"])
def test_quantizer_outputs_may_not_overlap(L, name):
    f = getattr(L, name)
    n, d = 300, 256                                    # 153600 bytes of X, 76800 of codes, 2400 of scales
    sc = 4 * (2 * n if name.endswith("act") else 6)
    assert f(A, 0, n, d, A, C, None) == ERR_ARG        # in place
    assert f(A, 0, n, d, A + 2 * n * d - 16, C, None) == ERR_ARG
    assert f(A, 0, n, d, A + 2 * n * d, C, None) == ERR_CUDA          # next to it
    assert f(A, 1, n, d, A + 2 * n * d, C, None) == ERR_ARG           # fp32: twice as long
    assert f(A, 0, n, d, A - n * d, C, None) == ERR_CUDA
    assert f(A, 0, n, d, A - n * d + 16, C, None) == ERR_ARG
    assert f(A, 0, n, d, B, A + 4, None) == ERR_ARG
    assert f(A, 0, n, d, B, B + n * d - 4, None) == ERR_ARG
    assert f(A, 0, n, d, B, B - sc, None) == ERR_CUDA
    assert f(A, 0, n, d, B, B - sc + 4, None) == ERR_ARG


def test_layer_output_may_overlap_nothing_but_a_residual_that_is_it(L):
    n, d, o = 40, 256, 512
    y = 2 * n * o

    def lin(**kw):
        return _linear(L, n=n, d=d, o=o, **kw)

    assert lin(R=E) == ERR_CUDA                        # in place
    assert lin(R=E + 16) == lin(R=E + y - 16) == lin(R=E - 16) == lin(R=E - y + 16) == ERR_ARG
    assert lin(R=E + y) == lin(R=E - y) == ERR_CUDA
    assert lin(R=E + y, dt=1) == ERR_ARG               # fp32: twice as long
    for at, size in (("X", n * d), ("W", o * d), ("sx", 4 * 2 * n), ("sw", 4 * 2 * 4)):
        base = dict(X=A, W=C, sx=B, sw=D)[at]
        assert lin(Y=base) == lin(Y=base - y + 16) == ERR_ARG, at
        assert lin(Y=base + (size + 15) // 16 * 16) == lin(Y=base - y) == ERR_CUDA, at
        assert lin(Y=base + (size - 1) // 16 * 16) == ERR_ARG, at


def test_cache_and_its_tokens_may_not_overlap(L):
    n, width = 4, 256
    for bits in (4, 8):
        plane = 2 * 64 * width * bits // 8
        for base, size in ((D, plane), (E, 2 * 64 * 4 * 2), (F, 2 * 64 * 4 * 2)):
            assert _write(L, bits=bits, K=base) == _write(L, bits=bits, V=base + size - 16) == ERR_ARG
            assert _write(L, bits=bits, slots=base + size - 8) == ERR_ARG
            assert _write(L, bits=bits, K=base + size) == ERR_CUDA
            assert _write(L, bits=bits, V=base - 2 * n * width) == ERR_CUDA
            assert _write(L, bits=bits, V=base - 2 * n * width, dt=1) == ERR_ARG
            assert _write(L, bits=bits, V=base - 2 * n * width, vs=264) == ERR_ARG
        out = 7 * width * 2
        for base, size in ((A, plane), (B, 2 * 64 * 4 * 2), (C, 2 * 64 * 4 * 2)):
            assert _read(L, bits=bits, K=base) == _read(L, bits=bits, V=base + size - 16) == ERR_ARG
            assert _read(L, bits=bits, K=base + size) == _read(L, bits=bits, V=base - out) == ERR_CUDA
    assert _read(L, V=E) == _read(L, V=E + out - 16) == _read(L, K=F + 16) == ERR_ARG
    assert _read(L, V=E + out) == ERR_CUDA


def test_the_largest_sizes_do_not_wrap(L):
    """Sizes whose bytes pass 64 bits still overlap what they cover."""
    n, o = (1 << 31) - 1, (1 << 31) - 1
    assert _linear(L, n=n, d=16, o=o, X=1 << 50, sx=1 << 51, W=1 << 52, sw=1 << 53, Y=4096, dt=1) == ERR_ARG
    assert _write(L, n=n, ks=1 << 31, dt=1, K=4096) == _write(L, n=n, vs=1 << 31, dt=1, V=4096) == ERR_ARG
