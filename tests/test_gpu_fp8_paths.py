"""Paths of the 8-bit layer that ordinary random inputs hardly reach: exact ties of the e4m3 codes
and their neighbours, and layers so deep that a CTA fills its table of scale factors several
times.

Codes are compared bit for bit with the nearest e4m3 value to the exact quotient x·448/a (halves
to even). The layer's sums are compared bit for bit too: codes of small integers and power-of-two
scales make every partial sum a multiple of 2^-4 below 2^20, which fp32 holds exactly.
"""

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _np(t):
    return t.detach().cpu().double().numpy()


# the 126 midpoints of neighbouring e4m3 magnitudes, from 2^-10 to 432
_VALUES = torch.arange(127, dtype=torch.uint8).view(E4M3).double()
MIDPOINTS = ((_VALUES[1:] + _VALUES[:-1]) / 2).numpy()


def _step(x, by):
    """The neighbour of each x > 0 that many representable values on."""
    bits = x.view(torch.int32 if x.dtype == F32 else torch.int16)
    return (bits + by).view(x.dtype)


def _rows(a, dtype):
    """[6, 128] values of blocks whose maximum is a: what lies on, just above and just below each
    midpoint (the nearest value of the type where the midpoint has none), in both signs."""
    a = float(torch.tensor(a, dtype=dtype))
    mid = torch.from_numpy(MIDPOINTS * a / 448.0).to(dtype)
    rows = []
    for by in (0, 1, -1):
        x = _step(mid, by)
        for sign in (1.0, -1.0):
            rows.append(torch.cat([torch.tensor([a, 0.0], dtype=dtype), sign * x]))
    return torch.stack(rows)


def _ties(x, a):
    """How many of the values lie on a midpoint: x·448 = m·a, both exact in fp64."""
    return int(np.isin(np.abs(_np(x)) * 448.0, MIDPOINTS * a).sum())


@pytest.mark.parametrize("dtype,powers", [(F16, (-3, 0, 6)), (BF16, (-90, -7, 0, 40, 118)),
                                          (F32, (-90, -7, 0, 40, 118))])
@pytest.mark.parametrize("a,ties", [(448.0, 252), (3.0, 32), (1.0, 32), (21.0, 252)])
def test_codes_of_ties_and_their_neighbours(cuda_lib, a, ties, dtype, powers):
    """a·2^k with a given number of exact ties among the six rows' values."""
    for k in powers:
        top = a * 2.0 ** k
        x = _rows(top, dtype)
        assert _ties(x, top) == ties
        codes, scales = cuda_lib.fp8_quantize_act(x.cuda())
        rc, rs = ofp8.quantize_act(_np(x))
        assert np.array_equal(_np(codes), rc), (k, int(np.sum(_np(codes) != rc)))
        assert np.array_equal(_np(scales), rs.astype(np.float64))
        codes, scales = cuda_lib.fp8_quantize_weight(x.cuda())
        rc, rs = ofp8.quantize_weight(_np(x))
        assert np.array_equal(_np(codes), rc), (k, int(np.sum(_np(codes) != rc)))
        assert np.array_equal(_np(scales), rs.astype(np.float64))


@pytest.mark.parametrize("kind", ["act", "weight"])
def test_codes_of_16_bit_values_held_in_fp32(cuda_lib, kind):
    """fp32 inputs that came from bf16 have thousands of ties; their codes are those of the bf16
    inputs, and the oracle's."""
    g = torch.Generator().manual_seed(4)
    x = (torch.randn(130, 1040, generator=g) * torch.exp(torch.randn(1040, generator=g))).to(BF16)
    f = cuda_lib.fp8_quantize_act if kind == "act" else cuda_lib.fp8_quantize_weight
    a, b = f(x.cuda()), f(x.float().cuda())
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
    rc, _ = (ofp8.quantize_act if kind == "act" else ofp8.quantize_weight)(_np(x))
    assert np.array_equal(_np(b[0]), rc)


@pytest.mark.parametrize("n,d_in,d_out,per_fill", [
    # A cluster has at most 8 CTAs, so each takes at least d_in / 1024 blocks, and its table holds
    # the factors of `per_fill` blocks: 32 for up to 32 tokens, 16 for more.
    (1, 40000, 24, 32),          # 313 blocks: 39 per CTA at least
    (16, 65536, 130, 32),        # 512: 64, filled twice to the last entry
    (20, 40000, 140, 32),
    (32, 65536, 17, 32),
    (50, 20000, 260, 16),        # 157: 19
    (64, 65536, 33, 16),         # four times
    (100, 20000, 24, 16),
    (128, 65536, 136, 16),
    (200, 33296, 120, 16),       # two tiles of tokens
])
def test_deep_layers_refill_their_factors(cuda_lib, n, d_in, d_out, per_fill):
    nb, no = -(-d_in // 128), -(-d_out // 128)
    assert nb // 8 > per_fill
    g = torch.Generator().manual_seed(n + d_in)
    x8 = torch.randint(-3, 4, (n, d_in), generator=g).float().to(E4M3)
    w8 = torch.randint(-3, 4, (d_out, d_in), generator=g).float().to(E4M3)
    sx = 2.0 ** torch.randint(-2, 2, (nb, n), generator=g).float()
    sw = 2.0 ** torch.randint(-2, 2, (no, nb), generator=g).float()
    R = torch.randint(-8, 9, (n, d_out), generator=g).float()
    Y = cuda_lib.fp8_linear(x8.cuda(), sx.cuda(), w8.cuda(), sw.cuda(), R=R.cuda(), dtype=F32)
    ref, mag = ofp8.linear(_np(x8), sx.numpy(), _np(w8), sw.numpy(), R=_np(R))
    assert np.max(mag) + 8 < 2.0 ** 20                 # every partial sum is exact in fp32
    assert np.array_equal(_np(Y), ref)
