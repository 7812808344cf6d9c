"""The layer where the product of two scales leaves fp32's normal range: what the header promises.

Below 2^-126 the product is off by at most 2^-150, so a term of a block sum up to 128·448² < 2^25
is off by less than 2^-125. Otherwise the tolerance is that of ordinary scales: a block's sum off
by less than 4·33·2^-23 of its Σ|x·w|, 2^-24 each for the product of the scales, the multiply-adds
over nb blocks and the join of 8 partial sums, half a step of Y's type.
"""

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32

# streaming calls of each width, and pairs of CTAs
SHAPES = [(3, 400, 24), (20, 272, 140), (50, 400, 33), (100, 272, 264), (1500, 256, 2056)]


def _np(t):
    return t.detach().cpu().double().numpy()


def _codes(a):
    return torch.from_numpy(np.asarray(a)).float().to(E4M3).cuda()


def _run(lib, xc, xs, wc, ws, dtype):
    return _np(lib.fp8_linear(_codes(xc), torch.from_numpy(xs).cuda(), _codes(wc),
                              torch.from_numpy(ws).cuda(), dtype=dtype))


def _check(lib, xc, xs, wc, ws, dtype):
    Y = _run(lib, xc, xs, wc, ws, dtype)
    ref, mag = ofp8.linear(xc, xs, wc, ws)
    nb = xs.shape[0]
    _, sums = ofp8.linear(xc, np.ones_like(xs), wc, np.ones_like(ws))
    assert np.max(sums) <= nb * 2.0 ** 25
    tol = (4 * 33 * 2.0 ** -23 + (nb + 10) * 2.0 ** -24) * mag + sums * 2.0 ** -150
    fi = torch.finfo(dtype)
    tol = tol + np.maximum(fi.eps / 2 * (np.abs(ref) + tol), fi.smallest_normal * fi.eps / 2)
    err = np.abs(Y - ref)
    assert np.all(err <= tol), (int(np.sum(~(err <= tol))), float(np.nanmax(err / tol)))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ex,ew", [(-60, -56), (-60, -70), (-20, -112), (-99, -30)])
@pytest.mark.parametrize("n,d_in,d_out", SHAPES)
def test_tiny_scales(cuda_lib, n, d_in, d_out, ex, ew, dtype):
    rng = np.random.default_rng(n)
    x = (rng.normal(size=(n, d_in)) * 2.0 ** ex).astype(np.float32)
    w = (rng.normal(size=(d_out, d_in)) * 2.0 ** ew).astype(np.float32)
    xc, xs = ofp8.quantize_act(x)
    wc, ws = ofp8.quantize_weight(w)
    assert np.any(xs.astype(np.float64).max() * ws.astype(np.float64).min() < 2.0 ** -126)
    _check(cuda_lib, xc, xs, wc, ws, dtype)


@pytest.mark.parametrize("n,d_in,d_out", SHAPES)
def test_scales_past_the_range_stay_with_their_tokens_and_channels(cuda_lib, n, d_in, d_out):
    """Products of 2^130 over block sums that are zero (NaN) or not (infinite): the tokens and
    channels of those blocks are not finite, all others are exact."""
    rng = np.random.default_rng(n + 1)
    nb, no = -(-d_in // 128), -(-d_out // 128)
    xc = rng.integers(-3, 4, (n, d_in)).astype(np.float64)
    wc = rng.integers(-3, 4, (d_out, d_in)).astype(np.float64)
    xs, ws = np.ones((nb, n), np.float32), np.ones((no, nb), np.float32)
    big = np.arange(n) % 3 != 1
    xs[1, big], ws[0, 1] = 2.0 ** 70, 2.0 ** 60
    xc[:, 128:256] *= rng.integers(0, 2, (n, 1))       # some tokens' block is all zero
    Y = _run(cuda_lib, xc, xs, wc, ws, F32)
    bad = np.zeros((n, d_out), bool)
    bad[big, :128] = True
    assert np.array_equal(np.isfinite(Y), ~bad)
    zero = np.abs(xc[:, 128:256]).sum(1) == 0
    assert np.all(np.isnan(Y[big & zero, :128])) or not np.any(big & zero)
    ordinary = np.zeros((n, d_out), bool)              # every scale of theirs is 1
    ordinary[~big, 128:] = True
    ref, _ = ofp8.linear(xc, xs, wc, ws)
    assert np.array_equal(Y[ordinary], ref[ordinary])


@pytest.mark.parametrize("n,d_in,d_out", SHAPES)
def test_zero_scales_are_exact(cuda_lib, n, d_in, d_out):
    """Blocks whose scale is zero, or tiny over codes that are zero (as of an all-zero block), add
    nothing."""
    rng = np.random.default_rng(n + 2)
    nb, no = -(-d_in // 128), -(-d_out // 128)
    xc = rng.integers(-3, 4, (n, d_in)).astype(np.float64)
    wc = rng.integers(-3, 4, (d_out, d_in)).astype(np.float64)
    xs, ws = np.ones((nb, n), np.float32), np.full((no, nb), 2.0 ** -30, np.float32)
    kind = rng.permutation(np.arange(n) % 3)
    xs[0, kind == 1] = 0.0
    xs[0, kind == 2] = 2.0 ** -100 / 448.0
    xc[kind == 2, :128] = 0.0
    Y = _run(cuda_lib, xc, xs, wc, ws, F32)
    ref, _ = ofp8.linear(xc, xs, wc, ws)
    assert np.array_equal(Y, ref)
